// The embedding of tokens and its gradient (include/adam_train.h states the
// formulas).
//
// Forward: a gather of rows, 8 elements a thread.  Bound by HBM.
//
// Gradient: the tokens are sorted (stably, so the rows of one token stay in their
// order), and the sorted list is cut into blocks of equal length, whatever the
// tokens: one frequent token keeps no workgroup longer than the others.  A wave
// takes a block and 512 columns, adds up the rows of each token in it, and
// writes the sums that are whole straight into dw; a token that goes on into
// another block leaves a float part for each, which a last kernel adds in their
// order.  No atomics: the sums depend on the tokens alone.
//
// dw without accumulate: the rows that no token names are cleared in the same
// launch, by waves that look their rows up in the sorted list.
#include <hip/hip_runtime.h>

#include <cmath>

#include "octets.h"

namespace train {
namespace {

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

template <class T>
__device__ inline void load8_cached(const T *row, int col, int cols, float (&v)[8])
{
    if (col <= cols - 8) {
        const vec<T, 8> p = *(const typename Loose<T>::type *)(row + col);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = float(p[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = col + e < cols ? float(row[col + e]) : 0.0f;
    }
}

struct Row8 {
    float v[8];
};

// Groups in flight a thread.
constexpr int kEmbedOctets = 2;

template <class W, class Y>
__global__ __launch_bounds__(kBlock) void embed_forward_kernel(const int64_t *token, int64_t rows, const W *w,
                                                               int64_t vocab, int hidden, int64_t w_stride,
                                                               float scale, int64_t ignore_index, Y *y,
                                                               int64_t y_stride)
{
    for_octets<kEmbedOctets, Row8>(
        rows, (int64_t(hidden) + 7) & ~int64_t(7),
        [&](int64_t row, int col) {
            const int64_t t = token[row];
            Row8 in;
            if (t != ignore_index && t >= 0 && t < vocab) {
                // w's rows stay in the caches: a batch names some of them often
                load8_cached(w + t * w_stride, col, hidden, in.v);
#pragma unroll
                for (int e = 0; e < 8; ++e) in.v[e] *= scale;
            } else {
                const float fill = t == ignore_index ? 0.0f : __builtin_nanf("");
#pragma unroll
                for (int e = 0; e < 8; ++e) in.v[e] = fill;
            }
            return in;
        },
        [&](int64_t row, int col, Row8 &in) { store8(y + row * y_stride, col, hidden, in.v); });
}

// ---------------------------------------------------------------------------
// Sorting
// ---------------------------------------------------------------------------

// A token's key: itself, or `vocab` (behind all others) where it adds nothing.
__device__ inline uint32_t key_of(int64_t t, int64_t vocab, int64_t ignore_index)
{
    return t == ignore_index || t < 0 || t >= vocab ? uint32_t(vocab) : uint32_t(t);
}

// Up to kRankRows tokens: each one's place is the count of the keys that come
// before it, 2 instructions a pair: 64 tokens a workgroup, whose 16 waves share
// the keys out among them.
constexpr int kRankRows = 16384, kRankThreads = 1024, kRankWaves = kRankThreads / 64;

__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(const int64_t *token, int rows, int64_t vocab,
                                                                  int64_t ignore_index, uint32_t *sorted,
                                                                  uint32_t *order)
{
    __shared__ __attribute__((aligned(16))) uint32_t keys[kRankRows];
    __shared__ int counts[kRankWaves][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int padded = (rows + 63) & ~63;
    constexpr int kAtOnce = 8;
    for (int base = threadIdx.x; base < padded; base += kRankThreads * kAtOnce) {
        int64_t t[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) t[e] = base + e * kRankThreads < rows ? token[base + e * kRankThreads] : -1;
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const int i = base + e * kRankThreads;
            if (i < padded) keys[i] = i < rows ? key_of(t[e], vocab, ignore_index) : 0xffffffffu;
        }
    }
    __syncthreads();
    const int first = blockIdx.x * 64;
    const uint32_t own = keys[first + lane];
    const int groups = padded >> 6;
    int count = 0;
    for (int g = wave; g < groups; g += kRankWaves) {
        const u32x4 *at = (const u32x4 *)(keys + g * 64);
        if (g != int(blockIdx.x)) {
            // keys of earlier tokens come first where equal too
            const uint32_t limit = own + (g < int(blockIdx.x) ? 1 : 0);
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const u32x4 k = at[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) count += k[e] < limit ? 1 : 0;
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const u32x4 k = at[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) count += k[e] < own + (i * 4 + e < lane ? 1 : 0) ? 1 : 0;
            }
        }
    }
    counts[wave][lane] = count;
    __syncthreads();
    if (wave == 0 && first + lane < rows) {
        int at = 0;
#pragma unroll
        for (int w = 0; w < kRankWaves; ++w) at += counts[w][lane];
        sorted[at] = own;
        order[at] = uint32_t(first + lane);
    }
}

// More tokens: passes over 8 bits of the key, the lowest first, each a count of
// the digits by block and a stable move, whose workgroups add up the counts of the
// blocks before theirs by themselves (at most 256 blocks of 1 KiB: less than a
// launch more).
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortWaves = 4, kSortThreads = kSortWaves * 64;
constexpr int kLeastSortBlock = 1024, kMostSortBlocks = 256;
static_assert(kDigits == kSortThreads, "a thread for each digit");

// The keys (and their tokens' places) of one pass.
struct Keys {
    const int64_t *token;  // the first pass: made from the tokens
    const uint32_t *keys, *order;
    int64_t vocab, ignore_index, rows, block;
    int shift;

    __device__ uint32_t key(int64_t i) const
    {
        return token != nullptr ? key_of(token[i], vocab, ignore_index) : keys[i];
    }
    __device__ uint32_t place(int64_t i) const { return token != nullptr ? uint32_t(i) : order[i]; }
    __device__ uint32_t digit(uint32_t k) const { return (k >> shift) & (kDigits - 1); }
};

__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(Keys in, uint32_t *counts)
{
    __shared__ uint32_t bins[kDigits];
    bins[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * in.block;
#pragma unroll 4
    for (int64_t o = threadIdx.x; o < in.block; o += kSortThreads)
        if (first + o < in.rows) atomicAdd(&bins[in.digit(in.key(first + o))], 1u);  // whole numbers: any order
    __syncthreads();
    counts[blockIdx.x * kDigits + threadIdx.x] = bins[threadIdx.x];
}

__global__ __launch_bounds__(kSortThreads) void embed_move_kernel(Keys in, const uint32_t *counts, uint32_t *keys,
                                                                  uint32_t *order)
{
    __shared__ uint32_t bins[kSortWaves][kDigits], sums[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int w = 0; w < kSortWaves; ++w) bins[w][threadIdx.x] = 0;
    // the digit's keys in earlier blocks, and in all
    uint32_t before = 0, all = 0;
#pragma unroll 16
    for (uint32_t b = 0; b < gridDim.x; ++b) {
        const uint32_t n = counts[b * kDigits + threadIdx.x];
        before += b < blockIdx.x ? n : 0;
        all += n;
    }
    uint32_t up = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(up, d);
        if (lane >= d) up += o;
    }
    if (lane == 63) sums[wave] = up;
    __syncthreads();
    uint32_t at = up - all + before;  // and those of lower digits
    for (int w = 0; w < wave; ++w) at += sums[w];
    // a wave takes a quarter of the block in a row: its counts, then where each
    // wave's keys of a digit begin
    const int64_t part = in.block / kSortWaves, first = int64_t(blockIdx.x) * in.block + wave * part;
    for (int64_t o = 0; o < part; o += 256) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = first + o + e * 64 + lane;
            if (i < in.rows) atomicAdd(&bins[wave][in.digit(in.key(i))], 1u);
        }
    }
    __syncthreads();
    for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t n = bins[w][threadIdx.x];
        bins[w][threadIdx.x] = at;
        at += n;
    }
    __syncthreads();
    for (int64_t o = 0; o < part; o += 256) {
        uint32_t key[4], place[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = first + o + e * 64 + lane;
            key[e] = i < in.rows ? in.key(i) : 0;
            place[e] = i < in.rows ? in.place(i) : 0;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool valid = first + o + e * 64 + lane < in.rows;
            const uint32_t digit = in.digit(key[e]);
            uint64_t same = __ballot(valid);
#pragma unroll
            for (int b = 0; b < kDigitBits; ++b) {
                const uint64_t set = __ballot((digit >> b) & 1);
                same &= (digit >> b) & 1 ? set : ~set;
            }
            const uint32_t lower = uint32_t(__popcll(same & ((uint64_t(1) << lane) - 1)));
            const uint32_t to = bins[wave][digit] + lower;
            // (a wave's LDS accesses are served in their order)
            asm volatile("" ::: "memory");
            if (valid && lower == 0) bins[wave][digit] += uint32_t(__popcll(same));
            asm volatile("" ::: "memory");
            if (valid) {
                keys[to] = key[e];
                order[to] = place[e];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------

constexpr int kSlab = 512;  // columns of a wave: 8 a lane
constexpr int kSumWaves = 4;

struct SumArgs {
    const uint32_t *sorted, *order;
    int64_t rows, vocab;
    int32_t hidden, slabs;
    int32_t block;          // sorted rows of a unit
    int64_t units;          // blocks * slabs, the waves that add
    int32_t clear_rows;     // rows of dw of a unit that clears
    int64_t clear_units;    // 0 where dw is added to
    float *parts;           // two a block: the sum that began before it, the one that goes on behind it
    int64_t pitch;          // of a part
    float scale;
};

// A lane's 8 columns of a slab: 8 in a row where both matrices are 16-bit, else 4
// and 4 more 256 on, so that a wave's accesses of floats are whole lines.
template <class G, class O>
struct Columns {
    static constexpr bool kSplit = sizeof(G) == 4 || sizeof(O) == 4;
    int first, second, count;  // of the matrix

    __device__ Columns(int slab, int lane, int hidden) : count(hidden)
    {
        first = slab * kSlab + lane * (kSplit ? 4 : 8);
        second = first + (kSplit ? 256 : 4);
    }
    __device__ bool any() const { return first < count; }

    template <class T>
    static __device__ void load4(const T *row, int col, int cols, float *v)
    {
        if (col <= cols - 4) {
            typedef vec<T, 4> loose __attribute__((aligned(sizeof(T))));
            const vec<T, 4> p = __builtin_nontemporal_load((const loose *)(row + col));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = float(p[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = col + e < cols ? float(row[col + e]) : 0.0f;
        }
    }
    template <class T>
    static __device__ void store4(T *row, int col, int cols, const float *v)
    {
        if (col <= cols - 4) {
            typedef vec<T, 4> loose __attribute__((aligned(sizeof(T))));
            loose p;
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = T(v[e]);
            __builtin_nontemporal_store(p, (loose *)(row + col));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < cols) row[col + e] = T(v[e]);
        }
    }
    template <class T>
    __device__ void load(const T *row, float (&v)[8]) const
    {
        if (!kSplit) {
            load8(row, first, count, v);
        } else {
            load4(row, first, count, v);
            load4(row, second, count, v + 4);
        }
    }
    template <class T>
    __device__ void store(T *row, float (&v)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm("" : "+v"(v[e]));  // rounded to float first, then to T
        if (!kSplit) {
            store8(row, first, count, v);
        } else {
            store4(row, first, count, v);
            store4(row, second, count, v + 4);
        }
    }
};

// A sum into its row of dw.
template <bool ACCUMULATE, class G, class O>
__device__ inline void write_row(const Columns<G, O> &c, O *dw, const float (&sum)[8], const float (&old)[8],
                                 float scale)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = sum[e] * scale;
        if (ACCUMULATE) v[e] += old[e];
    }
    c.store(dw, v);
}

// The first position of the sorted keys whose key is at least `key`.
__device__ inline int64_t lower_bound(const uint32_t *sorted, int64_t n, uint32_t key)
{
    int64_t lo = 0;
    while (n > 0) {
        const int64_t half = n >> 1;
        const bool below = sorted[lo + half] < key;
        lo = below ? lo + half + 1 : lo;
        n = below ? n - half - 1 : half;
    }
    return lo;
}

// Clears those of a unit's rows of dw that no token names.
template <class O>
__device__ inline void clear_unit(const SumArgs &a, int64_t unit, int lane, O *dw, int64_t dw_stride)
{
    const int64_t v0 = unit * a.clear_rows;
    const int n = int(a.vocab - v0 < a.clear_rows ? a.vocab - v0 : a.clear_rows);
    bool named = true;
    if (lane < n) {
        const uint32_t v = uint32_t(v0 + lane);
        const int64_t at = lower_bound(a.sorted, a.rows, v);
        named = at < a.rows && a.sorted[at] == v;
    }
    const uint64_t empty = __ballot(!named);
    constexpr int kEach = 16 / sizeof(O);
    const bool lines = (dw_stride * int64_t(sizeof(O))) % 128 == 0;
    for (int r = 0; r < n; ++r) {
        if (!((empty >> r) & 1)) continue;
        // whole 16-byte words, and what lies before the first and behind the last
        O *row = dw + (v0 + r) * dw_stride;
        const int64_t head = int64_t((16 - (uintptr_t(row) & 15)) & 15) / int64_t(sizeof(O));
        const int64_t before = head < a.hidden ? head : a.hidden;
        const int64_t words = (a.hidden - before) / kEach, behind = before + words * kEach;
        if (lane < before) row[lane] = O(0.0f);
        u32x4 *to = (u32x4 *)(row + before);
        if (lines) {
            for (int64_t w = lane; w < words; w += 64) __builtin_nontemporal_store(u32x4(0), to + w);
        } else {
            // through the caches, which join the ends of rows that share a line
            for (int64_t w = lane; w < words; w += 64) to[w] = u32x4(0);
        }
        if (behind + lane < a.hidden) row[behind + lane] = O(0.0f);
    }
}

// Adds up a block's rows, 512 columns of them.
template <bool ACCUMULATE, class G, class O>
__device__ inline void sum_unit(const SumArgs &a, int64_t unit, int lane, const G *dy, int64_t dy_stride, O *dw,
                                int64_t dw_stride)
{
    constexpr int kRows = ACCUMULATE ? 4 : 8;  // in flight
    const int64_t block = unit / a.slabs;
    const Columns<G, O> columns(int(unit - block * a.slabs), lane, a.hidden);
    const bool active = columns.any();
    const int64_t begin = block * a.block;
    const int64_t end = begin + a.block < a.rows ? begin + a.block : a.rows;
    const uint32_t none = uint32_t(a.vocab);
    const uint32_t previous = begin > 0 ? a.sorted[begin - 1] : none;
    const uint32_t next = end < a.rows ? a.sorted[end] : none;
    uint32_t current = none;
    bool from_before = false;
    float sum[8] = {};
    for (int64_t base = begin; base < end; base += 64) {
        const int n = int(end - base < 64 ? end - base : 64);
        uint32_t key = none, place = 0, after = none;
        if (lane < n) {
            key = a.sorted[base + lane];
            place = a.order[base + lane];
            after = base + lane + 1 < a.rows ? a.sorted[base + lane + 1] : none;
        }
        for (int i = 0; i < n; i += kRows) {
            float row[kRows][8], old[ACCUMULATE ? kRows : 1][8];
            bool last[kRows], whole[kRows];
            uint32_t k[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                k[r] = i + r < n ? uint32_t(__builtin_amdgcn_readlane(int(key), i + r)) : none;
                if (k[r] == none) continue;
                const int64_t t = uint32_t(__builtin_amdgcn_readlane(int(place), i + r));
                if (active) columns.load(dy + t * dy_stride, row[r]);
            }
            // the sums that end here whole, and what they are added to
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                last[r] = whole[r] = false;
                if (k[r] == none) continue;
                const bool at_end = base + i + r + 1 == end;
                last[r] = at_end || uint32_t(__builtin_amdgcn_readlane(int(after), i + r)) != k[r];
                whole[r] = last[r] && k[r] != previous && !(at_end && next == k[r]);
                if (ACCUMULATE && whole[r] && active) columns.load(dw + k[r] * dw_stride, old[ACCUMULATE ? r : 0]);
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (k[r] == none) continue;
                if (k[r] != current) {
                    current = k[r];
                    from_before = current == previous;
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += row[r][e];
                if (!last[r] || !active) continue;
                if (whole[r]) {
                    write_row<ACCUMULATE>(columns, dw + k[r] * dw_stride, sum, old[ACCUMULATE ? r : 0], a.scale);
                } else {
                    float *part = a.parts + (2 * block + (from_before ? 0 : 1)) * a.pitch;
                    *(f32x4 *)(part + columns.first) = f32x4{sum[0], sum[1], sum[2], sum[3]};
                    if (columns.second < a.pitch)
                        *(f32x4 *)(part + columns.second) = f32x4{sum[4], sum[5], sum[6], sum[7]};
                }
            }
        }
    }
}

template <bool ACCUMULATE, class G, class O>
__global__ __launch_bounds__(kSumWaves * 64) void embed_sum_kernel(SumArgs a, const G *dy, int64_t dy_stride, O *dw,
                                                                   int64_t dw_stride)
{
    const int lane = threadIdx.x & 63;
    for (int64_t u = int64_t(blockIdx.x) * kSumWaves + uniform(threadIdx.x >> 6); u < a.units + a.clear_units;
         u += int64_t(gridDim.x) * kSumWaves) {
        if (u < a.units)
            sum_unit<ACCUMULATE>(a, u, lane, dy, dy_stride, dw, dw_stride);
        else
            clear_unit(a, u - a.units, lane, dw, dw_stride);
    }
}

// The sums of tokens that lie in several blocks: a workgroup for each block in
// which such a token begins and every fourth slab, its waves a contiguous share of
// the parts each.
template <bool ACCUMULATE, class O>
__device__ inline void join_block(const SumArgs &a, int64_t block, int first, int step, float (*shares)[kSlab], O *dw,
                                  int64_t dw_stride)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t begin = block * a.block, end = begin + a.block;
    if (end >= a.rows) return;
    const uint32_t key = a.sorted[end];
    if (key == uint32_t(a.vocab) || a.sorted[end - 1] != key || (begin > 0 && a.sorted[begin - 1] == key)) return;
    const int64_t until = end + lower_bound(a.sorted + end, a.rows - end, key + 1);
    const int64_t blocks = (until - 1) / a.block - block + 1;  // with parts
    const int64_t share = (blocks + kSumWaves - 1) / kSumWaves;
    const int64_t from = wave * share, to = from + share < blocks ? from + share : blocks;
    for (int slab = first; slab < a.slabs; slab += step) {
        const Columns<float, O> columns(slab, lane, a.hidden);
        float sum[8] = {};
        if (columns.any()) {
#pragma unroll 8
            for (int64_t b = from; b < to; ++b) {
                const float *part = a.parts + (2 * (block + b) + (b == 0 ? 1 : 0)) * a.pitch;
                const f32x4 x = *(const f32x4 *)(part + columns.first);
                const f32x4 y = columns.second < a.pitch ? *(const f32x4 *)(part + columns.second) : f32x4(0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum[e] += x[e];
                    sum[4 + e] += y[e];
                }
            }
        }
        __syncthreads();  // the slab before this one is done with the shares
#pragma unroll
        for (int e = 0; e < 8; ++e) shares[wave][e * 64 + lane] = sum[e];
        __syncthreads();
        if (wave != 0 || !columns.any()) continue;
        for (int w = 1; w < kSumWaves; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += shares[w][e * 64 + lane];
        float old[8] = {};
        if (ACCUMULATE) columns.load(dw + key * dw_stride, old);
        write_row<ACCUMULATE>(columns, dw + key * dw_stride, sum, old, a.scale);
    }
}

template <bool ACCUMULATE, class O>
__global__ __launch_bounds__(kSumWaves * 64) void embed_join_kernel(SumArgs a, int64_t blocks, O *dw,
                                                                    int64_t dw_stride)
{
    __shared__ float shares[kSumWaves][kSlab];
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x)
        join_block<ACCUMULATE>(a, b, blockIdx.y, gridDim.y, shares, dw, dw_stride);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int bits_of(int64_t v)
{
    int n = 0;
    for (; v > 0; v >>= 1) ++n;
    return n;
}

// The gradient's sizes and its workspace.
struct EmbedPlan {
    SumArgs sum = {};
    uint32_t *keys[2], *order[2], *counts = nullptr;
    int64_t blocks, sort_block = 0, sort_blocks = 0;
    int passes = 0;
    int64_t bytes;

    EmbedPlan(int64_t rows, int64_t vocab, int64_t hidden, void *workspace)
    {
        sum.rows = rows;
        sum.vocab = vocab;
        sum.hidden = int32_t(hidden);
        sum.slabs = int32_t((hidden + kSlab - 1) / kSlab);
        // blocks of 16 to 256 rows, longer while 4096 waves stay
        sum.block = 16;
        while (sum.block < 256 && (rows / (2 * sum.block)) * sum.slabs >= 4096) sum.block *= 2;
        blocks = (rows + sum.block - 1) / sum.block;
        sum.units = blocks * sum.slabs;
        sum.clear_rows = int32_t(std::min<int64_t>(64, std::max<int64_t>(1, vocab / 8192)));
        sum.clear_units = (vocab + sum.clear_rows - 1) / sum.clear_rows;
        sum.pitch = round_up(hidden, 8);
        Workspace w{(char *)workspace};
        const bool radix = rows > kRankRows;
        for (int i = 0; i < 2; ++i) {
            keys[i] = radix || i == 0 ? w.take<uint32_t>(rows) : nullptr;
            order[i] = radix || i == 0 ? w.take<uint32_t>(rows) : nullptr;
        }
        if (radix) {
            passes = (bits_of(vocab) + kDigitBits - 1) / kDigitBits;
            sort_block = kLeastSortBlock;
            while (sort_block * kMostSortBlocks < rows) sort_block *= 2;
            sort_blocks = (rows + sort_block - 1) / sort_block;
            counts = w.take<uint32_t>(sort_blocks * kDigits);
        }
        if (blocks > 1) sum.parts = w.take<float>(2 * blocks * sum.pitch);
        bytes = w.used;
    }

    int sort(const int64_t *token, int64_t ignore_index, hipStream_t stream)
    {
        int now = 0;
        if (passes == 0) {
            hipLaunchKernelGGL(embed_rank_kernel, dim3(uint32_t((sum.rows + 63) / 64)), dim3(kRankThreads), 0, stream,
                               token, int(sum.rows), sum.vocab, ignore_index, keys[0], order[0]);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
        }
        for (int p = 0; p < passes; ++p) {
            const Keys in = {p == 0 ? token : nullptr, keys[now ^ 1], order[now ^ 1], sum.vocab, ignore_index, sum.rows,
                             sort_block, p * kDigitBits};
            const dim3 grid(static_cast<uint32_t>(sort_blocks)), block(kSortThreads);
            hipLaunchKernelGGL(embed_count_kernel, grid, block, 0, stream, in, counts);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            hipLaunchKernelGGL(embed_move_kernel, grid, block, 0, stream, in, counts, keys[now], order[now]);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            now ^= 1;
        }
        if (passes > 0) now ^= 1;
        sum.sorted = keys[now];
        sum.order = order[now];
        return ADAM_OK;
    }
};

bool embed_sizes(int64_t rows, int64_t vocab, int64_t hidden)
{
    return rows >= 0 && rows <= kMaxProductRows && vocab >= 0 && vocab <= kMaxSize && hidden >= 0 &&
           hidden <= kMaxProductRows;
}

}  // namespace
}  // namespace train

using namespace train;

extern "C" {

int adam_embed_forward(const int64_t *token, int64_t rows, const void *w, adam_dtype w_type, int64_t vocab,
                       int64_t hidden, int64_t w_stride, float scale, int64_t ignore_index, void *y,
                       adam_dtype y_type, int64_t y_stride, hipStream_t stream)
{
    if (!known_type(w_type) || !known_type(y_type)) return ADAM_EINVAL;
    if (!float_type(w_type) || !float_type(y_type)) return ADAM_EDTYPE;
    if (!embed_sizes(rows, vocab, hidden) || !valid_matrix(vocab, hidden, w_stride) ||
        !valid_matrix(rows, hidden, y_stride) || !std::isfinite(scale))
        return ADAM_EINVAL;
    if (rows == 0 || hidden == 0) return ADAM_OK;
    const int wb = dtype_bytes(w_type), yb = dtype_bytes(y_type);
    if (vocab == 0 || token == nullptr || w == nullptr || y == nullptr || !aligned(token, 8) || !aligned(w, wb) ||
        !aligned(y, yb))
        return ADAM_EINVAL;
    const View out = matrix(y, rows, hidden, y_stride, yb);
    if (overlap(out, matrix(w, vocab, hidden, w_stride, wb)) || overlap(out, flat(token, rows * 8)))
        return ADAM_EINVAL;
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return with_type(w_type, [&](auto wt) {
        return with_type(y_type, [&](auto yt) {
            using W = decltype(wt);
            using Y = decltype(yt);
            hipLaunchKernelGGL((embed_forward_kernel<W, Y>), octet_grid(rows, round_up(hidden, 8), kEmbedOctets),
                               dim3(kBlock), 0, stream, token, rows, (const W *)w, vocab, int(hidden), w_stride, scale,
                               ignore_index, (Y *)y, y_stride);
            return launched();
        });
    });
}

int adam_embed_backward_workspace(int64_t rows, int64_t vocab, int64_t hidden, int64_t *bytes)
{
    if (bytes == nullptr || !embed_sizes(rows, vocab, hidden)) return ADAM_EINVAL;
    *bytes = rows == 0 || vocab == 0 || hidden == 0 ? 0 : EmbedPlan(rows, vocab, hidden, nullptr).bytes;
    return ADAM_OK;
}

int adam_embed_backward(const int64_t *token, int64_t rows, const void *dy, adam_dtype dy_type, int64_t dy_stride,
                        float scale, int64_t ignore_index, void *dw, adam_dtype dw_type, int64_t vocab,
                        int64_t hidden, int64_t dw_stride, int32_t accumulate, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream)
{
    if (!known_type(dy_type) || !known_type(dw_type) || (accumulate != 0 && accumulate != 1)) return ADAM_EINVAL;
    if (!float_type(dy_type) || !float_type(dw_type)) return ADAM_EDTYPE;
    if (!embed_sizes(rows, vocab, hidden) || !valid_matrix(rows, hidden, dy_stride) ||
        !valid_matrix(vocab, hidden, dw_stride) || !std::isfinite(scale))
        return ADAM_EINVAL;
    if (hidden == 0 || (rows == 0 && (accumulate || vocab == 0))) return ADAM_OK;
    const int gb = dtype_bytes(dy_type), ob = dtype_bytes(dw_type);
    if (vocab == 0 || dw == nullptr || !aligned(dw, ob) ||
        (rows > 0 && (token == nullptr || dy == nullptr || !aligned(token, 8) || !aligned(dy, gb))))
        return ADAM_EINVAL;
    EmbedPlan plan(rows, vocab, hidden, workspace);
    if (rows > 0 && (workspace == nullptr || workspace_bytes < plan.bytes || !aligned(workspace, 256)))
        return ADAM_EINVAL;
    const View out[2] = {matrix(dw, vocab, hidden, dw_stride, ob), flat(workspace, rows > 0 ? plan.bytes : 0)};
    const View in[2] = {flat(token, rows * 8), matrix(dy, rows, hidden, dy_stride, gb)};
    for (const View &o : out)
        for (const View &i : in)
            if (overlap(o, i)) return ADAM_EINVAL;
    if (overlap(out[0], out[1])) return ADAM_EINVAL;
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    if (rows > 0) {
        const int rc = plan.sort(token, ignore_index, stream);
        if (rc != ADAM_OK) return rc;
    }
    plan.sum.scale = scale;
    if (accumulate) plan.sum.clear_units = 0;
    const int64_t groups =
        std::min((plan.sum.units + plan.sum.clear_units + kSumWaves - 1) / kSumWaves, kMaxGrid);
    const int64_t joins = std::min(plan.blocks, kMaxGrid);
    return with_type(dy_type, [&](auto gt) {
        return with_type(dw_type, [&](auto ot) {
            using G = decltype(gt);
            using O = decltype(ot);
            auto run = [&](auto acc) {
                constexpr bool ACC = decltype(acc)::value;
                hipLaunchKernelGGL((embed_sum_kernel<ACC, G, O>), dim3(uint32_t(groups)), dim3(kSumWaves * 64), 0,
                                   stream, plan.sum, (const G *)dy, dy_stride, (O *)dw, dw_stride);
                if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
                if (plan.blocks <= 1) return int(ADAM_OK);
                hipLaunchKernelGGL((embed_join_kernel<ACC, O>), dim3(uint32_t(joins), uint32_t(std::min(plan.sum.slabs, 4))), dim3(kSumWaves * 64), 0, stream,
                                   plan.sum, plan.blocks, (O *)dw, dw_stride);
                return launched();
            };
            return accumulate ? run(std::true_type()) : run(std::false_type());
        });
    });
}

}  // extern "C"
