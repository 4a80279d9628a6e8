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
    for (int i = threadIdx.x; i < padded; i += kRankThreads)
        keys[i] = i < rows ? key_of(token[i], vocab, ignore_index) : 0xffffffffu;
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
// the digits by block, one scan over all counts and a stable move.
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortWaves = 4, kSortRounds = 16;  // a wave takes 16 x 64 keys in a row
constexpr int kSortBlock = kSortWaves * kSortRounds * 64;

// The keys (and their tokens' places) of one pass.
struct Keys {
    const int64_t *token;  // the first pass: made from the tokens
    const uint32_t *keys, *order;
    int64_t vocab, ignore_index;

    __device__ uint32_t key(int64_t i) const
    {
        return token != nullptr ? key_of(token[i], vocab, ignore_index) : keys[i];
    }
    __device__ uint32_t place(int64_t i) const { return token != nullptr ? uint32_t(i) : order[i]; }
};

__global__ __launch_bounds__(kSortWaves * 64) void embed_count_kernel(Keys in, int64_t rows, int shift,
                                                                      uint32_t *counts)
{
    __shared__ uint32_t bins[kDigits];
    bins[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * kSortBlock;
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = first + r * (kSortWaves * 64) + threadIdx.x;
        if (i < rows) atomicAdd(&bins[(in.key(i) >> shift) & (kDigits - 1)], 1u);  // whole numbers: any order
    }
    __syncthreads();
    counts[int64_t(threadIdx.x) * gridDim.x + blockIdx.x] = bins[threadIdx.x];
}

// counts[digit][block] becomes the number of keys before it, by one workgroup.
constexpr int kScanThreads = 1024, kScanEach = 8;

__global__ __launch_bounds__(kScanThreads) void embed_scan_kernel(uint32_t *counts, int64_t n)
{
    __shared__ uint32_t sums[kScanThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    for (int64_t base = 0; base < n; base += kScanThreads * kScanEach) {
        const int64_t at = base + threadIdx.x * kScanEach;
        uint32_t v[kScanEach], sum = 0;
#pragma unroll
        for (int e = 0; e < kScanEach; ++e) {
            v[e] = at + e < n ? counts[at + e] : 0;
            sum += v[e];
        }
        uint32_t up = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(up, d);
            if (lane >= d) up += o;
        }
        if (lane == 63) sums[wave] = up;
        __syncthreads();
        uint32_t mine = before + up - sum, all = 0;
        for (int w = 0; w < kScanThreads / 64; ++w) {
            if (w < wave) mine += sums[w];
            all += sums[w];
        }
#pragma unroll
        for (int e = 0; e < kScanEach; ++e) {
            if (at + e < n) counts[at + e] = mine;
            mine += v[e];
        }
        before += all;
        __syncthreads();
    }
}

__global__ __launch_bounds__(kSortWaves * 64) void embed_move_kernel(Keys in, int64_t rows, int shift,
                                                                     const uint32_t *counts, uint32_t *keys,
                                                                     uint32_t *order)
{
    __shared__ uint32_t bins[kSortWaves][kDigits];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int w = 0; w < kSortWaves; ++w) bins[w][threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * kSortBlock + wave * (kSortRounds * 64);
    uint32_t key[kSortRounds], at[kSortRounds];
    // a key's place among its wave's keys of the same digit: those of earlier
    // rounds, then those of lower lanes
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = first + r * 64 + lane;
        const bool valid = i < rows;
        key[r] = valid ? in.key(i) : 0;
        const uint32_t digit = (key[r] >> shift) & (kDigits - 1);
        uint64_t same = __ballot(valid);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
            const uint64_t set = __ballot((digit >> b) & 1);
            same &= (digit >> b) & 1 ? set : ~set;
        }
        const uint32_t lower = uint32_t(__popcll(same & ((uint64_t(1) << lane) - 1)));
        at[r] = valid ? bins[wave][digit] + lower : 0;
        // (a wave's LDS accesses are served in their order)
        asm volatile("" ::: "memory");
        if (valid && lower == 0) bins[wave][digit] += uint32_t(__popcll(same));
        asm volatile("" ::: "memory");
    }
    __syncthreads();
    // where each wave's keys of a digit begin
    {
        uint32_t sum = counts[int64_t(threadIdx.x) * gridDim.x + blockIdx.x];
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t n = bins[w][threadIdx.x];
            bins[w][threadIdx.x] = sum;
            sum += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = first + r * 64 + lane;
        if (i >= rows) continue;
        const uint32_t to = bins[wave][(key[r] >> shift) & (kDigits - 1)] + at[r];
        keys[to] = key[r];
        order[to] = in.place(i);
    }
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------

constexpr int kSlab = 512;     // columns of a wave: 8 a lane
constexpr int kSumRows = 4;    // rows in flight a wave
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
    int32_t accumulate;
};

template <class O>
__device__ inline void write_row(O *dw, int col, int cols, const float (&sum)[8], const float (&old)[8], float scale,
                                 int accumulate)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = sum[e] * scale;
        if (accumulate) v[e] += old[e];
    }
    store8(dw, col, cols, v);
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
    float zero[8] = {};
    for (int r = 0; r < n; ++r) {
        if (!((empty >> r) & 1)) continue;
        O *row = dw + (v0 + r) * dw_stride;
        for (int64_t col = lane * 8; col < a.hidden; col += kSlab) store8(row, int(col), a.hidden, zero);
    }
}

// Adds up a block's rows, 512 columns of them.
template <class G, class O>
__device__ inline void sum_unit(const SumArgs &a, int64_t unit, int lane, const G *dy, int64_t dy_stride, O *dw,
                                int64_t dw_stride)
{
    const int64_t block = unit / a.slabs;
    const int col = int(unit - block * a.slabs) * kSlab + lane * 8;
    const bool active = col < a.hidden;
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
        for (int i = 0; i < n; i += kSumRows) {
            float row[kSumRows][8], old[kSumRows][8];
            bool last[kSumRows], whole[kSumRows];
            uint32_t k[kSumRows];
#pragma unroll
            for (int r = 0; r < kSumRows; ++r) {
                k[r] = i + r < n ? uint32_t(__builtin_amdgcn_readlane(int(key), i + r)) : none;
                if (k[r] == none) continue;
                const int64_t t = uint32_t(__builtin_amdgcn_readlane(int(place), i + r));
                if (active) load8(dy + t * dy_stride, col, a.hidden, row[r]);
            }
            // the sums that end here whole, and what they are added to
#pragma unroll
            for (int r = 0; r < kSumRows; ++r) {
                last[r] = whole[r] = false;
                if (k[r] == none) continue;
                const bool at_end = base + i + r + 1 == end;
                last[r] = at_end || uint32_t(__builtin_amdgcn_readlane(int(after), i + r)) != k[r];
                whole[r] = last[r] && k[r] != previous && !(at_end && next == k[r]);
                if (whole[r] && a.accumulate && active) load8(dw + k[r] * dw_stride, col, a.hidden, old[r]);
            }
#pragma unroll
            for (int r = 0; r < kSumRows; ++r) {
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
                    write_row(dw + k[r] * dw_stride, col, a.hidden, sum, old[r], a.scale, a.accumulate);
                } else {
                    vec<float, 8> o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = sum[e];
                    *(vec<float, 8> *)(a.parts + (2 * block + (from_before ? 0 : 1)) * a.pitch + col) = o;
                }
            }
        }
    }
}

template <class G, class O>
__global__ __launch_bounds__(kSumWaves * 64) void embed_sum_kernel(SumArgs a, const G *dy, int64_t dy_stride, O *dw,
                                                                   int64_t dw_stride)
{
    const int lane = threadIdx.x & 63;
    for (int64_t u = int64_t(blockIdx.x) * kSumWaves + uniform(threadIdx.x >> 6); u < a.units + a.clear_units;
         u += int64_t(gridDim.x) * kSumWaves) {
        if (u < a.units)
            sum_unit(a, u, lane, dy, dy_stride, dw, dw_stride);
        else
            clear_unit(a, u - a.units, lane, dw, dw_stride);
    }
}

// The sums of tokens that lie in several blocks: a workgroup for each block in
// which such a token begins, its waves a contiguous share of the parts each.
template <class O>
__device__ inline void join_unit(const SumArgs &a, int64_t unit, float (*shares)[kSlab], O *dw, int64_t dw_stride)
{
    const int64_t block = unit / a.slabs;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t begin = block * a.block, end = begin + a.block;
    if (end >= a.rows) return;
    const uint32_t key = a.sorted[end];
    if (key == uint32_t(a.vocab) || a.sorted[end - 1] != key || (begin > 0 && a.sorted[begin - 1] == key)) return;
    const int col = int(unit - block * a.slabs) * kSlab + lane * 8;
    const bool active = col < a.hidden;
    const int64_t until = end + lower_bound(a.sorted + end, a.rows - end, key + 1);
    const int64_t blocks = (until - 1) / a.block - block + 1;  // with parts
    const int64_t share = (blocks + kSumWaves - 1) / kSumWaves;
    const int64_t from = wave * share, to = from + share < blocks ? from + share : blocks;
    float sum[8] = {};
    if (active) {
#pragma unroll 8
        for (int64_t b = from; b < to; ++b) {
            const vec<float, 8> p =
                *(const vec<float, 8> *)(a.parts + (2 * (block + b) + (b == 0 ? 1 : 0)) * a.pitch + col);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += p[e];
        }
    }
    __syncthreads();  // the workgroup's unit before this one is done with the shares
#pragma unroll
    for (int e = 0; e < 8; ++e) shares[wave][lane * 8 + e] = sum[e];
    __syncthreads();
    if (wave != 0 || !active) return;
    for (int w = 1; w < kSumWaves; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += shares[w][lane * 8 + e];
    float old[8] = {};
    if (a.accumulate) load8(dw + key * dw_stride, col, a.hidden, old);
    write_row(dw + key * dw_stride, col, a.hidden, sum, old, a.scale, a.accumulate);
}

template <class O>
__global__ __launch_bounds__(kSumWaves * 64) void embed_join_kernel(SumArgs a, O *dw, int64_t dw_stride)
{
    __shared__ float shares[kSumWaves][kSlab];
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) join_unit(a, u, shares, dw, dw_stride);
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
    int64_t blocks, sort_blocks = 0;
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
            sort_blocks = (rows + kSortBlock - 1) / kSortBlock;
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
            const Keys in = {p == 0 ? token : nullptr, keys[now ^ 1], order[now ^ 1], sum.vocab, ignore_index};
            const int shift = p * kDigitBits;
            const dim3 grid(static_cast<uint32_t>(sort_blocks)), block(kSortWaves * 64);
            hipLaunchKernelGGL(embed_count_kernel, grid, block, 0, stream, in, sum.rows, shift, counts);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            hipLaunchKernelGGL(embed_scan_kernel, dim3(1), dim3(kScanThreads), 0, stream, counts,
                               sort_blocks * kDigits);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            hipLaunchKernelGGL(embed_move_kernel, grid, block, 0, stream, in, sum.rows, shift, counts, keys[now],
                               order[now]);
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
           hidden <= kMaxSize;
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
    plan.sum.accumulate = accumulate;
    if (accumulate) plan.sum.clear_units = 0;
    const int64_t groups =
        std::min((plan.sum.units + plan.sum.clear_units + kSumWaves - 1) / kSumWaves, kMaxGrid);
    const int64_t joins = std::min(plan.sum.units, kMaxGrid);
    return with_type(dy_type, [&](auto gt) {
        return with_type(dw_type, [&](auto ot) {
            using G = decltype(gt);
            using O = decltype(ot);
            hipLaunchKernelGGL((embed_sum_kernel<G, O>), dim3(uint32_t(groups)), dim3(kSumWaves * 64), 0, stream,
                               plan.sum, (const G *)dy, dy_stride, (O *)dw, dw_stride);
            if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
            if (plan.blocks <= 1) return int(ADAM_OK);
            hipLaunchKernelGGL((embed_join_kernel<O>), dim3(uint32_t(joins)), dim3(kSumWaves * 64), 0,
                               stream, plan.sum, (O *)dw, dw_stride);
            return launched();
        });
    });
}

}  // extern "C"
