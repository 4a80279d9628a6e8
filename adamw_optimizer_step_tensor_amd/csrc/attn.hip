// Attention over packed documents and its gradient (include/adam_train.h states
// the formulas).
//
// A mask of every kind that the header names leaves each query an interval of
// keys, and each key an interval of queries, whose ends do not decrease from row
// to row.  So a workgroup takes a tile of rows of the packed batch, whatever
// documents they belong to ("own" rows: queries in the forward pass and for dq,
// keys for dk and dv), walks the other side's rows ("inner" rows) over the union
// of its rows' intervals, and only tiles that some interval ends in are masked.
//
// The three kernels have one shape.  A wave owns 32 rows.  An inner tile lies in
// LDS; its product with the own rows, by the 32x32x16 instruction with the inner
// rows as first operand, leaves each lane the scores of one own row (lane % 32)
// with 16 inner rows: a row's maximum and sum stay inside two lanes.  The same
// registers, rounded to 16 bits, are the second operand of the next product: its
// k are the inner rows in the order that the lanes hold them, which the
// transposing LDS read of the first operand (the tile again, with its columns as
// rows) follows.  So no score leaves its lane:
//   forward  s = k q^T,                       o^T  += v^T p
//   dq       s = k q^T,   dp = v do^T,        dq^T += k^T ds
//   dk, dv   s = q k^T,   dp = do v^T,        dv^T += do^T p,  dk^T += q^T ds
// The own rows' operands stay in registers for the whole walk.
//
// One document of 16384 rows, 32 heads on 8 of 128, bf16: forward 2.01 to 2.05 ms
// (1.07 PFLOP/s), dq 2.86 to 2.93 (1.13), dk and dv 4.3 to 4.7 (0.94 to 1.02); the
// matrix unit is busy 57% of the forward pass's cycles at 1.73 GHz, the clock that
// its power leaves, and the LDS 29%.  8192 rows of 19 documents: 112, 169 and 283
// us, which the workgroups of the longest documents set.
#include <hip/hip_runtime.h>

#include <cmath>

#include "octets.h"

namespace train {
namespace {

using f32x16 = vec<float, 16>;

constexpr int kOwn = 32;                 // own rows of a wave
constexpr int kAttnWaves = 4, kAttnThreads = kAttnWaves * 64;
constexpr int kOwnTile = kOwn * kAttnWaves;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int64_t kMaxAttnDim = 256, kMaxHeads = 65535;

__device__ inline f32x16 mfma32(vec<bf16, 8> a, vec<bf16, 8> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16 mfma32(vec<f16, 8> a, vec<f16, 8> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

struct Heads {
    void *p;
    int64_t stride, head_stride;

    template <class T>
    __device__ T *at(int head, int64_t row) const
    {
        return (T *)p + head * head_stride + row * stride;
    }
};

struct AttnArgs {
    Heads q, k, v, o, dout, dq, dk, dv;
    float *lse;
    int32_t *flags;  // one a workgroup: its sums are not finite
    float *numbers;  // for each query head and row: lse in units of log 2, and (a plane of them on) delta
    const int32_t *offsets, *prefix;
    const float *slopes;
    int32_t rows, docs, heads, kv_heads, dim, causal, window;
    float scale, softcap;
    int32_t tiles;  // of own rows
    int32_t parts;  // that a long walk for dk and dv is split into, at most
    float *sums;    // of the parts
};

// ---------------------------------------------------------------------------
// The mask
// ---------------------------------------------------------------------------

// Rows lo .. hi - 1 of the other side; none where hi is 0.
struct Span {
    int lo, hi;
};

// The rows of i's document, clamped to the batch whatever the offsets hold.
__device__ inline Span document(const AttnArgs &a, int i, int &doc)
{
    doc = 0;
    if (i >= a.rows) return Span{0, 0};
    if (a.offsets == nullptr) return Span{0, a.rows};
    int lo = 0, n = a.docs + 1;  // the first offset above i
    while (n > 0) {
        const int half = n >> 1;
        const bool below = a.offsets[lo + half] <= i;
        lo = below ? lo + half + 1 : lo;
        n = below ? n - half - 1 : half;
    }
    if (lo == 0 || lo > a.docs) return Span{0, 0};
    doc = lo - 1;
    int begin = a.offsets[doc], end = a.offsets[lo];
    begin = begin < 0 ? 0 : begin;
    end = end > a.rows ? a.rows : end;
    return begin <= i && i < end ? Span{begin, end} : Span{0, 0};
}

__device__ inline int prefix_end(const AttnArgs &a, Span s, int doc)
{
    if (a.prefix == nullptr) return s.lo;
    const int n = a.prefix[doc];
    return n < s.hi - s.lo ? s.lo + (n > 0 ? n : 0) : s.hi;
}

// The keys that query i sees.
__device__ inline Span keys_of(const AttnArgs &a, int i)
{
    int doc;
    Span s = document(a, i, doc);
    if (s.hi == 0 || !a.causal) return s;
    const int p = prefix_end(a, s, doc);
    s.hi = p > i + 1 ? p : i + 1;
    if (a.window > 0 && i - s.lo >= a.window) s.lo = i - a.window + 1;
    return s;
}

// The queries that see key j.
__device__ inline Span queries_of(const AttnArgs &a, int j)
{
    int doc;
    Span s = document(a, j, doc);
    if (s.hi == 0 || !a.causal) return s;
    if (j >= prefix_end(a, s, doc)) s.lo = j;
    if (a.window > 0 && s.hi - j > a.window) s.hi = j + a.window;
    return s;
}

// What a wave's 32 intervals come to.  Both ends grow from row to row, so the
// first and the last row that has one hold the extremes.
struct WaveSpan {
    int lo, hi;          // their union
    int every_lo, every_hi;  // their intersection
    bool any;

    __device__ __attribute__((always_inline)) WaveSpan(Span s)
    {
        const uint64_t has = __ballot(s.hi > 0);
        any = has != 0;
        const int first = any ? __builtin_ctzll(has) : 0;
        const int last = any ? 31 - __builtin_clz(uint32_t(has)) : 0;
        lo = __builtin_amdgcn_readlane(s.lo, first);
        every_hi = __builtin_amdgcn_readlane(s.hi, first);
        every_lo = __builtin_amdgcn_readlane(s.lo, last);
        hi = __builtin_amdgcn_readlane(s.hi, last);
        // (what comes out for rows without an interval is not stored)
    }
};

// The same over the workgroup; `box` holds 4 values a wave.  Inner tiles are walked
// in pairs from lo on: those before `open` or from `close` on may hold hidden pairs.
struct GroupSpan {
    int lo, hi;
    int open, close;

    __device__ __attribute__((always_inline)) GroupSpan(const WaveSpan &w, int wave, int (&box)[4 * kAttnWaves], int pair)
    {
        if ((threadIdx.x & 63) == 0) {
            int *to = box + 4 * wave;
            to[0] = w.any ? w.lo : 0x7fffffff;
            to[1] = w.any ? w.hi : 0;
            to[2] = w.any ? w.every_lo : 0;
            to[3] = w.any ? w.every_hi : 0x7fffffff;
        }
        __syncthreads();
        int l = 0x7fffffff, h = 0, el = 0, eh = 0x7fffffff;
#pragma unroll
        for (int k = 0; k < kAttnWaves; ++k) {
            l = box[4 * k] < l ? box[4 * k] : l;
            h = box[4 * k + 1] > h ? box[4 * k + 1] : h;
            el = box[4 * k + 2] > el ? box[4 * k + 2] : el;
            eh = box[4 * k + 3] < eh ? box[4 * k + 3] : eh;
        }
        lo = uniform(l);
        hi = uniform(h);
        el = uniform(el) - lo;
        eh = uniform(eh) - lo;
        open = el > 0 ? lo + (el + pair - 1) / pair * pair : lo;
        close = eh > 0 ? lo + eh / pair * pair : lo;
        if (open > hi) open = hi;
        if (close < open) close = open;
    }
};

// ---------------------------------------------------------------------------
// Tiles in LDS
// ---------------------------------------------------------------------------

// Rows of DP values (the head dimension rounded up, zeros behind it), `kPitch`
// bytes apart.  The 16-byte chunk c of row r lies in slot c ^ twist(r): the 16
// lanes that a 16-byte read serves at once, which hold one chunk of 16 rows that
// differ in their low 4 bits, and the 4 rows x 64 bytes of the transposing
// reads of 32 lanes, both cover all banks.
template <int DP>
struct Layout {
    static constexpr int kPitch = DP <= 64 ? 128 : DP <= 128 ? 256 : 512;
    static constexpr int kChunks = kPitch / 16;
    static __device__ int twist(int row)
    {
        return kPitch == 128 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
    }
};

// Loads N inner rows of one operand into LDS, from `row` on; rows from `end` on
// become zeros.  DIRECT: by loads that write LDS, where every 8 values of a row
// lie at a multiple of 16 bytes.
template <class T, int DP, int N, bool DIRECT>
struct TileLoader {
    using L = Layout<DP>;
    static constexpr int kLoads = N * L::kChunks / kAttnThreads;
    static_assert(kLoads * kAttnThreads == N * L::kChunks, "whole rounds of loads");

    static __device__ __attribute__((always_inline)) void issue(const T *first, int64_t stride, int row, int end, int dim, char *tile)
    {
        const int tid = threadIdx.x;
        const T *base = first + row * stride;
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
            const int at = s * kAttnThreads + tid;
            const int r = at / L::kChunks;
            const int c = (at & (L::kChunks - 1)) ^ L::twist(r);
            const bool valid = r < end - row && c * 8 < dim;
            if (DIRECT) {
                __amdgpu_buffer_rsrc_t rsrc =
                    __builtin_amdgcn_make_buffer_rsrc((void *)base, short(0), 0x7fffffff, kBufferWord3);
                const uint32_t offset = valid ? uint32_t(r) * uint32_t(stride) * 2 + c * 16 : kOut;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (lds_void *)(tile + s * (kAttnThreads * 16) + uniform(tid >> 6) * 1024), 16, int(offset), 0,
                    0, 0);
            } else {
                vec<T, 8> v = {};
                if (valid) {
                    const T *p = base + int64_t(r) * stride + c * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c * 8 + e < dim) v[e] = p[e];
                }
                *(vec<T, 8> *)(tile + at * 16) = v;
            }
        }
    }
};

// Where a lane reads its fragments of a tile: offsets of which a fragment's own
// place is a constant, exclusive-or'ed and added.  fresh() keeps the compiler from
// holding all of these in registers through a loop.
template <class T, int DP>
struct Reader {
    using L = Layout<DP>;
    uint32_t rows, columns;

    __device__ explicit Reader(int lane)
    {
        const int half = lane >> 5, r = lane & 31;
        rows = r * L::kPitch + ((half ^ L::twist(r)) << 4);
        const int q = (lane & 15) >> 2, c = ((lane >> 3) & 2) + ((lane & 3) >> 1);
        columns = (4 * half + q) * L::kPitch + ((c ^ L::twist(4 * half + q)) << 4) + ((lane & 1) << 3);
    }
    __device__ Reader fresh() const
    {
        Reader r = *this;
        asm("" : "+v"(r.rows), "+v"(r.columns));
        return r;
    }
    // Inner rows as rows of the first operand (32 of them from `block * 32` on):
    // lane l holds row l % 32 and the 8 columns from 16 step + 8 (l / 32) on.
    __device__ __attribute__((always_inline)) vec<T, 8> by_rows(const char *tile, int block, int step) const
    {
        return *(const vec<T, 8> *)(tile + block * 32 * L::kPitch + (rows ^ (step << 5)));
    }
    // Inner rows as k, columns 32 block .. 32 block + 31 as rows of the first
    // operand.  k runs over inner rows 16 step .. 16 step + 15 in the order in which
    // a score tile's registers hold them: lane l has rows 4 (l / 32) + 0..3, then 8
    // more on.
    __device__ __attribute__((always_inline)) vec<T, 8> by_columns(const char *tile, int block, int step) const
    {
        const char *p = tile + step * 16 * L::kPitch;
        const vec<T, 4> x = Half<T>::read_transposed(p + (columns ^ (block << 6)));
        const vec<T, 4> y = Half<T>::read_transposed(p + 8 * L::kPitch + (columns ^ (block << 6) ^ 32));
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// The own rows as second operand: lane l holds row l % 32 and the 8 columns from
// 16 step + 8 (l / 32) on.  Zeros where the row is not valid.
template <class T, int DP, bool DIRECT>
__device__ __attribute__((always_inline)) inline void own_fragments(const T *row, bool valid, int dim, int lane, vec<T, 8> (&f)[DP / 16])
{
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int c = s * 16 + (lane >> 5) * 8;
        f[s] = vec<T, 8>(T(0.0f));
        if (!valid) continue;
        if (DIRECT) {
            if (c < dim) f[s] = *(const vec<T, 8> *)(row + c);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < dim) f[s][e] = row[c + e];
        }
    }
}

// The inner row that register r of a score tile holds, less 4 (lane / 32).
__device__ constexpr int inner_row(int r) { return (r >> 2) * 8 + (r & 3); }

// Adds, or takes the larger, over the two lanes that share an own row.
__device__ __attribute__((always_inline)) inline float other_half(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
    return (threadIdx.x & 32) ? a : b;
}

// A score tile's registers as the second operand's k of 16 rows from 16 step on.
template <class T>
__device__ __attribute__((always_inline)) inline vec<T, 8> as_operand(const f32x16 &s, int step)
{
    vec<T, 8> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = T(s[step * 8 + e]);
    return o;
}

// Writes a wave's 32 own rows (acc: columns x own rows, times `factor`) through
// its LDS, so that a row's stores are whole.
template <class T, int DP, bool DIRECT>
__device__ __attribute__((always_inline)) inline void store_own(const f32x16 (&acc)[DP / 32], float factor, char *lds, T *first, int64_t stride,
                                 int row0, int dim, uint32_t valid, int lane)
{
    using L = Layout<DP>;
    const int own = lane & 31;
#pragma unroll
    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            vec<T, 4> v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = acc[b][g * 4 + e] * factor;
                asm("" : "+v"(x));  // rounded to float first, then to T
                v[e] = T(x);
            }
            const int c = b * 4 + g;
            *(vec<T, 4> *)(lds + own * L::kPitch + ((c ^ L::twist(own)) << 4) + ((lane >> 5) << 3)) = v;
        }
    asm volatile("" ::: "memory");  // a wave's LDS accesses are served in their order
    constexpr int kRowsAtOnce = 64 / L::kChunks;
#pragma unroll
    for (int s = 0; s < 32 / kRowsAtOnce; ++s) {
        const int r = s * kRowsAtOnce + lane / L::kChunks;
        const int c = lane & (L::kChunks - 1);
        if (!((valid >> r) & 1) || c * 8 >= dim) continue;
        const vec<T, 8> v = *(const vec<T, 8> *)(lds + r * L::kPitch + ((c ^ L::twist(r)) << 4));
        T *to = first + int64_t(row0 + r) * stride + c * 8;
        if (DIRECT) {
            *(vec<T, 8> *)to = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c * 8 + e < dim) to[e] = v[e];
        }
    }
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------

// Constants of a head: scores in units of log 2.
struct Scoring {
    float scale;      // of a raw product, in units of log 2, without a cap
    float into_tanh;  // scale / softcap
    float cap;        // softcap in units of log 2, or 0
    float slope;      // in units of log 2, or 0

    __device__ __attribute__((always_inline)) Scoring(const AttnArgs &a, int head)
    {
        scale = a.scale * kLog2e;
        cap = a.softcap * kLog2e;
        into_tanh = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
        slope = a.slopes != nullptr ? a.slopes[head] * kLog2e : 0.0f;
    }
};

// Raw products -> scores in units of log 2, with cap and bias.  distance: own row
// minus the tile's first inner row, less 4 (lane / 32).  GRADIENT: also 1 - tanh^2.
template <bool GRADIENT>
__device__ __attribute__((always_inline)) inline void scores(const Scoring &k, float distance, f32x16 &s, f32x16 &factor)
{
    if (k.cap > 0.0f) {
        float most = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] *= k.into_tanh;
            most = fmaxf(most, fabsf(s[r]));
        }
        // Up to 1/2 the series of tanh x / x, to x^12 (the next term is below 2^-23):
        // 1 - 2 / (1 + e^(2 x)), exact at the ends e = 0 and inf, would lose the bits
        // of small scores.  NaN takes either.
        f32x16 t;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float y = s[r] * s[r];
            float c = fmaf(y, 3.5921280e-3f, -8.8632355e-3f);
            c = fmaf(y, c, 2.1869489e-2f);
            c = fmaf(y, c, -5.3968254e-2f);
            c = fmaf(y, c, 1.3333333e-1f);
            c = fmaf(y, c, -3.3333333e-1f);
            t[r] = fmaf(s[r] * y, c, s[r]);
        }
        if (__ballot(!(most <= 0.5f)) != 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(s[r] * (2.0f * kLog2e));
                const float large = fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + e), 1.0f);
                t[r] = fabsf(s[r]) <= 0.5f ? t[r] : large;
            }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = k.cap * t[r];
            if (GRADIENT) factor[r] = fmaf(-t[r], t[r], 1.0f);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] *= k.scale;
            if (GRADIENT) factor[r] = 1.0f;
        }
    }
    if (k.slope != 0.0f) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = fmaf(-k.slope, fabsf(distance - inner_row(r)), s[r]);
    }
}

// Hidden pairs of a tile that begins at `first` (with 4 (lane / 32) added) become
// `value`: at the upper ends of the own rows' intervals, at the lower ones, or both.
__device__ __attribute__((always_inline)) inline void hide(f32x16 &s, Span span, int first, bool above, bool below, float value)
{
    if (above) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = inner_row(r) < span.hi - first ? s[r] : value;
    }
    if (below) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = inner_row(r) >= span.lo - first ? s[r] : value;
    }
}

// Workgroup -> head and tile.  Workgroups go round the 8 XCDs in turn, so where
// the heads divide by 8 each XCD keeps an eighth of them, whose inner rows then
// share its L2.  `down`: the last tiles, which see most, come first.
__device__ inline void head_and_tile(int id, int heads, int tiles, bool down, int &head, int &tile)
{
    if (heads % 8 == 0) {
        const int each = heads >> 3, at = id >> 3;
        head = (id & 7) * each + at % each;
        tile = at / each;
    } else {
        head = id % heads;
        tile = id / heads;
    }
    if (down) tile = tiles - 1 - tile;
}

// Instruction groups for the scheduler: COUNT times one matrix instruction with
// LDS reads, vector and transcendental instructions behind it, which then run
// under it.  (Left alone, the compiler puts the products of a phase in a row.)
template <int COUNT, int READS, int VECTOR, int TRANSCENDENTAL>
__device__ inline void under_products()
{
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        if (VECTOR > 0) __builtin_amdgcn_sched_group_barrier(0x2, VECTOR, 0);
        if (TRANSCENDENTAL > 0) __builtin_amdgcn_sched_group_barrier(0x400, TRANSCENDENTAL, 0);
    }
}

template <class T>
constexpr float kWeightShift = std::is_same<T, f16>::value ? 7.0f : 0.0f;

// ---------------------------------------------------------------------------
// Infinities and NaN
// ---------------------------------------------------------------------------

// Workgroups of the second kernels, which look for flags among all tiles.
constexpr int kCarefulGroups = 256;

// A hidden pair's weight is 0, but 0 times an infinity or a NaN is NaN.  So a
// workgroup whose sums end as such leaves a flag, and a second kernel makes its
// tile again, carefully: inner rows that hold one are taken out of the LDS tile
// before the second products, and what they add to the own rows that see them is
// added by itself.  (In one kernel the two would share the registers: the careful
// walk behind the other one put 80 bytes a lane of dq's into scratch memory.)

// f(id) for the flags that are set: a workgroup looks after every gridDim.x-th,
// 256 of them at once.
template <class F>
__device__ inline void for_flags(const int32_t *flags, int n, F f)
{
    for (int64_t base = blockIdx.x; base < n; base += int64_t(gridDim.x) * kAttnThreads) {
        const int64_t at = base + int64_t(threadIdx.x) * gridDim.x;
        if (!__syncthreads_or(at < n && flags[at])) continue;
        for (int t = 0; t < kAttnThreads; ++t) {
            const int64_t id = base + int64_t(t) * gridDim.x;
            if (id >= n) break;
            if (!uniform(flags[id])) continue;
            f(int(id));
            __syncthreads();
        }
    }
}

template <int B>
__device__ __attribute__((always_inline)) inline bool all_finite(const f32x16 (&acc)[B])
{
    float zero = 0.0f;
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) zero = fmaf(acc[b][r], 0.0f, zero);
    return zero == 0.0f;
}

// Clears the rows of a tile that hold an infinity or a NaN and says which they
// are.  Every wave has to call it; none reads the tile meanwhile.
template <class T, int DP, int N>
__device__ __attribute__((always_inline)) inline uint64_t take_out(char *tile, uint32_t (&words)[2])
{
    using L = Layout<DP>;
    constexpr int kLoads = N * L::kChunks / kAttnThreads;
    constexpr uint16_t kExponent = std::is_same<T, f16>::value ? 0x7c00 : 0x7f80;
    __syncthreads();
    if (threadIdx.x < 2) words[threadIdx.x] = 0;
    __syncthreads();
    for (int s = 0; s < kLoads; ++s) {
        const int at = s * kAttnThreads + threadIdx.x, row = at / L::kChunks;
        const vec<uint16_t, 8> v = *(const vec<uint16_t, 8> *)(tile + at * 16);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) bad |= (v[e] & kExponent) == kExponent;
        if (bad) atomicOr(&words[row >> 5], 1u << (row & 31));
    }
    __syncthreads();
    const uint64_t rows = uint64_t(words[1]) << 32 | words[0];
    for (int s = 0; s < kLoads; ++s) {
        const int at = s * kAttnThreads + threadIdx.x;
        if ((rows >> (at / L::kChunks)) & 1) *(u32x4 *)(tile + at * 16) = u32x4(0);
    }
    __syncthreads();
    return uint64_t(uint32_t(uniform(int(rows >> 32)))) << 32 | uint32_t(uniform(int(rows)));
}

// Adds the products of the rows taken out with the weights of the own rows that
// see them.  w: the weights of inner rows, N / 32 tiles of them; values: the
// tile's first inner row.
template <class T, int DP, int B>
__device__ __attribute__((always_inline)) inline void add_taken_out(uint64_t rows, const f32x16 (&w)[B], const T *values, int64_t stride, int dim,
                                     int row, Span span, int lane, f32x16 (&acc)[DP / 32])
{
    while (rows != 0) {
        const int i = __builtin_ctzll(rows);
        rows &= rows - 1;
        float x = 0.0f;
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) x = (i & ~4) == b * 32 + inner_row(r) ? w[b][r] : x;
        const float y = other_half(x);
        const float weight = float(T(((i >> 2) & 1) == (lane >> 5) ? x : y));
        if (row + i < span.lo || row + i >= span.hi) continue;
        const T *v = values + int64_t(i) * stride + ((lane >> 5) << 2);
#pragma unroll
        for (int b = 0; b < DP / 32; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int d = b * 32 + inner_row(r);
                if (d + ((lane >> 5) << 2) < dim) acc[b][r] = fmaf(weight, float(v[d]), acc[b][r]);
            }
    }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

constexpr int kInner = 32;  // inner rows of a tile in the backward pass
// In the forward pass, whose maximum and rescaling each tile pays once.
template <int DP>
constexpr int kForwardInner = DP <= 128 ? 64 : 32;

template <class T, int DP, bool DIRECT, bool EXTRA, bool CAREFUL>
__device__ __attribute__((always_inline)) inline void forward_tile(const AttnArgs &a, int id)
{
    using L = Layout<DP>;
    constexpr int N = kForwardInner<DP>, B = N / 32;
    constexpr int kTileLds = N * L::kPitch;
    constexpr int kStage = 2 * kTileLds;
    using Loader = TileLoader<T, DP, N, DIRECT>;
    // Two stages of k and v, arrays of their own, or the compiler would wait for the
    // loads into one before it reads the other.
    __shared__ __attribute__((aligned(1024))) char lds0[kStage], lds1[kStage];
    __shared__ int box[4 * kAttnWaves];
    __shared__ uint32_t words[2];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int head, tile;
    head_and_tile(id, a.heads, a.tiles, true, head, tile);
    const int row0 = tile * kOwnTile + wave * kOwn;
    const int own = row0 + (lane & 31);
    const Span span = keys_of(a, own);
    const WaveSpan mine(span);
    const GroupSpan all(mine, wave, box, 2 * N);
    if (all.hi <= all.lo) {
        if (!CAREFUL && threadIdx.x == 0) a.flags[id] = 0;
        return;
    }
    const int kv = head / (a.heads / a.kv_heads);
    const T *k = a.k.at<T>(kv, 0), *v = a.v.at<T>(kv, 0);
    auto issue = [&](int row, char *stage) __attribute__((always_inline)) {
        Loader::issue(k, a.k.stride, row, all.hi, a.dim, stage);  // (behind the last tile: zeros, from nowhere)
        Loader::issue(v, a.v.stride, row, all.hi, a.dim, stage + kTileLds);
    };
    issue(all.lo, lds0);
    vec<T, 8> q[DP / 16];
    own_fragments<T, DP, DIRECT>(a.q.at<T>(head, own), span.hi > 0, a.dim, lane, q);
    const Scoring scoring(a, head);
    const float unit = EXTRA ? 1.0f : scoring.scale;

    const Reader<T, DP> reader(lane);
    f32x16 acc[DP / 32];
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) acc[b] = f32x16(0.0f);
    float top = -INFINITY;  // what the weights are taken from, at most 8 below the row's maximum
    float total = 0.0f;     // over this lane's inner rows

    auto tile_step = [&](auto masked, char *kt, int row, bool skip) __attribute__((always_inline)) {
        char *vt = kt + kTileLds;
        const Reader<T, DP> at = DP >= 128 ? reader.fresh() : reader;
        uint64_t out = 0;
        if (CAREFUL) {
            out = take_out<T, DP, N>(vt, words);
            if (skip) return;
        }
        f32x16 s[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            s[b] = f32x16(0.0f);
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) s[b] = mfma32(at.by_rows(kt, b, d), q[d], s[b]);
        }
        const int first = row + ((lane >> 5) << 2);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            f32x16 unused;
            if (EXTRA) scores<false>(scoring, float(own - first - b * 32), s[b], unused);
            if (decltype(masked)::value)
                hide(s[b], span, first + b * 32, row + N > mine.every_hi, row < mine.every_lo, -INFINITY);
        }
        float most = s[0][0];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) most = fmaxf(most, s[b][r]);
        most = fmaxf(most, other_half(most)) * unit;
        // Weights may exceed 1 up to 2^8 (all in float but for their rounding,
        // which is relative), so the sums are rescaled only where the maximum
        // rises by more.
        if (__ballot(most > top + 8.0f) != 0) {
            const float higher = fmaxf(most, top);
            const float keep = higher == top ? 1.0f : __builtin_amdgcn_exp2f(top - higher);
            top = higher;
            total *= keep;
#pragma unroll
            for (int b = 0; b < DP / 32; ++b) acc[b] *= keep;
        }
        const float from = (top == -INFINITY ? 0.0f : top) - kWeightShift<T>;
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], unit, -from));
                total += s[b][r];
            }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const vec<T, 8> p = as_operand<T>(s[b], i);
#pragma unroll
                for (int d = 0; d < DP / 32; ++d) acc[d] = mfma32(at.by_columns(vt, d, b * 2 + i), p, acc[d]);
            }
        if (CAREFUL && out != 0)
            add_taken_out<T, DP>(out, s, v + row * a.v.stride, a.v.stride, a.dim, row, span, lane, acc);
    };
    auto run = [&](auto masked, char *kt, char *next, int row) __attribute__((always_inline)) {
        issue(row + N, next);
        const bool skip = !mine.any || row >= mine.hi || row + N <= mine.lo;
        if (CAREFUL || !skip) tile_step(masked, kt, row, skip);
    };
    int row = all.lo;
    auto walk = [&](auto masked, int end) __attribute__((always_inline)) {
        for (; row < end; row += 2 * N) {
            wait_loads<0>();
            barrier();
            run(masked, lds0, lds1, row);
            wait_loads<0>();
            barrier();
            run(masked, lds1, lds0, row + N);
        }
    };
    walk(std::true_type(), all.open);
    if (!CAREFUL) walk(std::false_type(), all.close);
    walk(std::true_type(), all.hi);
    wait_loads<0>();
    const int bad = __syncthreads_or(span.hi > 0 && !all_finite(acc));  // (and every wave has read the last tile)
    if (!CAREFUL && threadIdx.x == 0) a.flags[id] = bad;
    total += other_half(total);
    const uint32_t valid = uint32_t(__ballot(span.hi > 0));
    store_own<T, DP, DIRECT>(acc, 1.0f / total, (wave < 2 ? lds0 : lds1) + (wave & 1) * (kOwn * L::kPitch), a.o.at<T>(head, 0), a.o.stride, row0, a.dim, valid, lane);
    if (a.lse != nullptr && span.hi > 0 && lane < 32)
        a.lse[int64_t(head) * a.rows + own] = (top - kWeightShift<T> + __builtin_amdgcn_logf(total)) * kLn2;
}

template <class T, int DP, bool DIRECT, bool EXTRA>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_forward_kernel(AttnArgs a)
{
    forward_tile<T, DP, DIRECT, EXTRA, false>(a, blockIdx.x);
}

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_forward_careful_kernel(AttnArgs a)
{
    for_flags(a.flags, a.tiles * a.heads, [&](int id) { forward_tile<T, DP, false, true, true>(a, id); });
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// fp16 only: ds in units of a power of two that follows the largest of an own
// row, so that neither small gradients lose bits nor large ones overflow: the
// largest lies in [2^13, 2^15], whatever its size.
template <class T>
struct Units {
    static constexpr bool kUsed = std::is_same<T, f16>::value;
    float unit = kUsed ? 0x1p126f : 1.0f;

    // Chooses the units of a tile's ds, and rescales the sums so far.
    template <int B>
    __device__ __attribute__((always_inline)) void apply(f32x16 &ds, f32x16 (&acc)[B])
    {
        if (!kUsed) return;
        float most = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) most = fmaxf(most, fabsf(ds[r]));
        most = fmaxf(most, other_half(most));
        const bool grow = most * unit > 0x1p15f;
        if (__ballot(grow) != 0) {
            int e = 127 + 127 + 13 - int(__float_as_uint(most) >> 23);  // 2^13 at the largest's exponent
            e = e > 253 ? 253 : e < 1 ? 1 : e;
            const float next = grow ? __uint_as_float(uint32_t(e) << 23) : unit;
            const float keep = next / unit;
            unit = next;
#pragma unroll
            for (int b = 0; b < B; ++b) acc[b] *= keep;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) ds[r] *= unit;
    }
};

// A tile of queries that sees at most this many keys takes delta from p and dp, and
// one whose bias leaves keys 32 away less than e^-8.
constexpr int kExactDelta = 256;

template <class T, int DP, bool DIRECT, bool EXTRA, bool CAREFUL>
__device__ __attribute__((always_inline)) inline void dq_tile(const AttnArgs &a, int id)
{
    using L = Layout<DP>;
    constexpr int N = kInner;
    constexpr int kTileLds = N * L::kPitch;
    constexpr int kStage = 2 * kTileLds;
    using Loader = TileLoader<T, DP, N, DIRECT>;
    __shared__ __attribute__((aligned(1024))) char lds0[kStage], lds1[kStage];
    __shared__ int box[4 * kAttnWaves];
    __shared__ uint32_t words[2];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int head, tile;
    head_and_tile(id, a.heads, a.tiles, true, head, tile);
    const int row0 = tile * kOwnTile + wave * kOwn;
    const int own = row0 + (lane & 31);
    const Span span = keys_of(a, own);
    const WaveSpan mine(span);
    const GroupSpan all(mine, wave, box, 2 * N);
    if (all.hi <= all.lo) {
        if (!CAREFUL && threadIdx.x == 0) a.flags[id] = 0;
        return;
    }
    const int kv = head / (a.heads / a.kv_heads);
    const T *k = a.k.at<T>(kv, 0), *v = a.v.at<T>(kv, 0);
    const bool valid = span.hi > 0;
    vec<T, 8> q[DP / 16], g[DP / 16];
    own_fragments<T, DP, DIRECT>(a.o.at<T>(head, own), valid, a.dim, lane, q);
    own_fragments<T, DP, DIRECT>(a.dout.at<T>(head, own), valid, a.dim, lane, g);
    float delta = 0.0f;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(float(q[d][e]), float(g[d][e]), delta);
    delta += other_half(delta);
    const float lse = valid ? a.lse[int64_t(head) * a.rows + own] * kLog2e : 0.0f;
    own_fragments<T, DP, DIRECT>(a.q.at<T>(head, own), valid, a.dim, lane, q);
    const Scoring scoring(a, head);
    const float unit = EXTRA ? 1.0f : scoring.scale;

    f32x16 acc[DP / 32];
    Units<T> units;
    const Reader<T, DP> reader(lane);
    // The sum of p dp is delta without o's rounding, which counts where a row sees
    // few keys: there a first walk takes the sum.  The other rows keep the one
    // from o for dq, and dk takes the sum everywhere.
    float sum = 0.0f;
    auto issue = [&](int row, char *stage) __attribute__((always_inline)) {
        Loader::issue(k, a.k.stride, row, all.hi, a.dim, stage);
        Loader::issue(v, a.v.stride, row, all.hi, a.dim, stage + kTileLds);
    };
    auto tile_step = [&](auto masked, auto sums_only, char *kt, int row, bool skip) __attribute__((always_inline)) {
        const Reader<T, DP> at = DP >= 128 ? reader.fresh() : reader;
        f32x16 x = f32x16(0.0f), dp = f32x16(0.0f), factor;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) x = mfma32(at.by_rows(kt, 0, d), q[d], x);
        const int first = row + ((lane >> 5) << 2);
        const bool above = row + N > mine.every_hi, below = row < mine.every_lo;
        if (EXTRA) scores<true>(scoring, float(own - first), x, factor);
        if (decltype(masked)::value) hide(x, span, first, above, below, -INFINITY);
        __builtin_amdgcn_sched_barrier(0);
        // dp, the products of v and dout, and under them the weights
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) dp = mfma32(at.by_rows(kt + kTileLds, 0, d), g[d], dp);
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], unit, -lse));
        under_products<DP / 16, 1, 2 * 128 / DP, 2 * 128 / DP>();
        __builtin_amdgcn_sched_barrier(0);
        uint64_t out = 0;
        if (CAREFUL) {
            out = take_out<T, DP, N>(kt, words);
            if (skip) return;
        }
        if (decltype(masked)::value) {
            hide(dp, span, first, above, below, 0.0f);
            if (EXTRA) hide(factor, span, first, above, below, 0.0f);
        }
        f32x16 ds[1];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            sum = fmaf(x[r], dp[r], sum);
            ds[0][r] = x[r] * (dp[r] - delta);
            if (EXTRA) ds[0][r] *= factor[r];
        }
        if (decltype(sums_only)::value) return;
        units.apply(ds[0], acc);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const vec<T, 8> y = as_operand<T>(ds[0], i);
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) acc[d] = mfma32(at.by_columns(kt, d, i), y, acc[d]);
        }
        if (CAREFUL && out != 0)
            add_taken_out<T, DP>(out, ds, k + row * a.k.stride, a.k.stride, a.dim, row, span, lane, acc);
    };
    auto run = [&](auto masked, auto sums_only, char *kt, char *next, int row) __attribute__((always_inline)) {
        issue(row + N, next);
        const bool skip = !mine.any || row >= mine.hi || row + N <= mine.lo;
        if (CAREFUL || !skip) tile_step(masked, sums_only, kt, row, skip);
    };
    int row;
    auto walk = [&](auto masked, auto sums_only, int end) __attribute__((always_inline)) {
        for (; row < end; row += 2 * N) {
            wait_loads<0>();
            barrier();
            run(masked, sums_only, lds0, lds1, row);
            wait_loads<0>();
            barrier();
            run(masked, sums_only, lds1, lds0, row + N);
        }
    };
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) acc[b] = f32x16(0.0f);
    issue(all.lo, lds0);
    row = all.lo;
    if (all.hi - all.lo <= kExactDelta || scoring.slope * 32.0f >= 8.0f * kLog2e) {
        walk(std::true_type(), std::true_type(), all.hi);
        delta = sum + other_half(sum);
        sum = 0.0f;
        wait_loads<0>();
        barrier();  // every wave has read the last tile
        issue(all.lo, lds0);
        row = all.lo;
    }
    walk(std::true_type(), std::false_type(), all.open);
    if (!CAREFUL) walk(std::false_type(), std::false_type(), all.close);
    walk(std::true_type(), std::false_type(), all.hi);
    wait_loads<0>();
    const int bad = __syncthreads_or(valid && !all_finite(acc));  // (and every wave has read the last tile)
    if (!CAREFUL && threadIdx.x == 0) a.flags[id] = bad;
    sum += other_half(sum);
    if (!CAREFUL && valid && lane < 32) {
        float *to = a.numbers + int64_t(head) * a.rows + own;
        to[0] = lse;
        to[int64_t(a.heads) * a.rows] = sum;
    }
    const uint32_t rows_in = uint32_t(__ballot(valid));
    store_own<T, DP, DIRECT>(acc, a.scale / units.unit, (wave < 2 ? lds0 : lds1) + (wave & 1) * (kOwn * L::kPitch),
                             a.dq.at<T>(head, 0), a.dq.stride, row0, a.dim, rows_in, lane);
}

template <class T, int DP, bool DIRECT, bool EXTRA>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_dq_kernel(AttnArgs a)
{
    dq_tile<T, DP, DIRECT, EXTRA, false>(a, blockIdx.x);
}

// A long walk for dk and dv is split into parts of at least 32 pairs of inner tiles,
// each a workgroup's, whose float sums a further kernel adds in their order: with
// few workgroups the tiles that many queries see would keep the others waiting
// (8192 rows of 19 documents, 32 heads on 8 of 128: 386 us whole, 320 in parts with
// their sums; with 16 pairs 2048 rows of one document took no less than whole).
// Up to 128 columns: wider ones, of which one workgroup fits a compute unit, took
// longer (4096 rows, 8 heads on 4 of 256: 215 us whole, 400 in parts).
constexpr int kLeastPairs = 32, kMostWalkParts = 8;

__device__ inline int parts_of(const AttnArgs &a, int pairs)
{
    const int n = pairs / kLeastPairs;
    return n <= 1 ? 1 : n < a.parts ? n : a.parts;
}

// A part's sums, as its waves hold them: 64 lanes of 4 values after each other.
template <int DP>
__device__ inline f32x4 *part_of(const AttnArgs &a, int index, int wave, int lane)
{
    return (f32x4 *)a.sums + (int64_t(index) * kAttnWaves + wave) * (DP / 32 * 8) * 64 + lane;
}
template <int DP, class F>
__device__ __attribute__((always_inline)) inline void each_quad(f32x16 (&dv)[DP / 32], f32x16 (&dk)[DP / 32], F f)
{
#pragma unroll
    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f(b * 4 + g, dv[b], g, false);
            f(DP / 8 + b * 4 + g, dk[b], g, true);
        }
}

template <class T, int DP, bool DIRECT, bool EXTRA, bool CAREFUL>
__device__ __attribute__((always_inline)) inline void dkdv_tile(const AttnArgs &a, int id)
{
    using L = Layout<DP>;
    constexpr int N = kInner;
    constexpr int kTileLds = N * L::kPitch;
    constexpr int kNumbers = 2 * N * 4;  // lse and delta of a stage's queries
    constexpr int kStage = 2 * kTileLds + kNumbers;
    using Loader = TileLoader<T, DP, N, DIRECT>;
    // From 128 columns on the sums of dk and dv leave no registers for v too: it
    // stays in LDS, so that two workgroups fit a compute unit (128 columns).
    constexpr bool kValuesInLds = DP >= 128 && !CAREFUL;
    __shared__ __attribute__((aligned(1024))) char values[kValuesInLds ? kOwnTile * L::kPitch : 16];
    __shared__ __attribute__((aligned(1024))) char lds0[kStage], lds1[kStage];
    __shared__ int box[4 * kAttnWaves];
    __shared__ uint32_t words[2];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int base = a.tiles * a.kv_heads, part = CAREFUL ? 0 : id / base;
    const int tile_id = CAREFUL ? id : id - part * base;
    int kv, tile;
    head_and_tile(tile_id, a.kv_heads, a.tiles, false, kv, tile);
    const int row0 = tile * kOwnTile + wave * kOwn;
    const int own = row0 + (lane & 31);
    const Span span = queries_of(a, own);
    const WaveSpan mine(span);
    const GroupSpan all(mine, wave, box, 2 * N);
    if (all.hi <= all.lo) {
        if (!CAREFUL && threadIdx.x == 0) a.flags[id] = 0;
        return;
    }
    const int group = a.heads / a.kv_heads;
    const int pairs = (all.hi - all.lo + 2 * N - 1) / (2 * N), total = group * pairs;  // pairs of inner tiles
    const int parts = CAREFUL || DP > 128 ? 1 : parts_of(a, total);
    if (part >= parts) {
        if (threadIdx.x == 0) a.flags[id] = 0;
        return;
    }
    const bool valid = span.hi > 0;
    vec<T, 8> k[DP / 16], v[DP / 16];
    own_fragments<T, DP, DIRECT>(a.k.at<T>(kv, own), valid, a.dim, lane, k);
    if (kValuesInLds)
        TileLoader<T, DP, kOwnTile, DIRECT>::issue(a.v.at<T>(kv, 0), a.v.stride, tile * kOwnTile, a.rows, a.dim, values);
    else
        own_fragments<T, DP, DIRECT>(a.v.at<T>(kv, own), valid, a.dim, lane, v);

    f32x16 dk[DP / 32], dv[DP / 32];
    Units<T> units;
    const Reader<T, DP> reader(lane);
    const char *mine_values = values + wave * (kOwn * L::kPitch);
    auto issue = [&](int head, int row, char *stage) __attribute__((always_inline)) {
        Loader::issue(a.q.at<T>(head, 0), a.q.stride, row, all.hi, a.dim, stage);
        Loader::issue(a.dout.at<T>(head, 0), a.dout.stride, row, all.hi, a.dim, stage + kTileLds);
        if (wave < 2 && lane < N) {
            const float *from = a.numbers + (int64_t(wave) * a.heads + head) * a.rows + row;
            __amdgpu_buffer_rsrc_t rsrc =
                __builtin_amdgcn_make_buffer_rsrc((void *)from, short(0), 0x7fffffff, kBufferWord3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(stage + 2 * kTileLds + wave * (N * 4)), 4,
                                                     int(row + lane < all.hi ? uint32_t(lane) * 4 : kOut), 0, 0, 0);
        }
    };
    auto tile_step = [&](auto masked, char *qt, int head, int row, bool skip) __attribute__((always_inline)) {
        const Scoring scoring(a, head);
        const float unit = EXTRA ? 1.0f : scoring.scale;
        char *gt = qt + kTileLds;
        const float *numbers = (const float *)(gt + kTileLds);
        const Reader<T, DP> at = DP >= 128 ? reader.fresh() : reader;
        f32x16 w[1] = {f32x16(0.0f)}, ds[1] = {f32x16(0.0f)};
        f32x16 factor;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) w[0] = mfma32(at.by_rows(qt, 0, d), k[d], w[0]);
        const int first = row + ((lane >> 5) << 2);
        const bool above = row + N > mine.every_hi, below = row < mine.every_lo;
        if (EXTRA) scores<true>(scoring, float(own - first), w[0], factor);
        __builtin_amdgcn_sched_barrier(0);
        // dp, the products of dout and v, and under them the weights
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            ds[0] = mfma32(at.by_rows(gt, 0, d), kValuesInLds ? at.by_rows(mine_values, 0, d) : v[d], ds[0]);
#pragma unroll
        for (int r = 0; r < 16; ++r)
            w[0][r] = __builtin_amdgcn_exp2f(fmaf(w[0][r], unit, -numbers[inner_row(r) + ((lane >> 5) << 2)]));
        under_products<DP / 16, kValuesInLds ? 3 : 2, 2 * 128 / DP, 2 * 128 / DP>();
        __builtin_amdgcn_sched_barrier(0);
        uint64_t out_q = 0, out_g = 0;
        if (CAREFUL) {
            out_q = take_out<T, DP, N>(qt, words);
            out_g = take_out<T, DP, N>(gt, words);
            if (skip) return;
        }
        if (decltype(masked)::value) hide(w[0], span, first, above, below, 0.0f);
        // dv, and under it ds
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const vec<T, 8> p = as_operand<T>(w[0], i);
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) dv[d] = mfma32(at.by_columns(gt, d, i), p, dv[d]);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            ds[0][r] = w[0][r] * (ds[0][r] - numbers[N + inner_row(r) + ((lane >> 5) << 2)]);
            if (EXTRA) ds[0][r] *= factor[r];
        }
        under_products<DP / 16, 2, 5 * 128 / DP, 0>();
        __builtin_amdgcn_sched_barrier(0);
        if (decltype(masked)::value) hide(ds[0], span, first, above, below, 0.0f);
        units.apply(ds[0], dk);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const vec<T, 8> y = as_operand<T>(ds[0], i);
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) dk[d] = mfma32(at.by_columns(qt, d, i), y, dk[d]);
        }
        if (CAREFUL && out_g != 0)
            add_taken_out<T, DP>(out_g, w, a.dout.at<T>(head, row), a.dout.stride, a.dim, row, span, lane, dv);
        if (CAREFUL && out_q != 0)
            add_taken_out<T, DP>(out_q, ds, a.q.at<T>(head, row), a.q.stride, a.dim, row, span, lane, dk);
    };
    auto run = [&](auto masked, char *qt, char *next, int head, int row) __attribute__((always_inline)) {
        issue(head, row + N, next);  // (behind the last tile: zeros, from nowhere)
        const bool skip = !mine.any || row >= mine.hi || row + N <= mine.lo;
        if (CAREFUL || !skip) tile_step(masked, qt, head, row, skip);
    };
    auto walk = [&](auto masked, int head, int &row, int end) __attribute__((always_inline)) {
        for (; row < end; row += 2 * N) {
            wait_loads<0>();
            barrier();
            run(masked, lds0, lds1, head, row);
            wait_loads<0>();
            barrier();
            run(masked, lds1, lds0, head, row + N);
        }
    };
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) dk[b] = dv[b] = f32x16(0.0f);
    const int until = int(int64_t(total) * (part + 1) / parts);
    for (int at = int(int64_t(total) * part / parts); at < until;) {
        const int head = kv * group + at / pairs, from = at % pairs;
        const int n = pairs - from < until - at ? pairs - from : until - at;
        at += n;
        int row = all.lo + from * (2 * N);
        const int end = from + n < pairs ? row + n * (2 * N) : all.hi;
        issue(head, row, lds0);
        walk(std::true_type(), head, row, all.open < end ? all.open : end);
        if (!CAREFUL) walk(std::false_type(), head, row, all.close < end ? all.close : end);
        walk(std::true_type(), head, row, end);
        wait_loads<0>();
        barrier();  // every wave has read the last tile
    }
    wait_loads<0>();
    const int bad = __syncthreads_or(valid && !(all_finite(dk) && all_finite(dv)));  // (and every wave has read the last tile)
    if (!CAREFUL && threadIdx.x == 0) a.flags[id] = bad;
    if (parts > 1) {
        f32x4 *to = part_of<DP>(a, part * base + tile_id, wave, lane);
        each_quad<DP>(dv, dk, [&](int i, f32x16 &acc, int g, bool is_dk) __attribute__((always_inline)) {
            const float factor = is_dk ? a.scale / units.unit : 1.0f;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[g * 4 + e] * factor;
            to[i * 64] = v;
        });
        return;
    }
    const uint32_t rows_in = uint32_t(__ballot(valid));
    char *mine_lds = (wave < 2 ? lds0 : lds1) + (wave & 1) * (kOwn * L::kPitch);
    store_own<T, DP, DIRECT>(dv, 1.0f, mine_lds, a.dv.at<T>(kv, 0), a.dv.stride, row0, a.dim, rows_in, lane);
    asm volatile("" ::: "memory");
    store_own<T, DP, DIRECT>(dk, a.scale / units.unit, mine_lds, a.dk.at<T>(kv, 0), a.dk.stride, row0, a.dim, rows_in,
                             lane);
}

template <class T, int DP, bool DIRECT, bool EXTRA>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_dkdv_kernel(AttnArgs a)
{
    a.flags += a.tiles * a.heads;  // behind dq's
    dkdv_tile<T, DP, DIRECT, EXTRA, false>(a, blockIdx.x);
}

// Adds up the parts of the tiles that were split.
template <class T, int DP, bool DIRECT>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_join_kernel(AttnArgs a)
{
    using L = Layout<DP>;
    __shared__ __attribute__((aligned(1024))) char lds[kOwnTile * L::kPitch];
    __shared__ int box[4 * kAttnWaves];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int kv, tile;
    head_and_tile(blockIdx.x, a.kv_heads, a.tiles, false, kv, tile);
    const int row0 = tile * kOwnTile + wave * kOwn;
    const Span span = queries_of(a, row0 + (lane & 31));
    const GroupSpan all(WaveSpan(span), wave, box, 2 * kInner);
    if (all.hi <= all.lo) return;
    const int parts =
        parts_of(a, a.heads / a.kv_heads * ((all.hi - all.lo + 2 * kInner - 1) / (2 * kInner)));
    if (parts == 1) return;
    f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) dk[b] = dv[b] = f32x16(0.0f);
    for (int p = 0; p < parts; ++p) {
        const f32x4 *from = part_of<DP>(a, p * a.tiles * a.kv_heads + blockIdx.x, wave, lane);
        each_quad<DP>(dv, dk, [&](int i, f32x16 &acc, int g, bool) __attribute__((always_inline)) {
            const f32x4 v = from[i * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g * 4 + e] += v[e];
        });
    }
    const uint32_t rows_in = uint32_t(__ballot(span.hi > 0));
    char *mine = lds + wave * (kOwn * L::kPitch);
    store_own<T, DP, DIRECT>(dv, 1.0f, mine, a.dv.at<T>(kv, 0), a.dv.stride, row0, a.dim, rows_in, lane);
    asm volatile("" ::: "memory");
    store_own<T, DP, DIRECT>(dk, 1.0f, mine, a.dk.at<T>(kv, 0), a.dk.stride, row0, a.dim, rows_in, lane);
}

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_backward_careful_kernel(AttnArgs a)
{
    const int first = a.tiles * a.heads, base = a.tiles * a.kv_heads;
    for_flags(a.flags, first + base * a.parts, [&](int id) {
        if (id < first) {
            dq_tile<T, DP, false, true, true>(a, id);
        } else {
            // (once for a tile several of whose parts are flagged)
            for (int other = id - base; other >= first; other -= base)
                if (uniform(a.flags[other])) return;
            dkdv_tile<T, DP, false, true, true>(a, (id - first) % base);
        }
    });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// A tensor of rows x heads x dim elements of `bytes` each, for the overlap checks.
struct HeadView {
    const void *p;
    int64_t rows, heads, dim, stride, head_stride;  // bytes from dim on

    bool none() const { return p == nullptr || rows <= 0; }
    int64_t extent() const { return (rows - 1) * stride + (heads - 1) * head_stride + dim; }
    // No element lies on another: heads side by side in a row, or rows in a head.
    bool distinct() const
    {
        const bool by_row = (heads == 1 || head_stride >= dim) && (rows == 1 || stride >= (heads - 1) * head_stride + dim);
        const bool by_head = (rows == 1 || stride >= dim) && (heads == 1 || head_stride >= (rows - 1) * stride + dim);
        return by_row || by_head;
    }
};

bool overlap(const HeadView &a, const HeadView &b)
{
    if (a.none() || b.none()) return false;
    const int64_t a0 = int64_t(uintptr_t(a.p)), b0 = int64_t(uintptr_t(b.p));
    if (a0 + a.extent() <= b0 || b0 + b.extent() <= a0) return false;
    // views of one parent whose rows, or whose heads, lie between each other's
    auto apart = [&](int64_t period, int64_t a_bytes, int64_t b_bytes) {
        if (period <= 0) return false;
        int64_t d = (b0 - a0) % period;
        if (d < 0) d += period;
        return d >= a_bytes && d + b_bytes <= period;
    };
    const int64_t a_row = (a.heads - 1) * a.head_stride + a.dim, b_row = (b.heads - 1) * b.head_stride + b.dim;
    const int64_t a_head = (a.rows - 1) * a.stride + a.dim, b_head = (b.rows - 1) * b.stride + b.dim;
    const bool rows_alike = a.stride == b.stride, heads_alike = a.head_stride == b.head_stride;
    if (rows_alike && apart(a.stride, a_row, b_row)) return false;
    if (heads_alike && apart(a.head_stride, a_head, b_head)) return false;
    if (rows_alike && heads_alike) {
        // both strides multiples of the smaller one: all elements lie at multiples of it
        const int64_t small = std::min(a.stride, a.head_stride), large = std::max(a.stride, a.head_stride);
        if (small > 0 && large % small == 0 && apart(small, a.dim, b.dim)) return false;
    }
    return true;
}

HeadView view(const void *p, int64_t rows, int64_t heads, int64_t dim, int64_t stride, int64_t head_stride, int bytes)
{
    return HeadView{p, rows, heads, dim * bytes, stride * bytes, head_stride * bytes};
}

HeadView flat_view(const void *p, int64_t bytes) { return HeadView{p, bytes > 0 ? 1 : 0, 1, bytes, bytes, bytes}; }

bool valid_strides(int64_t stride, int64_t head_stride)
{
    return stride >= 0 && stride <= kMaxDirectStride && head_stride >= 0 && head_stride <= int64_t(1) << 40;
}

// Sizes, types and the mask: what both passes and the plan need.
int check_attn(const adam_attn_desc *d)
{
    if (d == nullptr || !known_type(d->type)) return ADAM_EINVAL;
    if (!is_half(d->type)) return ADAM_EDTYPE;
    if (d->rows < 0 || d->rows > kMaxProductRows || d->heads < 1 || d->heads > kMaxHeads || d->kv_heads < 1 ||
        d->heads % d->kv_heads != 0 || d->head_dim < 1 || d->head_dim > kMaxAttnDim)
        return ADAM_EINVAL;
    if ((d->causal != 0 && d->causal != 1) || d->window < 0 || d->docs < 0 || d->docs > kMaxProductRows)
        return ADAM_EINVAL;
    if (d->doc_offsets == nullptr && d->docs != 1) return ADAM_EINVAL;
    if ((d->prefix != nullptr || d->window > 0) && !d->causal) return ADAM_EINVAL;
    if (d->prefix != nullptr && d->window > 0) return ADAM_EINVAL;
    if (!std::isfinite(d->scale) || !(d->scale > 0.0f) || !std::isfinite(d->softcap) || !(d->softcap >= 0.0f))
        return ADAM_EINVAL;
    const int64_t tiles = (d->rows + kOwnTile - 1) / kOwnTile;
    // a dispatch counts its work-items in 32 bits
    if (tiles * d->heads * kAttnThreads >= int64_t(1) << 32) return ADAM_EINVAL;
    return ADAM_OK;
}

struct AttnPlan {
    int32_t *flags;
    float *numbers = nullptr, *sums = nullptr;
    int64_t parts = 1;
    int64_t bytes;
    AttnPlan(const adam_attn_desc &d, bool backward, void *workspace)
    {
        const int64_t tiles = (d.rows + kOwnTile - 1) / kOwnTile;
        Workspace w{(char *)workspace};
        if (backward) {
            // With 1024 workgroups (two rounds) and more the tiles even out by
            // themselves; fewer are split towards 2048.
            const int64_t base = tiles * d.kv_heads, longest = d.heads / d.kv_heads * (d.rows / (2 * kInner));
            if (base < 1024 && d.head_dim <= 128) parts = std::min<int64_t>(kMostWalkParts, 2048 / base);
            parts = std::max<int64_t>(1, std::min(parts, longest / kLeastPairs));
            numbers = w.take<float>(2 * d.heads * d.rows);
            if (parts > 1) {
                const int dp = d.head_dim <= 64 ? 64 : 128;
                sums = w.take<float>(base * parts * kOwnTile * dp * 2);
            }
        }
        flags = w.take<int32_t>(tiles * (d.heads + (backward ? d.kv_heads * parts : 0)));
        bytes = w.used;
    }
};

AttnArgs args_of(const adam_attn_desc &d)
{
    AttnArgs a = {};
    a.q = Heads{(void *)d.q, d.q_stride, d.q_head_stride};
    a.k = Heads{(void *)d.k, d.k_stride, d.k_head_stride};
    a.v = Heads{(void *)d.v, d.v_stride, d.v_head_stride};
    a.o = Heads{d.o, d.o_stride, d.o_head_stride};
    a.lse = d.lse;
    a.offsets = d.doc_offsets;
    a.prefix = d.prefix;
    a.slopes = d.slopes;
    a.rows = int32_t(d.rows);
    a.docs = int32_t(d.docs);
    a.heads = int32_t(d.heads);
    a.kv_heads = int32_t(d.kv_heads);
    a.dim = int32_t(d.head_dim);
    a.causal = d.causal;
    a.window = d.window >= d.rows ? 0 : int32_t(d.window);  // one that spans the batch hides nothing
    a.scale = d.scale;
    a.softcap = d.softcap;
    a.tiles = int32_t((d.rows + kOwnTile - 1) / kOwnTile);
    return a;
}

// Whether every 8 values of a row lie at a multiple of 16 bytes.
bool direct(const Heads &h, int64_t dim)
{
    return aligned(h.p, 16) && h.stride % 8 == 0 && h.head_stride % 8 == 0 && dim % 8 == 0;
}

// Calls f(type, padded head dimension, direct, extra).
template <class F>
int with_attn(const adam_attn_desc &d, bool is_direct, F f)
{
    const bool extra = d.softcap > 0.0f || d.slopes != nullptr;
    auto flags = [&](auto t, auto dp) {
        if (!is_direct) return f(t, dp, std::false_type(), std::true_type());
        return extra ? f(t, dp, std::true_type(), std::true_type()) : f(t, dp, std::true_type(), std::false_type());
    };
    auto dims = [&](auto t) {
        if (d.head_dim <= 64) return flags(t, std::integral_constant<int, 64>());
        if (d.head_dim <= 128) return flags(t, std::integral_constant<int, 128>());
        return flags(t, std::integral_constant<int, 256>());
    };
    return d.type == ADAM_DT_BF16 ? dims(bf16()) : dims(f16());
}

}  // namespace
}  // namespace train

using namespace train;

extern "C" {

int adam_attn_plan(const adam_attn_desc *desc, adam_attn_stats *stats)
{
    if (stats == nullptr) return ADAM_EINVAL;
    const int rc = check_attn(desc);
    if (rc != ADAM_OK) return rc;
    const bool none = desc->rows == 0 || desc->docs == 0;
    stats->forward_bytes = none ? 0 : AttnPlan(*desc, false, nullptr).bytes;
    stats->backward_bytes = none ? 0 : AttnPlan(*desc, true, nullptr).bytes;
    return ADAM_OK;
}

int adam_attn_forward(const adam_attn_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    const int rc = check_attn(desc);
    if (rc != ADAM_OK) return rc;
    const adam_attn_desc &d = *desc;
    if (!valid_strides(d.q_stride, d.q_head_stride) || !valid_strides(d.k_stride, d.k_head_stride) ||
        !valid_strides(d.v_stride, d.v_head_stride) || !valid_strides(d.o_stride, d.o_head_stride))
        return ADAM_EINVAL;
    if (d.rows == 0 || d.docs == 0) return ADAM_OK;
    if (d.q == nullptr || d.k == nullptr || d.v == nullptr || d.o == nullptr || !aligned(d.q, 2) || !aligned(d.k, 2) ||
        !aligned(d.v, 2) || !aligned(d.o, 2) || !aligned(d.lse, 4) || !aligned(d.doc_offsets, 4) ||
        !aligned(d.prefix, 4) || !aligned(d.slopes, 4))
        return ADAM_EINVAL;
    const AttnPlan plan(d, false, workspace);
    if (workspace == nullptr || workspace_bytes < plan.bytes || !aligned(workspace, 256)) return ADAM_EINVAL;
    const HeadView in[6] = {view(d.q, d.rows, d.heads, d.head_dim, d.q_stride, d.q_head_stride, 2),
                            view(d.k, d.rows, d.kv_heads, d.head_dim, d.k_stride, d.k_head_stride, 2),
                            view(d.v, d.rows, d.kv_heads, d.head_dim, d.v_stride, d.v_head_stride, 2),
                            flat_view(d.doc_offsets, (d.docs + 1) * 4), flat_view(d.prefix, d.docs * 4),
                            flat_view(d.slopes, d.heads * 4)};
    const HeadView out[3] = {view(d.o, d.rows, d.heads, d.head_dim, d.o_stride, d.o_head_stride, 2),
                             flat_view(d.lse, d.heads * d.rows * 4), flat_view(workspace, plan.bytes)};
    for (int i = 0; i < 3; ++i) {
        if (!out[i].distinct()) return ADAM_EINVAL;
        for (const HeadView &v : in)
            if (overlap(out[i], v)) return ADAM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return ADAM_EINVAL;
    }
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    AttnArgs a = args_of(d);
    a.flags = plan.flags;
    const bool is_direct = direct(a.q, d.head_dim) && direct(a.k, d.head_dim) && direct(a.v, d.head_dim) &&
                           direct(a.o, d.head_dim);
    return with_attn(d, is_direct, [&](auto t, auto dp, auto dir, auto extra) {
        hipLaunchKernelGGL((attn_forward_kernel<decltype(t), decltype(dp)::value, decltype(dir)::value,
                                                decltype(extra)::value>),
                           dim3(uint32_t(a.tiles * a.heads)), dim3(kAttnThreads), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
        hipLaunchKernelGGL((attn_forward_careful_kernel<decltype(t), decltype(dp)::value>),
                           dim3(uint32_t(std::min(a.tiles * a.heads, kCarefulGroups))), dim3(kAttnThreads), 0, stream,
                           a);
        return launched();
    });
}

int adam_attn_backward(const adam_attn_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    const int rc = check_attn(desc);
    if (rc != ADAM_OK) return rc;
    const adam_attn_desc &d = *desc;
    if (!valid_strides(d.q_stride, d.q_head_stride) || !valid_strides(d.k_stride, d.k_head_stride) ||
        !valid_strides(d.v_stride, d.v_head_stride) || !valid_strides(d.o_stride, d.o_head_stride) ||
        !valid_strides(d.dout_stride, d.dout_head_stride) || !valid_strides(d.dq_stride, d.dq_head_stride) ||
        !valid_strides(d.dk_stride, d.dk_head_stride) || !valid_strides(d.dv_stride, d.dv_head_stride))
        return ADAM_EINVAL;
    if (d.rows == 0 || d.docs == 0) return ADAM_OK;
    for (const void *p : {d.q, d.k, d.v, (const void *)d.o, d.dout, (const void *)d.dq, (const void *)d.dk,
                          (const void *)d.dv})
        if (p == nullptr || !aligned(p, 2)) return ADAM_EINVAL;
    if (d.lse == nullptr || !aligned(d.lse, 4) || !aligned(d.doc_offsets, 4) || !aligned(d.prefix, 4) ||
        !aligned(d.slopes, 4))
        return ADAM_EINVAL;
    const AttnPlan plan(d, true, workspace);
    if (workspace == nullptr || workspace_bytes < plan.bytes || !aligned(workspace, 256)) return ADAM_EINVAL;
    const HeadView in[9] = {view(d.q, d.rows, d.heads, d.head_dim, d.q_stride, d.q_head_stride, 2),
                            view(d.k, d.rows, d.kv_heads, d.head_dim, d.k_stride, d.k_head_stride, 2),
                            view(d.v, d.rows, d.kv_heads, d.head_dim, d.v_stride, d.v_head_stride, 2),
                            view(d.o, d.rows, d.heads, d.head_dim, d.o_stride, d.o_head_stride, 2),
                            view(d.dout, d.rows, d.heads, d.head_dim, d.dout_stride, d.dout_head_stride, 2),
                            flat_view(d.lse, d.heads * d.rows * 4), flat_view(d.doc_offsets, (d.docs + 1) * 4),
                            flat_view(d.prefix, d.docs * 4), flat_view(d.slopes, d.heads * 4)};
    const HeadView out[4] = {view(d.dq, d.rows, d.heads, d.head_dim, d.dq_stride, d.dq_head_stride, 2),
                             view(d.dk, d.rows, d.kv_heads, d.head_dim, d.dk_stride, d.dk_head_stride, 2),
                             view(d.dv, d.rows, d.kv_heads, d.head_dim, d.dv_stride, d.dv_head_stride, 2),
                             flat_view(workspace, plan.bytes)};
    for (int i = 0; i < 4; ++i) {
        if (!out[i].distinct()) return ADAM_EINVAL;
        for (const HeadView &v : in)
            if (overlap(out[i], v)) return ADAM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return ADAM_EINVAL;
    }
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    AttnArgs a = args_of(d);
    a.dout = Heads{(void *)d.dout, d.dout_stride, d.dout_head_stride};
    a.dq = Heads{d.dq, d.dq_stride, d.dq_head_stride};
    a.dk = Heads{d.dk, d.dk_stride, d.dk_head_stride};
    a.dv = Heads{d.dv, d.dv_stride, d.dv_head_stride};
    a.flags = plan.flags;
    a.numbers = plan.numbers;
    a.sums = plan.sums;
    a.parts = int32_t(plan.parts);
    bool is_direct = true;
    for (const Heads &h : {a.q, a.k, a.v, a.o, a.dout, a.dq, a.dk, a.dv}) is_direct &= direct(h, d.head_dim);
    return with_attn(d, is_direct, [&](auto t, auto dp, auto dir, auto extra) {
        using T = decltype(t);
        constexpr int DP = decltype(dp)::value;
        constexpr bool DIR = decltype(dir)::value, EXTRA = decltype(extra)::value;
        hipLaunchKernelGGL((attn_dq_kernel<T, DP, DIR, EXTRA>), dim3(uint32_t(a.tiles * a.heads)), dim3(kAttnThreads),
                           0, stream, a);
        if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
        hipLaunchKernelGGL((attn_dkdv_kernel<T, DP, DIR, EXTRA>), dim3(uint32_t(a.tiles * a.kv_heads * a.parts)),
                           dim3(kAttnThreads), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
        if constexpr (DP <= 128) {
            if (a.parts > 1) {
                hipLaunchKernelGGL((attn_join_kernel<T, DP, DIR>), dim3(uint32_t(a.tiles * a.kv_heads)),
                                   dim3(kAttnThreads), 0, stream, a);
                if (hipGetLastError() != hipSuccess) return int(ADAM_EHIP);
            }
        }
        hipLaunchKernelGGL((attn_backward_careful_kernel<T, DP>),
                           dim3(uint32_t(std::min(a.tiles * (a.heads + a.kv_heads * a.parts), kCarefulGroups))),
                           dim3(kAttnThreads), 0, stream, a);
        return launched();
    });
}

}  // extern "C"
