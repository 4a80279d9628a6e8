// Matrix product core of the training operators (gfx950, MFMA).
//
//   out[j][i] (+)= sum over k of Y(j, k) * X(i, k)
//
// i runs over the contiguous dimension of the output, j over its rows.  Each
// operand is a 16-bit matrix held either with k contiguous (kRows: row i holds
// its k values) or with k as the row index (kCols: row k holds the values of
// all i), or, for X, an 8-bit checkpoint with k as the row index.
//
// Layout.  A workgroup of 8 waves makes a 256 x 256 tile of the output; a wave
// holds 128 (i) x 64 (j) of it in 128 accumulator registers as 8 x 4 blocks of
// the 16x16x32 matrix instruction.  (With 4 x 2 blocks of the 32x32x16 one, which
// moves twice the accumulator bytes per product, the three products of cross
// entropy took 5% longer.)  Per 32 values of k a wave reads 12 KiB from LDS for
// 32 instructions of 16 cycles, so with two waves per SIMD the LDS supplies 96
// KiB per 1024 cycles, 3/8 of the 256 bytes a cycle that it was measured at.
//
// The tiles of four successive k steps live in LDS (4 x 32 KiB).  They arrive
// by buffer loads that write LDS directly (16 bytes a lane, no registers), three
// steps ahead of their use, with one barrier a step.  A wave reads its fragments
// half a step ahead of the products, so that the matrix unit does not wait
// behind the barrier.  Every load goes through a buffer descriptor: rows and k
// beyond the end read as 0 and no address outside the operand is touched, but
// for an odd last value's dword and, within its rows, what fills the last 16
// bytes of a row (the stride is a multiple of them).
//
// Bank layout.  A direct load places lane l's 16 bytes at base + 16 l, so the
// permutation that avoids bank conflicts is applied to the global address:
//   kRows tile: 256 rows x 64 bytes; 16-byte chunk c of row r sits in slot
//     c ^ row_twist(r).  A 16-byte read serves lanes 0-3, 12-15, 20-23, 24-27
//     (and so on) at once: rows 0-3 and 12-15 of one chunk, 4-11 of the next,
//     which then cover all 64 banks.
//   kCols tile: 32 rows (k) x 512 bytes; 32-byte unit u (16 values of i) of row
//     r sits in slot u ^ column_twist(r): the 4 rows x 32 bytes that a 16-lane
//     group of the transposing LDS read takes, and its neighbour's 8 rows on,
//     cover all banks.
//
// What bounds it: at 7373 x 131072 x 4096 in bf16 the matrix unit is busy 64-82%
// of the cycles, at 1.75-1.9 GHz: the card holds its power by its clock, and a
// library product of the same size runs at 81% and 1.7 GHz.  The accumulators and
// fragments leave few of the 256 registers: the kernels with k as the row index of
// both operands keep two (8-bit X) or four in scratch memory.
#ifndef ADAMW_MI355X_GEMM_H
#define ADAMW_MI355X_GEMM_H

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

namespace train {

using bf16 = __bf16;
using f16 = _Float16;
template <class T, int N>
using vec = T __attribute__((ext_vector_type(N)));
using f32x4 = vec<float, 4>;
using f16x4 = vec<f16, 4>;
using u32x4 = vec<uint32_t, 4>;

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kTile = 256;     // output tile, both ways
constexpr int kStep = 32;      // k values per step
constexpr int kStages = 4;     // steps held in LDS
constexpr int kThreads = 512;  // 8 waves
constexpr int kTileBytes = kTile * kStep * 2;
constexpr int kWaveBytes = kStages * 2 * kTileBytes / 8;  // LDS of a wave in the epilogue: 16 KiB
constexpr uint32_t kBufferWord3 = 0x00027000;  // raw buffer, 32-bit data format
constexpr uint32_t kOut = 0x80000000u;         // an offset beyond every descriptor (each is shorter than 2 GiB)

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The permutations of the bank layouts (see the top of the file).
__device__ inline int row_twist(int row)
{
    const int q = (row >> 2) & 3;
    return ((q & 1) << 1) ^ (q >> 1) * 3;  // 0, 2, 3, 1
}
__device__ inline int column_twist(int row) { return ((row & 3) << 1) ^ ((row >> 3) & 1); }

enum Mode { kRows = 0, kCols = 1, kE4M3 = 2, kE5M2 = 3 };

// The 16-bit types: matrix instruction, transposing LDS read, decoding.
template <class T>
struct Half;

template <>
struct Half<bf16> {
    static constexpr int kHalvings = 0;  // 8-bit values are decoded times 2^-kHalvings
    static __device__ f32x4 mfma(vec<bf16, 8> a, vec<bf16, 8> b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ vec<bf16, 4> read_transposed(const char *p)
    {
        typedef __attribute__((address_space(3))) vec<bf16, 4> at;
        return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((at *)p);
    }
    template <bool E4M3, bool HIGH>
    static __device__ vec<bf16, 2> decode(uint32_t codes, float scale)
    {
        return E4M3 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HIGH)
                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, scale, HIGH);
    }
};

// One halving: the 8-bit value nearest to an fp16 one may be 65536, which fp16
// does not hold.  (Its 4 significant bits stay down to 2^-20.)
template <>
struct Half<f16> {
    static constexpr int kHalvings = 1;
    static __device__ f32x4 mfma(vec<f16, 8> a, vec<f16, 8> b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ vec<f16, 4> read_transposed(const char *p)
    {
        typedef __attribute__((address_space(3))) vec<__fp16, 4> at;
        return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((at *)p));
    }
    template <bool E4M3, bool HIGH>
    static __device__ vec<f16, 2> decode(uint32_t codes, float scale)
    {
        return E4M3 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, HIGH)
                    : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(codes, scale, HIGH);
    }
};

// One operand.  kRows: `extent` rows of `depth` values; kCols and the 8-bit
// modes: `depth` rows of `extent` values.  Strides in elements.
struct Operand {
    const void *base;
    const uint8_t *scales;  // 8-bit modes: one byte per 32 values of a row
    int64_t stride;         // below 2^21
    int32_t extent;
    int32_t depth;
};

// How the tiles of a product go round the 256 compute units: the first `full`
// tiles (a multiple of 256) are made by one workgroup each; the `rest`, which
// would leave units idle, are split over k into `splits` parts each, whose
// float sums meet in a workspace.
struct Rounds {
    int32_t full, rest, splits;
    int32_t steps;  // of a part (a whole tile takes all): a multiple of kStages

    __host__ __device__ int units() const { return full + rest * splits; }
};

constexpr int kUnits = 256;      // compute units
constexpr int kMostSplits = 16;
constexpr int kMostParts = 5 * kUnits;  // 320 MiB of sums

// Chooses the split of the rest: the one whose rounds take the fewest k steps,
// where a round pays about 8 for its start and end, a part 1/8 for its sums'
// way through memory (256 KiB written and read at 4 MiB a step of all units),
// and joining 8 more.  (With 2 or 4 for joining, or half the way through memory,
// ten sizes of weight gradients and cross entropy took -3 to +10% longer.)
__host__ __device__ inline Rounds rounds_of(int tiles, int depth)
{
    const int steps = (depth + kStep - 1) / kStep;
    Rounds r;
    r.full = tiles / kUnits * kUnits;
    r.rest = tiles - r.full;
    r.splits = 1;
    if (r.rest > 0) {
        int64_t least = 0;
        for (int s = 1; s <= kMostSplits; ++s) {
            if (s > 1 && (steps / s < 8 || r.rest * s > kMostParts)) break;
            const int64_t cost = int64_t(8) * ((r.rest * s + kUnits - 1) / kUnits) * ((steps + s - 1) / s + 8) +
                             (s > 1 ? r.rest * s + 64 : 0);
            if (s == 1 || cost < least) {
                least = cost;
                r.splits = s;
            }
        }
    }
    r.steps = ((steps + r.splits - 1) / r.splits + kStages - 1) / kStages * kStages;
    return r;
}

struct GemmArgs {
    Operand x, y;
    int32_t tiles_x;
    Rounds rounds;
    // Where `count` is set, rows *count - first (at least 0, at most `most`)
    // replace y's extent (count_is_depth 0) or both depths (1): the number of
    // rows is known on the device only.  With `replan` the rounds are chosen
    // again for that extent.
    const int32_t *count;
    int32_t first, most, count_is_depth, replan;

    __device__ int counted() const
    {
        const int n = *count - first;
        return n < 0 ? 0 : n > most ? most : n;
    }
    // The tiles of y that the rounds cover: without a new plan all of them, of
    // which those past the counted rows make nothing.
    __device__ int tiles_y(int extent_y) const { return ((replan ? extent_y : y.extent) + kTile - 1) / kTile; }
    __device__ Rounds rounds_for(int extent_y) const
    {
        if (!replan) return rounds;
        return rounds_of(tiles_x * tiles_y(extent_y), x.depth > y.depth ? x.depth : y.depth);
    }
};

// What a workgroup makes.
struct TilePlace {
    int x, y;
    int split;   // which part of k
    int part;    // its place in the workspace of the parts, or -1: the whole tile
    bool none;
};

// A tile's coordinates: 4 tiles of y by 1 of x come first, so that the 32
// workgroups that an XCD runs at once share 4 y and 8 x tiles through its L2.
// Groups of 2, 3, 5, 6, 8 and 16 took 2 to 16% longer over the three products of
// cross entropy (18.6 ms with 4, 19.0 with 8, 21.6 with 16 at 7373 x 131072 x
// 4096), and so did squares of 16 x 16 tiles shared out over the XCDs (19.0).
// Elsewhere 2 and 8 took 0 to 3% longer (losses of 2048 x 4096 x 131072, training
// at 2048 x 2048 x 32768 and 1003 x 1000 x 50021, weight gradients of 8192 x 4096 x
// 14336 and 8192 x 28672 x 4096), but at 4096 x 4096 x 4096, one round of 256
// tiles, 8% less: 119 and 121 us, 130 with 4.
constexpr int kGroup = 4;

__device__ inline void tile_at(int t, int tiles_x, int tiles_y, int &x, int &y)
{
    const int group = t / (kGroup * tiles_x);
    const int y0 = group * kGroup;
    const int height = tiles_y - y0 < kGroup ? tiles_y - y0 : kGroup;
    t -= group * kGroup * tiles_x;
    x = t / height;
    y = y0 + t - x * height;
}

// Workgroup -> tile and part.  Workgroups go round the 8 XCDs in turn, so each
// XCD is given a contiguous eighth of the full tiles, and of the parts.
__device__ inline TilePlace place_of(const Rounds &r, int tiles_x, int tiles_y)
{
    const bool whole = int(blockIdx.x) < r.full;
    const int total = whole ? r.full : r.rest * r.splits;
    const int id = whole ? blockIdx.x : blockIdx.x - r.full;
    TilePlace p;
    p.none = id >= total;
    const int xcd = id & 7, q = total >> 3, m = total & 7;
    const int t = xcd * q + (xcd < m ? xcd : m) + (id >> 3);
    if (p.none) return p;
    p.split = whole ? 0 : t / r.rest;
    const int tile = whole ? t : r.full + t - p.split * r.rest;
    p.part = whole || r.splits == 1 ? -1 : t;
    tile_at(tile, tiles_x, tiles_y, p.x, p.y);
    return p;
}

// What a descriptor of a step's tile may reach, in bytes: everything before the
// last step (32 whole rows, and more behind them), the exact rest in the last
// one, nothing after it.
struct Reach {
    int32_t steps;  // left, the present one among them
    int32_t last;   // bytes of the last

    __device__ void init(int depth, int step, int64_t row_bytes, int64_t part_bytes)
    {
        steps = (depth + kStep - 1) / kStep - step;
        last = int32_t(((depth - 1) & (kStep - 1)) * row_bytes + part_bytes);
    }
    __device__ int32_t records() const { return steps > 1 ? 0x7fffffff : steps == 1 ? last : 0; }
};

// Loads one operand's tiles into LDS, one k step after the other.  Tiles past
// the depth read as 0.
template <class T, int MODE>
struct Loader {
    const char *at;       // the next tile's first value
    int64_t advance;      // bytes from one tile to the next
    uint32_t offset[2];   // the lane's offset of each load
    int32_t k_left;       // kRows: values of k left, less the lane's place in a step
    Reach reach;          // kCols
    int wave;

    __device__ void init(const Operand &o, int tile, int extent, int depth, int step)
    {
        const int tid = threadIdx.x;
        wave = uniform(tid >> 6);
        const int64_t row_bytes = o.stride * 2;
        const int first = tile * kTile;
        const int valid = extent - first < kTile ? extent - first : kTile;
        if (MODE == kRows) {
            advance = kStep * 2;
            at = (const char *)o.base + first * row_bytes + step * advance;
            for (int s = 0; s < 2; ++s) {
                const int row = s * 128 + (tid >> 2);
                const int chunk = (tid & 3) ^ row_twist(row);
                k_left = depth - step * kStep - chunk * 8;  // the same for both: rows 128 apart
                offset[s] = row < valid ? uint32_t(row * row_bytes) + chunk * 16 : kOut;
            }
        } else {
            advance = kStep * row_bytes;
            at = (const char *)o.base + int64_t(first) * 2 + step * advance;
            // to a whole dword: an odd last value shares its dword, which the
            // allocation holds (the base is 16-byte aligned), with a value
            // that no stored output uses
            reach.init(depth, step, row_bytes, (valid * 2 + 3) & ~3);
            for (int s = 0; s < 2; ++s) {
                const int row = s * 16 + (tid >> 5);
                const int slot = tid & 31;
                const int column = (((slot >> 1) ^ column_twist(row)) << 4) + ((slot & 1) << 3);
                offset[s] = column < valid ? uint32_t(row * row_bytes) + column * 2 : kOut;
            }
        }
    }

    // The tile `ahead` steps past the next one, which lies before the last one.
    __device__ void issue_inside(char *stage, int ahead) const
    {
        __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc((void *)at, short(0), 0x7fffffff, kBufferWord3);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(stage + s * (kThreads * 16) + wave * 1024), 16,
                                                     int(offset[s]), ahead * int(advance), 0, 0);
    }
    __device__ void skip(int steps)
    {
        at += steps * advance;
        if (MODE == kRows)
            k_left -= steps * kStep;
        else
            reach.steps -= steps;
    }

    __device__ void issue(char *stage)
    {
        // kRows: a lane reads its 16 bytes only where all of them are valid
        __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void *)at, short(0), MODE == kRows ? 0x7fffffff : reach.records(), kBufferWord3);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t lane_at = offset[s];
            if (MODE == kRows) lane_at = k_left > 0 ? lane_at : kOut;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(stage + s * (kThreads * 16) + wave * 1024), 16,
                                                     int(lane_at), 0, 0, 0);
        }
        at += advance;
        if (MODE == kRows)
            k_left -= kStep;
        else
            --reach.steps;
    }
};

// A thread's part of an 8-bit tile.
struct CodeRegs {
    u32x4 codes;
    uint32_t scale;
};

// The 8-bit X tile of a step: 32 rows of 256 codes, 16 codes (half a scale
// block) and their scale byte a thread, through registers: decoded to T
// (cvt_scalef32 applies the scale's exponent exactly) and written as one
// 32-byte unit of a kCols tile.
template <class T, int MODE>
struct Loader8 {
    static constexpr bool kE4 = MODE == kE4M3;
    const char *codes, *scales;  // the next tile's
    int64_t advance, scales_advance;
    Reach reach, scales_reach;
    uint32_t offset, scale_offset;
    uint32_t place;  // LDS offset of the thread's unit

    __device__ void init(const Operand &o, int tile, int, int depth, int step)
    {
        const int row = threadIdx.x >> 4, unit = threadIdx.x & 15;
        const int first = tile * kTile;
        const int pitch = int(o.stride);
        const int valid = pitch - first < kTile ? pitch - first : kTile;  // a multiple of 32
        advance = int64_t(kStep) * pitch;
        scales_advance = int64_t(kStep) * (pitch >> 5);
        codes = (const char *)o.base + first + step * advance;
        scales = (const char *)o.scales + (first >> 5) + step * scales_advance;
        reach.init(depth, step, pitch, valid);
        scales_reach.init(depth, step, pitch >> 5, valid >> 5);
        offset = unit * 16 < valid ? uint32_t(row * pitch) + unit * 16 : kOut;
        scale_offset = unit * 16 < valid ? uint32_t(row * (pitch >> 5)) + (unit >> 1) : kOut;
        place = row * 512 + ((unit ^ column_twist(row)) << 5);
    }

    __device__ CodeRegs load()
    {
        __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc((void *)codes, short(0), reach.records(), kBufferWord3);
        __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)scales, short(0), scales_reach.records(), kBufferWord3);
        CodeRegs g;
        g.codes = __builtin_amdgcn_raw_buffer_load_b128(r, int(offset), 0, 0);
        g.scale = __builtin_amdgcn_raw_buffer_load_b8(rs, int(scale_offset), 0, 0);
        codes += advance;
        scales += scales_advance;
        --reach.steps;
        --scales_reach.steps;
        return g;
    }

    __device__ CodeRegs load_inside(int ahead) const
    {
        __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc((void *)codes, short(0), 0x7fffffff, kBufferWord3);
        __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)scales, short(0), 0x7fffffff, kBufferWord3);
        CodeRegs g;
        g.codes = __builtin_amdgcn_raw_buffer_load_b128(r, int(offset), ahead * int(advance), 0);
        g.scale = __builtin_amdgcn_raw_buffer_load_b8(rs, int(scale_offset), ahead * int(scales_advance), 0);
        return g;
    }
    __device__ void skip(int steps)
    {
        codes += steps * advance;
        scales += steps * scales_advance;
        reach.steps -= steps;
        scales_reach.steps -= steps;
    }

    __device__ void commit(const CodeRegs &g, char *stage) const
    {
        // (2^-127, as which 0 is taken, is not halved: its values are 0 in fp16
        // both ways)
        float scale = __uint_as_float(g.scale << 23);
        if (Half<T>::kHalvings > 0) scale *= 1.0f / (1 << Half<T>::kHalvings);
        uint32_t w[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            w[2 * d] = __builtin_bit_cast(uint32_t, (Half<T>::template decode<kE4, false>(g.codes[d], scale)));
            w[2 * d + 1] = __builtin_bit_cast(uint32_t, (Half<T>::template decode<kE4, true>(g.codes[d], scale)));
        }
        *(u32x4 *)(stage + place) = u32x4{w[0], w[1], w[2], w[3]};
        *(u32x4 *)(stage + place + 16) = u32x4{w[4], w[5], w[6], w[7]};
    }
};

// A lane's place in a tile's fragments (16 rows, the 32 values of k of the
// step): lane l holds row l % 16 and the 8 values of k that start at 8 (l / 16).
template <int MODE>
__device__ inline uint32_t place_in_fragment(int lane)
{
    if (MODE == kRows) return (lane & 15) * 64 + (((lane >> 4) ^ row_twist(lane)) << 4);
    const int row = ((lane >> 4) << 3) + ((lane & 15) >> 2);
    return row * 512 + (column_twist(row) << 5) + ((lane & 3) << 3);
}

// The fragment of rows first .. first + 15 (first a multiple of 16).  kCols: the
// transposing read fills the 8 values in two parts of 4 rows of k each.
template <class T, int MODE>
__device__ inline vec<T, 8> fragment(const char *stage, int first, uint32_t place)
{
    if (MODE == kRows) return *(const vec<T, 8> *)(stage + first * 64 + place);
    const char *p = stage + (place ^ (uint32_t(first) << 1));
    const vec<T, 4> a = Half<T>::read_transposed(p);
    const vec<T, 4> b = Half<T>::read_transposed(p + 4 * 512);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Waits until at most N of this wave's loads are outstanding, and for all its
// LDS accesses: its reads of a stage are done before another wave may load it.
template <int N>
__device__ inline void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

__device__ inline void barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Accumulators of a wave: v[x][y] is a 16 x 16 block; in it lane l, register r
// hold i = 4 (l / 16) + r and j = l % 16.
struct Accumulators {
    f32x4 v[8][4];
};

// The fragments of half a step: half of X's, and all of Y's.
template <class T>
struct Fragments {
    vec<T, 8> x[4];
};
template <class T>
struct YFragments {
    vec<T, 8> y[4];
};

template <class T, int MODE>
__device__ inline void read_x(Fragments<T> &f, const char *stage, int half, int wx, uint32_t place)
{
#pragma unroll
    for (int x = 0; x < 4; ++x) f.x[x] = fragment<T, MODE>(stage, wx + half * 64 + x * 16, place);
}

template <class T, int MODE>
__device__ inline void read_y(YFragments<T> &f, const char *stage, int wy, uint32_t place)
{
#pragma unroll
    for (int y = 0; y < 4; ++y) f.y[y] = fragment<T, MODE>(stage + kTileBytes, wy + y * 16, place);
}

// Orders the instructions of half a step: the 16 products, one of the LDS reads
// for the next half behind each of the first ones, so that they are all on
// their way early and none delays a product; then the loads of the tile that is
// furthest ahead.  (Left alone, the compiler puts each read right before its
// use and waits for it.)
template <int READS, int LOADS>
__device__ inline void order_half()
{
    constexpr int kScalar = 0x4, kProduct = 0x8, kLoad = 0x10, kRead = 0x100;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
        if (k < READS) __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
        if (LOADS > 0 && k >= 4) {
            __builtin_amdgcn_sched_group_barrier(kScalar, 3, 0);
            if (k >= 16 - 2 * LOADS && k % 2 == 0) __builtin_amdgcn_sched_group_barrier(kLoad, 1, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// One step of a wave.  Its first half's fragments are in registers already;
// the second half's are read under the first half's products, and the next
// step's first under the second half's, so the matrix unit does not wait for
// LDS after the barrier.  The four stages are distinct; `restrict` says so, or
// the compiler would wait for the loads into `next` before it reads the others.
template <class T, int XMODE, int YMODE, bool INSIDE, class LX, class LY>
__device__ __attribute__((always_inline)) inline void run_step(Accumulators &acc, Fragments<T> &first,
                                                               YFragments<T> &y,
                                                               const char *__restrict now,
                                                               const char *__restrict soon, char *__restrict after,
                                                               char *__restrict next, LX &lx, LY &ly, CodeRegs &ready,
                                                               CodeRegs &loading, int ahead, int wx, int wy,
                                                               uint32_t place_x, uint32_t place_y)
{
    constexpr bool k8 = XMODE >= kE4M3;
    constexpr int kXTile = k8 ? kCols : XMODE;
    constexpr int kXReads = kXTile == kCols ? 8 : 4, kYReads = YMODE == kCols ? 8 : 4;
    Fragments<T> second;
    read_x<T, kXTile>(second, now, 1, wx, place_x);
    if constexpr (INSIDE) {
        if constexpr (k8)
            loading = lx.load_inside(ahead);
        else
            lx.issue_inside(next, ahead);
        ly.issue_inside(next + kTileBytes, ahead);
    } else {
        if constexpr (k8)
            loading = lx.load();
        else
            lx.issue(next);
        ly.issue(next + kTileBytes);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc.v[x][j] = Half<T>::mfma(first.x[x], y.y[j], acc.v[x][j]);
    order_half<kXReads, 4>();
    read_x<T, kXTile>(first, soon, 0, wx, place_x);
    if constexpr (k8) lx.commit(ready, after);
    // y by y: the registers of each are free for the next step's when its last
    // product is under way
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) acc.v[4 + x][j] = Half<T>::mfma(second.x[x], y.y[j], acc.v[4 + x][j]);
        y.y[j] = fragment<T, YMODE>(soon + kTileBytes, wy + j * 16, place_y);
    }
    order_half<kXReads + kYReads, 0>();
}

// The last step from which kStages steps load, each kStages - 1 ahead, only tiles
// that lie before the last one of `depth`: there a row read in whole 16-byte
// chunks is followed by another.  The last tile's own descriptor ends where the
// operand does.
__host__ __device__ constexpr int last_inside(int depth) { return (depth - 1) / kStep - 2 * kStages + 1; }

// Steps past the depth (a part's count is a multiple of kStages) multiply zeros.
//
// An epilogue's prepare() runs before the products (for loads that they hide);
// its call operator gets the wave's accumulators and 16 KiB of LDS.
template <class T, int XMODE, int YMODE, class Epilogue>
__global__ __launch_bounds__(kThreads, 2) void gemm_kernel(GemmArgs a, Epilogue epilogue)
{
    __shared__ __attribute__((aligned(1024))) char lds[kStages * 2 * kTileBytes];
    int extent_y = a.y.extent, depth_x = a.x.depth, depth_y = a.y.depth;
    if (a.count != nullptr) {
        const int n = uniform(a.counted());
        if (a.count_is_depth)
            depth_x = depth_y = n;
        else
            extent_y = n;
    }
    const Rounds rounds = a.rounds_for(extent_y);
    const TilePlace place = place_of(rounds, a.tiles_x, a.tiles_y(extent_y));
    if (place.none || place.y * kTile >= extent_y) return;
    const int depth = depth_x > depth_y ? depth_x : depth_y;
    int step = 0;
    int end = (depth + kStep - 1) / kStep;
    if (place.part >= 0) {
        step = place.split * rounds.steps;
        if (end > step + rounds.steps) end = step + rounds.steps;
    }

    constexpr bool k8 = XMODE >= kE4M3;
    constexpr int kXTile = k8 ? kCols : XMODE;  // how the X tile lies in LDS
    std::conditional_t<k8, Loader8<T, XMODE>, Loader<T, kXTile>> lx;
    Loader<T, YMODE> ly;
    lx.init(a.x, place.x, a.x.extent, depth_x, step);
    ly.init(a.y, place.y, extent_y, depth_y, step);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wx = (wave & 1) * 128, wy = (wave >> 1) * 64;

    const auto ahead = epilogue.prepare(place.y * kTile + wy, extent_y, lane);
    Accumulators acc;
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc.v[x][y] = f32x4(0.0f);

    // 8-bit X: the tile of step t + 3 is loaded into registers at step t and
    // written to LDS in step t + 1
    CodeRegs regs[2];
    if constexpr (k8) {
        regs[0] = lx.load();
        regs[1] = lx.load();
        lx.commit(regs[0], lds);
        lx.commit(regs[1], lds + 2 * kTileBytes);
        regs[0] = lx.load();
    }
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if constexpr (!k8) lx.issue(lds + s * 2 * kTileBytes);
        ly.issue(lds + s * 2 * kTileBytes + kTileBytes);
    }
    // Loads of a step, X and Y together: 4 (8-bit X: 2 into registers, first).
    // Here the first step's have to be there; the 8-bit form, whose prologue
    // has fewer in flight, waits for the second's too.
    wait_loads<k8 ? 2 : 8>();
    barrier();
    Fragments<T> first;
    YFragments<T> y;
    const uint32_t place_x = place_in_fragment<kXTile>(lane), place_y = place_in_fragment<YMODE>(lane);
    read_x<T, kXTile>(first, lds, 0, wx, place_x);
    read_y<T, YMODE>(y, lds, wy, place_y);
    auto run_stages = [&](auto inside) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            // this wave's loads of the next step have landed, then every
            // wave's; and every wave has read the stage that is written next
            wait_loads<4>();
            barrier();
            char *stage[kStages];
#pragma unroll
            for (int k = 0; k < kStages; ++k) stage[k] = lds + ((s + k) % kStages) * 2 * kTileBytes;
            run_step<T, XMODE, YMODE, decltype(inside)::value>(acc, first, y, stage[0], stage[1], stage[2], stage[3],
                                                               lx, ly, regs[s & 1], regs[(s + 1) & 1], s, wx, wy,
                                                               place_x, place_y);
        }
    };
    // While the tiles that are loaded lie before the last one, no load is limited
    // and an operand's base moves once in kStages steps.
    const int inside = last_inside(depth_x < depth_y ? depth_x : depth_y);
    for (; step < end && step <= inside; step += kStages) {
        run_stages(std::true_type());
        lx.skip(kStages);
        ly.skip(kStages);
    }
    for (; step < end; step += kStages) run_stages(std::false_type());
    // loads issued past the end are still on their way to LDS; then each wave
    // has 16 KiB of it for its epilogue
    wait_loads<0>();
    barrier();
    epilogue(acc, ahead, lds + wave * kWaveBytes, place, place.x * kTile + wx, place.y * kTile + wy, a.x.extent,
             extent_y, lane);
}

}  // namespace train

#endif
