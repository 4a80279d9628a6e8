// What the training operators share: host-side checks, the device guard, the
// epilogues of the matrix product core and its work split.
#ifndef ADAMW_MI355X_TRAIN_H
#define ADAMW_MI355X_TRAIN_H

#include <algorithm>

#include "adam_train.h"
#include "gemm.h"

namespace train {

constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1;  // rows, columns, strides
// Strides that the matrix core's 32-bit offsets inside a 256-row tile allow.
constexpr int64_t kMaxDirectStride = int64_t(1) << 21;
// Rows that the products and the gathering of rows count in 32 bits.
constexpr int64_t kMaxProductRows = int64_t(1) << 30;
// Tiles of a product: a dispatch counts its work-items, 512 a tile, in 32 bits.
constexpr int64_t kMaxTiles = int64_t(1) << 22;

inline bool too_many_tiles(int64_t nx, int64_t ny)
{
    return ((nx + kTile - 1) / kTile) * ((ny + kTile - 1) / kTile) > kMaxTiles;
}

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

inline int dtype_bytes(adam_dtype t)
{
    return t == ADAM_DT_F32 ? 4 : t == ADAM_DT_BF16 || t == ADAM_DT_F16 ? 2 : 0;
}

inline bool is_half(adam_dtype t) { return t == ADAM_DT_BF16 || t == ADAM_DT_F16; }

// A row-major matrix in memory, for the overlap checks.  A NULL pointer or a
// matrix without elements overlaps nothing.
struct View {
    const void *p;
    int64_t rows, row_bytes, stride_bytes;
};

inline bool empty(const View &v) { return v.p == nullptr || v.rows <= 0 || v.row_bytes <= 0; }

// Whether two matrices share a byte.  Views of one parent (equal strides) may
// interleave: they are apart when their columns are.
inline bool overlap(const View &a, const View &b)
{
    if (empty(a) || empty(b)) return false;
    const int64_t a0 = int64_t(uintptr_t(a.p)), b0 = int64_t(uintptr_t(b.p));
    const int64_t a1 = a0 + (a.rows - 1) * a.stride_bytes + a.row_bytes;
    const int64_t b1 = b0 + (b.rows - 1) * b.stride_bytes + b.row_bytes;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.stride_bytes != b.stride_bytes || a.stride_bytes == 0) return true;
    // columns of b relative to a's rows, in [0, stride)
    int64_t d = (b0 - a0) % a.stride_bytes;
    if (d < 0) d += a.stride_bytes;
    return d < a.row_bytes || d + b.row_bytes > a.stride_bytes;
}

inline View matrix(const void *p, int64_t rows, int64_t cols, int64_t stride, int bytes)
{
    return View{p, rows, cols * bytes, stride * bytes};
}

inline View flat(const void *p, int64_t bytes) { return View{p, bytes > 0 ? 1 : 0, bytes, bytes}; }

inline bool aligned(const void *p, uintptr_t a) { return uintptr_t(p) % a == 0; }

// rows and columns in range, stride at least the columns.
inline bool valid_matrix(int64_t rows, int64_t cols, int64_t stride)
{
    return rows >= 0 && rows <= kMaxSize && cols >= 0 && cols <= kMaxSize && stride >= cols && stride <= kMaxSize;
}

// Makes the stream's device current for the life of the guard (a NULL stream:
// the current device stays).
struct StreamGuard {
    int previous = -1;
    bool switched = false;
    hipError_t status = hipSuccess;
    explicit StreamGuard(hipStream_t stream)
    {
        if (stream == nullptr) return;
        hipDevice_t device = 0;
        status = hipGetDevice(&previous);
        if (status == hipSuccess) status = hipStreamGetDevice(stream, &device);
        if (status == hipSuccess && device != previous) {
            status = hipSetDevice(device);
            switched = status == hipSuccess;
        }
        if (status != hipSuccess) (void)hipGetLastError();
    }
    ~StreamGuard()
    {
        if (switched) (void)hipSetDevice(previous);
    }
};

inline int launched() { return hipGetLastError() == hipSuccess ? ADAM_OK : ADAM_EHIP; }

// A bump allocator over the caller's workspace; with a NULL base it only adds
// up sizes, so that the plan and the call cannot disagree.
struct Workspace {
    char *base;
    int64_t used = 0;
    template <class P>
    P *take(int64_t count)
    {
        P *p = base == nullptr ? nullptr : (P *)(base + used);
        used += round_up(count * int64_t(sizeof(P)), 256);
        return p;
    }
};

// ---------------------------------------------------------------------------
// Epilogues
// ---------------------------------------------------------------------------

struct Nothing {};

// 8 elements at any alignment of their type: global accesses of 16 bytes need
// no more than that.
template <class O>
struct Loose;
template <>
struct Loose<bf16> {
    typedef vec<bf16, 8> type __attribute__((aligned(2)));
};
template <>
struct Loose<f16> {
    typedef vec<f16, 8> type __attribute__((aligned(2)));
};
template <>
struct Loose<float> {
    typedef vec<float, 8> type __attribute__((aligned(4)));
};

// Rows 32 y .. 32 y + 31 (j) of a wave's tile, 128 values each, through the
// wave's LDS: f(row, column, 8 values) with 16 lanes on a row, so that the
// stores of a row are whole 128-byte lines; from the registers' own layout a
// store would write 16 bytes to each of 16 rows.  16-byte chunk c of row j sits
// in slot c ^ j: neither the writes nor the reads conflict.
template <class F>
__device__ inline void by_rows(const Accumulators &acc, int y, char *lds, int lane, F f)
{
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int j = b * 16 + (lane & 15), chunk = x * 4 + (lane >> 4);
            *(vec<float, 4> *)(lds + j * 512 + ((chunk ^ j) << 4)) = acc.v[x][y * 2 + b];
        }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int row = k * 4 + (lane >> 4);
        const int chunk = (lane & 15) * 2;
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const vec<float, 4> p = *(const vec<float, 4> *)(lds + row * 512 + (((chunk + h) ^ row) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h * 4 + e] = p[e];
        }
        f(row, (lane & 15) * 8, v);
    }
}

constexpr int kTileFloats = kTile * kTile;

// A wave's sums of a tile's part into the workspace of the parts (part, row,
// column).
__device__ inline void store_part(const Accumulators &acc, float *parts, const TilePlace &place, int i0, int j0,
                                  char *lds, int lane)
{
    float *to = parts + int64_t(place.part) * kTileFloats + (j0 - place.y * kTile) * kTile + i0 - place.x * kTile;
#pragma unroll
    for (int y = 0; y < 2; ++y)
        by_rows(acc, y, lds, lane, [&](int row, int column, float (&v)[8]) {
            vec<float, 8> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = v[e];
            *(vec<float, 8> *)(to + (y * 32 + row) * kTile + column) = o;
        });
}

// N values of a split tile: the sum of its parts, in their order.
template <int N>
__device__ inline vec<float, N> sum_parts(const float *parts, const Rounds &r, int tile, int row, int column)
{
    const vec<float, N> *p = (const vec<float, N> *)(parts + int64_t(tile) * kTileFloats + row * kTile + column);
    vec<float, N> v = *p;
    for (int s = 1; s < r.splits; ++s) v += p[int64_t(s) * r.rest * (kTileFloats / N)];
    return v;
}

// out[row(j)][i] = (accumulate ? out : 0) + add + alpha * factor * acc, rounded
// once to O.  row(j) is j, or rows[j].
template <class O>
struct StoreEpilogue {
    O *out;
    int64_t stride;
    const float *alpha;   // NULL: 1
    float factor;         // a power of two beside alpha
    const int32_t *rows;  // NULL: j itself
    const float *add;     // a float matrix that is added too, or NULL
    int64_t add_stride;
    int32_t accumulate;
    int32_t pairs;        // 1: rows 2 n and 2 n + 1 are one sum, stored by the first
    float *parts;         // sums of tiles that are split over k: part, row, column

    __device__ Nothing prepare(int, int, int) const { return Nothing(); }

    __device__ void write8(int64_t j, int i, int nx, float s, float (&v)[8]) const
    {
        O *line = out + (rows != nullptr ? rows[j] : j) * stride;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= s;
        if (add != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < nx) v[e] += add[j * add_stride + i + e];
        }
        if (i + 8 <= nx) {
            typename Loose<O>::type *p = (typename Loose<O>::type *)(line + i);
            if (accumulate) {
                const vec<O, 8> old = *p;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += float(old[e]);
            }
            vec<O, 8> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = O(v[e]);
            // past the caches: the dw of a large vocabulary would push out what
            // the next products read (2 x 4096 x 98915: 605 us, 662 through them;
            // 1003 x 1000 x 50021: 353 and 373)
            __builtin_nontemporal_store(o, p);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < nx) line[i + e] = O(accumulate ? v[e] + float(line[i + e]) : v[e]);
        }
    }

    __device__ void operator()(const Accumulators &acc, Nothing, char *lds, const TilePlace &place, int i0, int j0,
                               int nx, int ny, int lane) const
    {
        if (place.part >= 0) {
            store_part(acc, parts, place, i0, j0, lds, lane);
            return;
        }
        const float s = alpha != nullptr ? *alpha * factor : factor;
#pragma unroll
        for (int y = 0; y < 2; ++y)
            by_rows(acc, y, lds, lane, [&](int row, int column, float (&v)[8]) {
                const int j = j0 + y * 32 + row;
                if (pairs) {  // the next row is 16 lanes on
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += __shfl_xor(v[e], 16);
                    if (row & 1) return;
                }
                if (j < ny && i0 + column < nx) write8(j, i0 + column, nx, s, v);
            });
    }
};

// Joins the parts of the split tiles in their order.  8 rows of a tile a
// workgroup, 8 values a thread.
template <class O>
__global__ __launch_bounds__(256) void join_parts(GemmArgs a, StoreEpilogue<O> e)
{
    const int extent_y = a.count != nullptr && !a.count_is_depth ? a.counted() : a.y.extent;
    const Rounds r = a.rounds_for(extent_y);
    const int tile = blockIdx.x >> 5;
    if (r.splits == 1 || tile >= r.rest) return;
    int x, y;
    tile_at(r.full + tile, a.tiles_x, a.tiles_y(extent_y), x, y);
    const int row = (blockIdx.x & 31) * 8 + (threadIdx.x >> 5), column = (threadIdx.x & 31) * 8;
    const int64_t j = int64_t(y) * kTile + row;
    const int i = x * kTile + column;
    if (j >= extent_y || i >= a.x.extent) return;
    vec<float, 8> v = sum_parts<8>(e.parts, r, tile, row, column);
    if (e.pairs) {
        if (row & 1) return;
        v += sum_parts<8>(e.parts, r, tile, row + 1, column);
    }
    float w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = v[c];
    e.write8(j, i, a.x.extent, e.alpha != nullptr ? *e.alpha * e.factor : e.factor, w);
}

// One matrix product's tiles, and the most workgroups, split tiles and parts
// that it has: where y's rows are counted on the device (`counted`), over all
// counts of tiles that it may come to.
struct Product {
    int32_t tiles_x;
    Rounds rounds;
    bool counted;
    int64_t units = 0, split_tiles = 0, parts = 0;

    Product(int64_t nx, int64_t ny, int64_t depth, bool counted_ = false) : counted(counted_)
    {
        tiles_x = int32_t((nx + kTile - 1) / kTile);
        const int tiles_y = int((ny + kTile - 1) / kTile);
        rounds = rounds_of(tiles_x * tiles_y, int(depth));
        for (int y = counted ? 1 : tiles_y; y <= tiles_y; ++y) {
            const Rounds r = rounds_of(tiles_x * y, int(depth));
            units = std::max<int64_t>(units, r.units());
            if (r.splits == 1) continue;
            split_tiles = std::max<int64_t>(split_tiles, r.rest);
            parts = std::max<int64_t>(parts, int64_t(r.rest) * r.splits);
        }
    }
    int64_t part_floats() const { return parts * kTileFloats; }
};

template <class T, int XM, int YM, class O>
int run_product(const Product &p, GemmArgs a, StoreEpilogue<O> e, float *parts, hipStream_t stream)
{
    a.tiles_x = p.tiles_x;
    a.rounds = p.rounds;
    a.replan = p.counted;
    e.parts = parts;
    hipLaunchKernelGGL((gemm_kernel<T, XM, YM, StoreEpilogue<O>>), dim3(uint32_t(p.units)), dim3(kThreads), 0,
                       stream, a, e);
    if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
    if (p.split_tiles == 0) return ADAM_OK;
    hipLaunchKernelGGL((join_parts<O>), dim3(uint32_t(p.split_tiles * 32)), dim3(256), 0, stream, a, e);
    return launched();
}

// A 16-bit matrix that the core reads where it lies: whole 16-byte chunks, and
// where k is contiguous, no chunk that reaches past it.
inline bool direct(const void *p, int64_t stride, int64_t cols, bool k_contiguous)
{
    return aligned(p, 16) && stride % 8 == 0 && stride <= kMaxDirectStride && (!k_contiguous || cols % 8 == 0);
}

// One row of 16-bit values copied into a row of `pitch` (a multiple of 8) with
// zeros behind the columns, by a workgroup of 256.
__device__ inline void copy_row(const uint16_t *from, int cols, uint16_t *to, int64_t pitch)
{
    typedef vec<uint16_t, 8> octet;
    typedef octet loose __attribute__((aligned(2)));
    for (int c = threadIdx.x * 8; c < pitch; c += 256 * 8) {
        octet v;
        if (c + 8 <= cols) {
            v = *(const loose *)(from + c);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? from[c + e] : uint16_t(0);
        }
        *(octet *)(to + c) = v;
    }
}

// Copies a matrix into rows of `pitch`.
int pack(const void *from, int64_t stride, int64_t rows, int64_t cols, void *to, int64_t pitch, hipStream_t stream);

}  // namespace train

#endif
