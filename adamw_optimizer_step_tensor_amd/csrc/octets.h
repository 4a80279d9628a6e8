// Streaming over row-major matrices in groups of 8 elements: what the 8-bit
// checkpoints, the gated activation and the embedding share.
#ifndef ADAMW_MI355X_OCTETS_H
#define ADAMW_MI355X_OCTETS_H

#include "train.h"

namespace train {

constexpr int kBlock = 256;
constexpr int64_t kMaxGrid = 1 << 22;

// 8 values from `col` on, a multiple of 8 up to 2^31 - 8, so that col + 8 may not
// fit an int.
template <class T>
__device__ inline void load8(const T *row, int col, int cols, float (&v)[8])
{
    if (col <= cols - 8) {
        const vec<T, 8> p = __builtin_nontemporal_load((const typename Loose<T>::type *)(row + col));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = float(p[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = col + e < cols ? float(row[col + e]) : 0.0f;
    }
}

// v is rounded to float before it is rounded to T: the compiler would otherwise
// join a product and its conversion to fp16 in some kernels and not in others.
template <class T>
__device__ inline void store8(T *row, int col, int cols, float (&v)[8])
{
    if (std::is_same<T, f16>::value) {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm("" : "+v"(v[e]));
    }
    if (col <= cols - 8) {
        typename Loose<T>::type p;
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = T(v[e]);
        __builtin_nontemporal_store(p, (typename Loose<T>::type *)(row + col));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < cols) row[col + e] = T(v[e]);
    }
}

// Which group of 8 elements a thread works on.
struct Position {
    int64_t row;
    int col;
};

// Groups of a rows x pitch matrix, numbered along its rows.  A workgroup takes
// kBlock * N in a row: one 64-bit division a workgroup, a 32-bit one a
// thread.
struct Walk {
    int64_t row0;
    uint32_t rest, per_row;
    __device__ Walk(int64_t first, uint32_t per_row_) : per_row(per_row_)
    {
        row0 = first / per_row;
        rest = uint32_t(first - row0 * per_row);
    }
    __device__ Position at(uint32_t offset) const
    {
        const uint32_t t = rest + offset;
        const uint32_t r = t / per_row;
        return Position{row0 + r, int(t - r * per_row) * 8};
    }
};

// Groups of 8 of the whole matrix, workgroup by workgroup: first the loads of
// all of a thread's groups (In load(row, col)), then f(row, col, in) of each, so
// that no store holds up a load.  Whole blocks of 4 lanes run or not together.
template <int N, class In, class Load, class F>
__device__ inline void for_octets(int64_t rows, int64_t pitch, Load load, F f)
{
    const uint32_t per_row = uint32_t(pitch >> 3);
    const int64_t total = rows * per_row;
    for (int64_t first = int64_t(blockIdx.x) * (kBlock * N); first < total;
         first += int64_t(gridDim.x) * (kBlock * N)) {
        const Walk walk(first, per_row);
        In in[N];
        Position at[N];
#pragma unroll
        for (int o = 0; o < N; ++o) {
            const uint32_t offset = o * kBlock + threadIdx.x;
            if (first + offset < total) {
                at[o] = walk.at(offset);
                in[o] = load(at[o].row, at[o].col);
            }
        }
#pragma unroll
        for (int o = 0; o < N; ++o)
            if (first + o * kBlock + threadIdx.x < total) f(at[o].row, at[o].col, in[o]);
    }
}

template <class T>
struct Values {
    float v[8];
    __device__ Values() {}
    __device__ Values(const T *line, int col, int cols) { load8(line, col, cols, v); }
};

inline bool float_type(adam_dtype t) { return t == ADAM_DT_F32 || t == ADAM_DT_BF16 || t == ADAM_DT_F16; }

inline bool known_type(int t) { return t >= ADAM_DT_NONE && t <= ADAM_DT_F16; }

inline dim3 octet_grid(int64_t rows, int64_t pitch, int octets)
{
    const int64_t blocks = (rows * (pitch / 8) + kBlock * octets - 1) / (kBlock * octets);
    return dim3(uint32_t(std::min(blocks, kMaxGrid)));
}

// Calls f with a value of the type (as a template argument would be).
template <class F>
int with_type(adam_dtype t, F f)
{
    if (t == ADAM_DT_F32) return f(float());
    if (t == ADAM_DT_BF16) return f(bf16());
    return f(f16());
}

}  // namespace train

#endif
