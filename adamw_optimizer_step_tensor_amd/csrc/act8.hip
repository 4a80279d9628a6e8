// Activation checkpoints in 8 bits and the backward steps that read them
// (include/adam_train.h states the format and the formulas).
//
// The streaming kernels (store, load, gated activation forward and backward)
// take 8 elements a lane, so 4 neighbouring lanes hold one scale block and
// agree on its largest magnitude with two lane exchanges.  They are bound by
// HBM: one pass, every input read once, every output written once, both without
// a stay in the caches (nothing reads a line again before the caches have turned
// over: 115 us instead of 131 for store and load, 359 instead of 389 for the
// gated activation).
#include <hip/hip_runtime.h>

#include "octets.h"

namespace train {
namespace {

// Groups of 8 elements per thread: two in flight for one matrix, one where a
// group already loads two or three (store and load together 115 us with two,
// 130 with one or four, at 8192 x 14336 bf16; the gated activation's passes 345
// us with one, 359 with two).
constexpr int kOctets = 2, kGluOctets = 1;

struct Checkpoint {
    uint8_t *codes, *scales;
    int64_t pitch;
};

template <int CTRL>
__device__ inline uint32_t lane_exchange(uint32_t v)
{
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 15, 15, true));
}

// The largest over the 4 lanes of a scale block.
__device__ inline uint32_t over_block(uint32_t v)
{
    uint32_t o = lane_exchange<0xB1>(v);  // lanes 1, 0, 3, 2
    v = o > v ? o : v;
    o = lane_exchange<0x4E>(v);  // lanes 2, 3, 0, 1
    return o > v ? o : v;
}

// The block's scale byte and the 8 codes of this lane.  The 4 lanes of a block
// are neighbours and all active (a row's pitch is a multiple of 32).
template <int FMT>
__device__ inline void encode8(const float (&v)[8], uint32_t &byte, uint64_t &codes)
{
    constexpr int kExp = FMT == kE4M3 ? 8 : 15;  // MAX = 1.75 * 2^kExp
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
        amax = b > amax ? b : amax;
    }
    amax = over_block(amax);
    const bool special = amax >= 0x7f800000u;  // a block with an infinity or NaN: the largest of the others
    if (special) {
        amax = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
            if (b < 0x7f800000u && b > amax) amax = b;
        }
        amax = over_block(amax);
    }
    // amax = 1.f * 2^k: the smallest e with amax <= 1.75 * 2^(kExp + e) is
    // k - kExp, and one more where 1.f > 1.75 (f has its top two bits set and
    // another); a subnormal amax ends below -127 and is clamped
    const int e = int(amax >> 23) - kExp + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    byte = e > 0 ? uint32_t(e) : 0u;
    // the conversion divides by the power of two that the scale's exponent
    // field says (2^-127 for 0), then rounds once
    const float scale = __uint_as_float(byte << 23);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        vec<short, 2> r = {0, 0};
        if (FMT == kE4M3) {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h], v[4 * h + 1], scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h + 2], v[4 * h + 3], scale, true);
        } else {
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, v[4 * h], v[4 * h + 1], scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, v[4 * h + 2], v[4 * h + 3], scale, true);
        }
        w[h] = __builtin_bit_cast(uint32_t, r);
    }
    codes = uint64_t(w[1]) << 32 | w[0];
    if (special) {
        // the conversion's own treatment of these depends on a mode bit
#pragma unroll
        for (int e2 = 0; e2 < 8; ++e2) {
            const uint32_t b = __float_as_uint(v[e2]);
            const uint32_t m = b & 0x7fffffffu;
            if (m >= 0x7f800000u) {
                const uint64_t code = FMT == kE4M3 || m > 0x7f800000u ? 0x7f : 0x7c | (b >> 31 << 7);
                codes = (codes & ~(uint64_t(0xff) << (8 * e2))) | code << (8 * e2);
            }
        }
    }
}

template <int FMT>
__device__ inline void write8(const float (&v)[8], const Checkpoint &c, int64_t row, int col)
{
    uint32_t byte;
    uint64_t codes;
    encode8<FMT>(v, byte, codes);
    __builtin_nontemporal_store(codes, (uint64_t *)(c.codes + row * c.pitch + col));
    if ((col & 31) == 0) c.scales[row * (c.pitch >> 5) + (col >> 5)] = uint8_t(byte);
}

struct Codes {
    uint64_t codes;
    uint32_t byte;
};

__device__ inline Codes read_codes(const Checkpoint &c, int64_t row, int col)
{
    return Codes{*(const uint64_t *)(c.codes + row * c.pitch + col), c.scales[row * (c.pitch >> 5) + (col >> 5)]};
}

template <int FMT>
__device__ inline void decode8(const Codes &c, float (&v)[8])
{
    // the conversion multiplies by the power of two of the scale's exponent field
    const float scale = __uint_as_float(c.byte << 23);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w = uint32_t(c.codes >> (32 * h));
        vec<float, 2> lo, hi;
        if (FMT == kE4M3) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, true);
        }
        v[4 * h] = lo[0];
        v[4 * h + 1] = lo[1];
        v[4 * h + 2] = hi[0];
        v[4 * h + 3] = hi[1];
    }
}

template <class T, int FMT>
__global__ __launch_bounds__(kBlock) void act8_store_kernel(const T *x, int64_t rows, int cols, int64_t stride,
                                                            Checkpoint c)
{
    for_octets<kOctets, Values<T>>(
        rows, c.pitch, [&](int64_t row, int col) { return Values<T>(x + row * stride, col, cols); },
        [&](int64_t row, int col, const Values<T> &in) { write8<FMT>(in.v, c, row, col); });
}

template <class T, int FMT>
__global__ __launch_bounds__(kBlock) void act8_load_kernel(Checkpoint c, int64_t rows, int cols, T *x, int64_t stride)
{
    for_octets<kOctets, Codes>(
        rows, c.pitch, [&](int64_t row, int col) { return read_codes(c, row, col); },
        [&](int64_t row, int col, const Codes &in) {
            float v[8];
            decode8<FMT>(in, v);
            store8(x + row * stride, col, cols, v);
        });
}

// a(x) = x s(q(x)) with s the logistic function: q = x for silu; for gelu
// 1/2 (1 + tanh y) = s(2 y), so q = 2 sqrt(2/pi) (x + 0.044715 x^3), which
// keeps its relative accuracy where 1 + tanh cancels.
// a'(x) = s + x s (1 - s) q'(x).
template <int ACT, bool DERIVATIVE, bool EXACT>
__device__ inline float gate(float x, float &derivative)
{
    constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2/pi)
    float q = x, dq = 1.0f;
    if (ACT == ADAM_ACT_GELU) {
        const float x2 = x * x;
        q = kTwoC * fmaf(0.044715f * x2, x, x);
        dq = kTwoC * fmaf(3 * 0.044715f, x2, 1.0f);
    }
    // exp(-q) = 2^t (1 + r ln 2): t the rounded product, r what it lost.  For
    // float results r is put back, so that the error stays near one unit for
    // large |q| too; 2^-17 |q| / 88 of it is nothing to a 16-bit one.
    constexpr float kLog2e = 1.4426950408889634f, kLow = 1.925963033500926e-08f;
    const float t = -q * kLog2e;
    float e = __builtin_amdgcn_exp2f(t);
    if (EXACT) {
        const float r = fmaf(-q, kLog2e, -t) - q * kLow;
        e = fabsf(t) < 128.0f ? fmaf(e, r * 0.6931471805599453f, e) : e;
    }
    // 1 / (1 + e), by quarters: the reciprocal instruction makes 0 of a result
    // below the normal range, which 1 + e reaches at 2^126
    const float s = __builtin_amdgcn_rcpf(fmaf(e, 0.25f, 0.25f)) * 0.25f;
    if (DERIVATIVE) {
        const float w = e * s * s;  // s (1 - s)
        // not 0 times inf, where e or dq is infinite; s may be 1 while this term
        // is still several units of it
        derivative = s + (w > 0.0f ? x * w * dq : 0.0f);
    }
    return x * s;
}

template <class T>
constexpr bool kExact = std::is_same<T, float>::value;

template <class T, int FMT, int ACT, bool CKPT>
__global__ __launch_bounds__(kBlock) void glu_forward_kernel(const T *g, const T *u, int64_t rows, int cols,
                                                             int64_t in_stride, T *h, int64_t h_stride, Checkpoint cg,
                                                             Checkpoint cu)
{
    struct In {
        Values<T> g, u;
    };
    for_octets<kGluOctets, In>(
        rows, cg.pitch,
        [&](int64_t row, int col) {
            return In{Values<T>(g + row * in_stride, col, cols), Values<T>(u + row * in_stride, col, cols)};
        },
        [&](int64_t row, int col, const In &in) {
            float y[8], unused;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = gate<ACT, false, kExact<T>>(in.g.v[e], unused) * in.u.v[e];
            store8(h + row * h_stride, col, cols, y);
            if (CKPT) {
                write8<FMT>(in.g.v, cg, row, col);
                write8<FMT>(in.u.v, cu, row, col);
            }
        });
}

template <class T, int FMT, int ACT>
__global__ __launch_bounds__(kBlock) void glu_backward_kernel(const T *dh, int64_t rows, int cols, int64_t dh_stride,
                                                              Checkpoint cg, Checkpoint cu, T *dg, T *du,
                                                              int64_t d_stride, T *h, int64_t h_stride, Checkpoint ch)
{
    struct In {
        Values<T> d;
        Codes g, u;
    };
    for_octets<kGluOctets, In>(
        rows, cg.pitch,
        [&](int64_t row, int col) {
            return In{Values<T>(dh + row * dh_stride, col, cols), read_codes(cg, row, col), read_codes(cu, row, col)};
        },
        [&](int64_t row, int col, const In &in) {
            float a[8], b[8], x[8], y[8], z[8];
            decode8<FMT>(in.g, a);
            decode8<FMT>(in.u, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float da;
                const float f = gate<ACT, true, kExact<T>>(a[e], da);
                x[e] = in.d.v[e] * b[e] * da;
                y[e] = in.d.v[e] * f;
                z[e] = f * b[e];
            }
            store8(dg + row * d_stride, col, cols, x);
            store8(du + row * d_stride, col, cols, y);
            if (h != nullptr) store8(h + row * h_stride, col, cols, z);
            if (ch.codes != nullptr) write8<FMT>(z, ch, row, col);
        });
}

// One row of the copy a workgroup.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t *from, int64_t stride, int64_t rows, int cols,
                                                   uint16_t *to, int64_t pitch)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) copy_row(from + r * stride, cols, to + r * pitch, pitch);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct CheckpointShape {
    int64_t pitch, scales_at, bytes;
};

// Sizes of a checkpoint; false where rows or cols are out of range or the
// byte count would not fit 63 bits.
bool shape_of(int64_t rows, int64_t cols, CheckpointShape &s)
{
    if (rows < 0 || rows > kMaxSize || cols < 0 || cols > kMaxSize) return false;
    s.pitch = round_up(cols, 32);
    s.scales_at = round_up(rows * s.pitch, 256);
    s.bytes = s.scales_at + rows * (s.pitch / 32);
    return true;
}

Checkpoint checkpoint(const void *p, const CheckpointShape &s)
{
    return Checkpoint{(uint8_t *)p, p == nullptr ? nullptr : (uint8_t *)p + s.scales_at, s.pitch};
}

bool valid_format(adam_act8_format f) { return f == ADAM_ACT8_E4M3 || f == ADAM_ACT8_E5M2; }

template <int V>
using constant = std::integral_constant<int, V>;

template <class F>
int with_format(adam_act8_format format, F f)
{
    return format == ADAM_ACT8_E4M3 ? f(constant<kE4M3>()) : f(constant<kE5M2>());
}

template <class F>
int with_act(adam_act act, F f)
{
    return act == ADAM_ACT_SILU ? f(constant<ADAM_ACT_SILU>()) : f(constant<ADAM_ACT_GELU>());
}

// Sizes that the core's 32-bit offsets and counts allow a weight gradient.
bool wgrad_sizes(int64_t rows, int64_t n, int64_t k)
{
    return rows >= 0 && rows <= kMaxProductRows && n >= 0 && n <= kMaxDirectStride && k >= 0 &&
           k <= kMaxDirectStride && !too_many_tiles(n, k);
}

// The weight gradient is one product of the matrix core, x = the checkpoint and
// y = dy, both with the tokens as k: 0.75 ms at 8192 x 4096 x 14336 (1.29
// PFLOP/s; 0.73 once the card's clock has settled, up to 0.99 in the first dozen
// calls after a pause), 75 us at 8192 x 1024 x 4096 (64 tiles in four parts each:
// 0.92 PFLOP/s).  The decoded tile's LDS writes conflict two ways (20% of the LDS's
// cycles), which is not what bounds it: the LDS works 39% of the time, and
// exchanging the halves of every other lane to avoid them took 4 to 6% longer.
struct WgradPlan {
    Product product;
    uint16_t *packed;  // dy, where it cannot be read where it lies
    float *part;
    int64_t bytes;

    WgradPlan(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t dy_stride, void *workspace)
        : product(k, n, rows)
    {
        Workspace w{(char *)workspace};
        packed = direct(dy, dy_stride, n, false) ? nullptr : w.take<uint16_t>(rows * round_up(n, 8));
        is_packed = !direct(dy, dy_stride, n, false);
        part = w.take<float>(product.part_floats());
        bytes = w.used;
    }
    bool is_packed;
};

}  // namespace

int pack(const void *from, int64_t stride, int64_t rows, int64_t cols, void *to, int64_t pitch, hipStream_t stream)
{
    if (rows <= 0) return ADAM_OK;
    hipLaunchKernelGGL(pack_kernel, dim3(uint32_t(std::min<int64_t>(rows, 1 << 20))), dim3(256), 0, stream,
                       (const uint16_t *)from, stride, rows, int(cols), (uint16_t *)to, pitch);
    return launched();
}

}  // namespace train

using namespace train;

extern "C" {

int adam_act8_bytes(int64_t rows, int64_t cols, int64_t *bytes)
{
    CheckpointShape s;
    if (bytes == nullptr || !shape_of(rows, cols, s)) return ADAM_EINVAL;
    *bytes = s.bytes;
    return ADAM_OK;
}

int adam_act8_store(const void *x, adam_dtype x_type, int64_t rows, int64_t cols, int64_t x_stride,
                    adam_act8_format format, void *ckpt, hipStream_t stream)
{
    CheckpointShape s;
    if (!known_type(x_type) || !valid_format(format)) return ADAM_EINVAL;
    if (!float_type(x_type)) return ADAM_EDTYPE;
    if (!shape_of(rows, cols, s) || !valid_matrix(rows, cols, x_stride)) return ADAM_EINVAL;
    if (s.bytes == 0) return ADAM_OK;
    const int b = dtype_bytes(x_type);
    if (x == nullptr || ckpt == nullptr || !aligned(x, b) || !aligned(ckpt, 16)) return ADAM_EINVAL;
    if (overlap(matrix(x, rows, cols, x_stride, b), flat(ckpt, s.bytes))) return ADAM_EINVAL;
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return with_type(x_type, [&](auto t) {
        return with_format(format, [&](auto f) {
            using T = decltype(t);
            hipLaunchKernelGGL((act8_store_kernel<T, decltype(f)::value>), octet_grid(rows, s.pitch, kOctets), dim3(kBlock), 0,
                               stream, (const T *)x, rows, int(cols), x_stride, checkpoint(ckpt, s));
            return launched();
        });
    });
}

int adam_act8_load(const void *ckpt, adam_act8_format format, int64_t rows, int64_t cols, void *x,
                   adam_dtype x_type, int64_t x_stride, hipStream_t stream)
{
    CheckpointShape s;
    if (!known_type(x_type) || !valid_format(format)) return ADAM_EINVAL;
    if (!float_type(x_type)) return ADAM_EDTYPE;
    if (!shape_of(rows, cols, s) || !valid_matrix(rows, cols, x_stride)) return ADAM_EINVAL;
    if (s.bytes == 0) return ADAM_OK;
    const int b = dtype_bytes(x_type);
    if (x == nullptr || ckpt == nullptr || !aligned(x, b) || !aligned(ckpt, 16)) return ADAM_EINVAL;
    if (overlap(matrix(x, rows, cols, x_stride, b), flat(ckpt, s.bytes))) return ADAM_EINVAL;
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return with_type(x_type, [&](auto t) {
        return with_format(format, [&](auto f) {
            using T = decltype(t);
            hipLaunchKernelGGL((act8_load_kernel<T, decltype(f)::value>), octet_grid(rows, s.pitch, kOctets), dim3(kBlock), 0,
                               stream, checkpoint(ckpt, s), rows, int(cols), (T *)x, x_stride);
            return launched();
        });
    });
}

int adam_glu_forward(const void *gate, const void *up, adam_dtype type, int64_t rows, int64_t cols,
                     int64_t in_stride, adam_act act, void *h, int64_t h_stride, adam_act8_format format,
                     void *ckpt_gate, void *ckpt_up, hipStream_t stream)
{
    CheckpointShape s;
    if (!known_type(type) || !valid_format(format) || (act != ADAM_ACT_SILU && act != ADAM_ACT_GELU))
        return ADAM_EINVAL;
    if (!float_type(type)) return ADAM_EDTYPE;
    if (!shape_of(rows, cols, s) || !valid_matrix(rows, cols, in_stride) || !valid_matrix(rows, cols, h_stride))
        return ADAM_EINVAL;
    if ((ckpt_gate == nullptr) != (ckpt_up == nullptr)) return ADAM_EINVAL;
    if (s.bytes == 0) return ADAM_OK;
    const int b = dtype_bytes(type);
    if (gate == nullptr || up == nullptr || h == nullptr || !aligned(gate, b) || !aligned(up, b) || !aligned(h, b) ||
        !aligned(ckpt_gate, 16) || !aligned(ckpt_up, 16))
        return ADAM_EINVAL;
    const View in[2] = {matrix(gate, rows, cols, in_stride, b), matrix(up, rows, cols, in_stride, b)};
    const View out[3] = {matrix(h, rows, cols, h_stride, b), flat(ckpt_gate, s.bytes), flat(ckpt_up, s.bytes)};
    for (int i = 0; i < 3; ++i) {
        for (const View &v : in)
            if (overlap(out[i], v)) return ADAM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return ADAM_EINVAL;
    }
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return with_type(type, [&](auto t) {
        return with_format(format, [&](auto f) {
            return with_act(act, [&](auto a) {
                using T = decltype(t);
                constexpr int F = decltype(f)::value, A = decltype(a)::value;
                const auto kernel = ckpt_gate != nullptr ? glu_forward_kernel<T, F, A, true>
                                                         : glu_forward_kernel<T, F, A, false>;
                hipLaunchKernelGGL(kernel, octet_grid(rows, s.pitch, kGluOctets), dim3(kBlock), 0, stream, (const T *)gate,
                                   (const T *)up, rows, int(cols), in_stride, (T *)h, h_stride,
                                   checkpoint(ckpt_gate, s), checkpoint(ckpt_up, s));
                return launched();
            });
        });
    });
}

int adam_glu_backward(const void *dh, adam_dtype type, int64_t rows, int64_t cols, int64_t dh_stride,
                      adam_act act, adam_act8_format format, const void *ckpt_gate, const void *ckpt_up,
                      void *dgate, void *dup, int64_t d_stride, void *h, int64_t h_stride, void *ckpt_h,
                      hipStream_t stream)
{
    CheckpointShape s;
    if (!known_type(type) || !valid_format(format) || (act != ADAM_ACT_SILU && act != ADAM_ACT_GELU))
        return ADAM_EINVAL;
    if (!float_type(type)) return ADAM_EDTYPE;
    if (!shape_of(rows, cols, s) || !valid_matrix(rows, cols, dh_stride) || !valid_matrix(rows, cols, d_stride) ||
        (h != nullptr && !valid_matrix(rows, cols, h_stride)))
        return ADAM_EINVAL;
    if (s.bytes == 0) return ADAM_OK;
    const int b = dtype_bytes(type);
    if (dh == nullptr || ckpt_gate == nullptr || ckpt_up == nullptr || dgate == nullptr || dup == nullptr ||
        !aligned(dh, b) || !aligned(dgate, b) || !aligned(dup, b) || !aligned(h, b) || !aligned(ckpt_gate, 16) ||
        !aligned(ckpt_up, 16) || !aligned(ckpt_h, 16))
        return ADAM_EINVAL;
    const View in[3] = {matrix(dh, rows, cols, dh_stride, b), flat(ckpt_gate, s.bytes), flat(ckpt_up, s.bytes)};
    const View out[4] = {matrix(dgate, rows, cols, d_stride, b), matrix(dup, rows, cols, d_stride, b),
                         matrix(h, rows, cols, h_stride, b), flat(ckpt_h, s.bytes)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j) {
            const bool in_place = i < 2 && j == 0 && out[i].p == dh && (d_stride == dh_stride || rows == 1);
            if (!in_place && overlap(out[i], in[j])) return ADAM_EINVAL;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return ADAM_EINVAL;
    }
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return with_type(type, [&](auto t) {
        return with_format(format, [&](auto f) {
            return with_act(act, [&](auto a) {
                using T = decltype(t);
                hipLaunchKernelGGL((glu_backward_kernel<T, decltype(f)::value, decltype(a)::value>),
                                   octet_grid(rows, s.pitch, kGluOctets), dim3(kBlock), 0, stream, (const T *)dh, rows, int(cols),
                                   dh_stride, checkpoint(ckpt_gate, s), checkpoint(ckpt_up, s), (T *)dgate, (T *)dup,
                                   d_stride, (T *)h, h_stride, checkpoint(ckpt_h, s));
                return launched();
            });
        });
    });
}

int adam_act8_wgrad_workspace(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t dy_stride,
                              int64_t *bytes)
{
    if (bytes == nullptr || !wgrad_sizes(rows, n, k) || !valid_matrix(rows, n, dy_stride)) return ADAM_EINVAL;
    *bytes = n == 0 || k == 0 ? 0 : WgradPlan(rows, n, k, dy, dy_stride, nullptr).bytes;
    return ADAM_OK;
}

int adam_act8_wgrad(const void *dy, adam_dtype dy_type, int64_t dy_stride, const void *ckpt,
                    adam_act8_format format, int64_t rows, int64_t n, int64_t k, void *dw, adam_dtype dw_type,
                    int64_t dw_stride, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                    hipStream_t stream)
{
    CheckpointShape s;
    if (!known_type(dy_type) || !known_type(dw_type) || !valid_format(format) || (accumulate != 0 && accumulate != 1))
        return ADAM_EINVAL;
    if (!is_half(dy_type) || (dw_type != ADAM_DT_F32 && dw_type != dy_type)) return ADAM_EDTYPE;
    if (!wgrad_sizes(rows, n, k) || !shape_of(rows, k, s) || !valid_matrix(rows, n, dy_stride) ||
        !valid_matrix(n, k, dw_stride))
        return ADAM_EINVAL;
    if (n == 0 || k == 0) return ADAM_OK;
    const int ob = dtype_bytes(dw_type);
    if (dw == nullptr || !aligned(dw, ob) ||
        (rows > 0 && (dy == nullptr || ckpt == nullptr || !aligned(dy, 2) || !aligned(ckpt, 16))))
        return ADAM_EINVAL;
    const WgradPlan plan(rows, n, k, dy, dy_stride, workspace);
    if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes || !aligned(workspace, 256)))
        return ADAM_EINVAL;
    const View in[2] = {rows > 0 ? matrix(dy, rows, n, dy_stride, 2) : View{}, flat(ckpt, rows > 0 ? s.bytes : 0)};
    const View out[2] = {matrix(dw, n, k, dw_stride, ob), flat(workspace, plan.bytes)};
    for (const View &o : out)
        for (const View &i : in)
            if (overlap(o, i)) return ADAM_EINVAL;
    if (overlap(out[0], out[1])) return ADAM_EINVAL;
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    if (plan.is_packed) {
        const int rc = pack(dy, dy_stride, rows, n, plan.packed, round_up(n, 8), stream);
        if (rc != ADAM_OK) return rc;
        dy = plan.packed;
        dy_stride = round_up(n, 8);
    }
    GemmArgs a = {};
    a.x = Operand{ckpt, (const uint8_t *)ckpt + s.scales_at, s.pitch, int32_t(k), int32_t(rows)};
    a.y = Operand{dy, nullptr, dy_stride, int32_t(n), int32_t(rows)};
    return with_format(format, [&](auto f) {
        constexpr int F = decltype(f)::value;
        auto run = [&](auto t, auto o) {
            using T = decltype(t);
            using O = decltype(o);
            StoreEpilogue<O> e = {};
            e.out = (O *)dw;
            e.stride = dw_stride;
            e.factor = float(1 << Half<T>::kHalvings);
            e.accumulate = accumulate;
            return run_product<T, F, kCols>(plan.product, a, e, plan.part, stream);
        };
        if (dy_type == ADAM_DT_BF16) return dw_type == ADAM_DT_F32 ? run(bf16(), float()) : run(bf16(), bf16());
        return dw_type == ADAM_DT_F32 ? run(f16(), float()) : run(f16(), f16());
    });
}

}  // extern "C"
