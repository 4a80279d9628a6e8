// Softmax cross entropy over a large vocabulary, with its gradient
// (include/adam_train.h states the formulas).
//
// Per piece of rows (those whose target is not ignore_index, gathered):
//   1. z = h W^T in 256 x 256 tiles of (vocabulary x rows), whose epilogue
//      reduces each row's 128 logits of a wave (a part of the vocabulary) to
//      their maximum m and the sum of exp(z - m), keeps the target's logit in
//      float, and (for the gradient) stores E = exp(z - m) times a power of two
//      in 16 bits; the logits themselves are never stored.
//   2. lse and loss per row from the sums of all parts.
//   3. G = weight (E exp(m - lse) - [v = target]), in place of E, in h's
//      type: the rounding that the matrix instruction asks of its operands.
//      The target's entry comes from its float logit, as expm1(z - lse).
//   4. dh = G W and dW = G^T h, float sums.
// 6 rows x vocab x hidden operations in all.  Computing the logits a second
// time instead of storing E would make them 8; E costs 4 bytes of traffic each
// way per logit, 4% of the whole at hidden 4096.
//
// At 8192 rows (7373 of them not ignored) x 131072 x 4096 in bf16: logits 6.3 ms
// (1.26 PFLOP/s, of which the epilogue's exponentials take about 0.3), G 0.67
// (3.9 GB at 5.8 TB/s), dh 5.8 (1.36 PFLOP/s), dw 5.4 (1.46 PFLOP/s); 18.5 ms in
// all.  The products are bound by the matrix units at the clock that the card's
// power leaves (1.7-1.8 GHz).
#include <hip/hip_runtime.h>

#include "train.h"

namespace train {
namespace {

using u16x4 = vec<uint16_t, 4>;

constexpr int kPart = 128;  // logits that a wave reduces per row
constexpr float kLog2e = 1.4426950408889634f;

// Exponentials are taken to base 2, of t = z * kLog2e with the product unrounded
// (fma).  With m a part's largest logit and r = shift - kLog2e m, rounded, its
// E = 2^(t + r) are exp(z - m) 2^b, where b is the shift and what r's rounding
// adds to it: at most 2^-4 while |m| is below 2^20, so that E fits its 16 bits
// (they hold b + 1).  Beyond, or where m is no number, t is taken of z - m, at
// one more operation a logit, and b is the shift.  What is kept of a part, m and
// the sum l of its E before rounding, stands for a sum of exp(z - m) of l 2^-b.
constexpr float kLarge = 0x1p20f;

__device__ inline bool is_large(float m) { return !(fabsf(m) < kLarge); }
__device__ inline float reference(float m, float shift) { return fmaf(-m, kLog2e, shift); }

// b; exact, since the product of two floats is exact in double.
__device__ inline double unit_exponent(float m, float shift)
{
    return is_large(m) ? double(shift) : double(reference(m, shift)) + double(m) * kLog2e;
}

// The exponent of exp(m - top): the difference is taken first, so that it does
// not cancel however large both are.  Two that are equal may be infinite.
__device__ inline double exponent_below(float m, float top)
{
    return m == top ? 0.0 : (double(m) - double(top)) * kLog2e;
}

// How E is kept in 16 bits.  G is rounded to T once more, so E should be a few
// bits finer than T.
template <class T>
struct Kept;

// For bf16 (8 bits): fp16 with E about 2^15 at most: 11 bits down to 2^-29 of the part's
// largest.
template <>
struct Kept<bf16> {
    static constexpr float kShift = 15.0f;
    static __device__ vec<uint16_t, 4> pack(const float *e)
    {
        return __builtin_bit_cast(u16x4, f16x4{f16(e[0]), f16(e[1]), f16(e[2]), f16(e[3])});
    }
    static __device__ float unpack(uint16_t k) { return float(__builtin_bit_cast(f16, k)); }
};

// For fp16 (11 bits): 5 bits of exponent and 11 of mantissa, no sign, E about 1 at most:
// 12 bits down to 2^-30 of the part's largest.  As fp16, E would cost as much as
// G's rounding does: with both alike a gradient without a sharp top is off by
// sqrt(3) times the error of its own rounding, with this by sqrt(2.25) at most.
// The bits are those of the float E 2^-96 (its exponent field is 31 for E = 1,
// and values below 2^-30 are subnormal), rounded to 11 bits of mantissa.
template <>
struct Kept<f16> {
    static constexpr float kShift = 0.0f;
    static __device__ vec<uint16_t, 4> pack(const float *e)
    {
        u16x4 k;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = __float_as_uint(e[i] * 0x1p-96f);
            k[i] = uint16_t((u + 0x7ffu + ((u >> 12) & 1u)) >> 12);
        }
        return k;
    }
    static __device__ float unpack(uint16_t k) { return __uint_as_float(uint32_t(k) << 12) * 0x1p96f; }
};

// G is multiplied by a power of two before its rounding (and the sums by its
// inverse).  bf16 has the range of float: 1.  fp16 would keep small probabilities
// as subnormals only: 2^14 without weights, so that G is at most 2^14 and
// probabilities down to 2^-28 keep all bits; with weights what brings the
// largest magnitude among the computed rows' to 2^14 or more, below 2^15.
template <class T>
constexpr float kUnit = std::is_same<T, f16>::value ? 0x1p14f : 1.0f;

// The unit that the gathering kernels choose from the bits of the largest finite
// |weight|, and what it makes of the loss scale.
struct Unit {
    float unit, scale;

    __device__ void set(uint32_t most, const float *loss_scale)
    {
        const int e = int(most >> 23) - 127;        // -127 for a subnormal or zero
        const int k = 14 - e < 126 ? 14 - e : 126;  // 2^-126 is the least that is no subnormal
        unit = __uint_as_float(uint32_t(127 + k) << 23);
        scale = __uint_as_float(uint32_t(127 - k) << 23) * (loss_scale != nullptr ? *loss_scale : 1.0f);
    }
};

// What a row's weight adds to `most`.
__device__ inline void note_weight(uint32_t &most, float weight)
{
    const uint32_t b = __float_as_uint(weight) & 0x7fffffffu;
    if (b < 0x7f800000u && b > most) most = b;
}

// Up to this many rows, each is gathered twice and its G kept as a sum of two
// 16-bit values, in one row the rounded G, in the next what the rounding lost:
// with few rows the roundings do not average out (dw of two rows in bf16 was off
// by 1.8 times the error of its own rounding), and the tiles of 256 rows have
// room for both.
constexpr int64_t kTwiceRows = 128;

// What the later kernels need of a gathered row.
struct RowState {
    double log2_sum;  // of the sum of exp(z - top)
    float top;        // the largest logit
    float weight;     // NaN for a bad target, or a logit of +inf or NaN
    int32_t target;   // -1 for a bad one
    float own;        // G of the target
};

struct Rows {
    const int32_t *index;   // gathered row -> row
    const int32_t *target;  // of the gathered row; -1 for one outside the vocabulary
    const int32_t *count;   // gathered rows
    int32_t first, most;    // this piece
    int32_t copies;         // 2: every row is gathered twice

    __device__ int here() const
    {
        const int n = *count - first;
        return n < 0 ? 0 : n > most ? most : n;
    }
};

// Numbers the rows that are computed; the others' loss and lse are 0.
__global__ __launch_bounds__(1024) void xent_gather(const int64_t *target, int64_t ignore, int rows, int64_t vocab,
                                                    int32_t *index, int32_t *targets, int32_t *places, int32_t *count,
                                                    float *loss, float *lse, const float *weight,
                                                    const float *loss_scale, Unit *unit)
{
    __shared__ int32_t waves[16];
    __shared__ uint32_t wave_most[16];
    uint32_t most = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0;
    for (int first = 0; first < rows; first += 1024) {
        const int r = first + threadIdx.x;
        const bool in = r < rows;
        const int64_t t = in ? target[r] : ignore;
        const bool keep = t != ignore;
        const uint64_t mask = __ballot(keep);
        if (lane == 0) waves[wave] = __popcll(mask);
        __syncthreads();
        int before = base, total = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int n = waves[w];
            before += w < wave ? n : 0;
            total += n;
        }
        if (keep) {
            const int at = before + __popcll(mask & ((uint64_t(1) << lane) - 1));
            places[r] = at;
            index[at] = r;
            targets[at] = t >= 0 && t < vocab ? int32_t(t) : -1;
            if (unit != nullptr) note_weight(most, weight[r]);
        }
        if (in && !keep) {
            places[r] = -1;
            loss[r] = 0.0f;
            if (lse != nullptr) lse[r] = 0.0f;
        }
        base += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) *count = base;
    if (unit == nullptr) return;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = max(most, uint32_t(__shfl_xor(int(most), d)));
    if (lane == 0) wave_most[wave] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) most = max(most, wave_most[w]);
        unit->set(most, loss_scale);
    }
}

// The hidden states of a piece's gathered rows, one after the other in rows of
// `pitch`, and (zero_dh, in the first piece) zeros in the rows of dh that are
// not computed.  One row a workgroup.
__global__ __launch_bounds__(256) void xent_rows(const int32_t *places, int rows, int first, int most,
                                                 const uint16_t *h, int64_t h_stride, int hidden, uint16_t *to,
                                                 int64_t pitch, uint16_t *zero_dh, int64_t dh_stride)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int at = places[r];
        if (at < 0) {
            if (zero_dh != nullptr)
                for (int c = threadIdx.x; c < hidden; c += 256) zero_dh[r * dh_stride + c] = 0;
        } else if (at >= first && at - first < most) {
            copy_row(h + r * h_stride, hidden, to + (at - first) * pitch, pitch);
        }
    }
}

// xent_gather and xent_rows in one, for up to kDirectRows rows in one piece: each
// workgroup counts the computed rows before its own, so the targets are read
// rows times; the first one takes the largest weight.  200 rows x 1024 x 4000:
// 78.2 us, 80.3 with two kernels; 1020 x 512 x 600: 70.0 and 71.8; the losses of
// 64 x 512 x 2000: 23.0 and 24.7.
constexpr int kDirectRows = 1024;

__global__ __launch_bounds__(256) void xent_gather_rows(const int64_t *target, int64_t ignore, int rows,
                                                        int64_t vocab, int copies, int32_t *index, int32_t *targets,
                                                        int32_t *count, float *loss, float *lse, const uint16_t *h,
                                                        int64_t h_stride, int hidden, uint16_t *to, int64_t pitch,
                                                        uint16_t *zero_dh, int64_t dh_stride, const float *weight,
                                                        const float *loss_scale, Unit *unit)
{
    __shared__ int waves[8];
    __shared__ uint32_t wave_most[4];
    const int r = blockIdx.x;
    const bool weigh = unit != nullptr && r == 0;
    int before = 0, total = 0;
    uint32_t most = 0;
    for (int i = threadIdx.x; i < rows; i += 256) {
        const int kept = target[i] != ignore;
        total += kept;
        before += i < r ? kept : 0;
        if (weigh && kept) note_weight(most, weight[i]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        total += __shfl_xor(total, d);
        before += __shfl_xor(before, d);
        if (weigh) most = max(most, uint32_t(__shfl_xor(int(most), d)));
    }
    if ((threadIdx.x & 63) == 0) {
        waves[threadIdx.x >> 6] = total;
        waves[4 + (threadIdx.x >> 6)] = before;
        wave_most[threadIdx.x >> 6] = most;
    }
    __syncthreads();
    if (weigh && threadIdx.x == 0)
        unit->set(max(max(wave_most[0], wave_most[1]), max(wave_most[2], wave_most[3])), loss_scale);
    total = waves[0] + waves[1] + waves[2] + waves[3];
    const int at = (waves[4] + waves[5] + waves[6] + waves[7]) * copies;
    if (r == 0 && threadIdx.x == 0) *count = total * copies;
    const int64_t t = target[r];
    if (t == ignore) {
        if (threadIdx.x == 0) {
            loss[r] = 0.0f;
            if (lse != nullptr) lse[r] = 0.0f;
        }
        if (zero_dh != nullptr)
            for (int c = threadIdx.x; c < hidden; c += 256) zero_dh[r * dh_stride + c] = 0;
        return;
    }
    if (threadIdx.x < copies) {
        index[at + threadIdx.x] = r;
        targets[at + threadIdx.x] = t >= 0 && t < vocab ? int32_t(t) : -1;
    }
    for (int c = 0; c < copies; ++c) copy_row(h + r * h_stride, hidden, to + int64_t(at + c) * pitch, pitch);
}

// A part's largest logit as it is kept.  Where it is +inf or NaN the part's sum
// says so.
__device__ inline float finite_top(float m) { return fminf(m, 0x1.fffffep127f); }

// What the exponentials of a part are taken of: z - from, with reference r.
struct Basis {
    float r, from;
    bool large;
};

__device__ inline Basis basis_of(float m, float shift)
{
    Basis b;
    b.large = is_large(m);
    b.r = b.large ? shift : reference(m, shift);
    // a NaN logit makes its E NaN, and with it the sum; one of +inf makes them
    // inf, since m is taken as the largest float there; a part of -inf alone has
    // E = 0
    b.from = b.large && m != -INFINITY ? finite_top(m) : 0.0f;
    return b;
}

// Epilogue of the logits' product: i is the vocabulary, j the gathered row.  A
// lane holds 32 of a row's 128 logits of the wave, the lanes 16, 32 and 48 from
// it the others.
template <class T, bool GRAD>
struct LogitsEpilogue {
    Rows rows;
    float *target_logit;
    vec<float, 2> *stats;  // [row][part]: m, l
    int32_t parts;
    uint16_t *e;           // [row][pitch]
    int64_t pitch;
    float *split;          // sums of tiles that are split over k

    struct Targets {
        int32_t t[4];
    };

    __device__ Targets prepare(int j0, int ny, int lane) const
    {
        Targets a;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int j = j0 + y * 16 + (lane & 15);
            a.t[y] = j < ny ? rows.target[rows.first + j] : -1;
        }
        return a;
    }

    __device__ void operator()(const Accumulators &acc, const Targets &targets, char *lds, const TilePlace &place,
                               int i0, int j0, int nx, int ny, int lane) const
    {
        if (place.part >= 0) {
            store_part(acc, split, place, i0, j0, lds, lane);
            return;
        }
        const int quarter = (lane >> 4) << 2;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int j = j0 + y * 16 + (lane & 15);
            float z[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) z[k] = acc.v[k >> 2][y][k & 3];
            if (i0 + kPart > nx) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (i0 + (k >> 2) * 16 + quarter + (k & 3) >= nx) z[k] = -INFINITY;
            }
            const int at = targets.t[y] >= 0 ? targets.t[y] - i0 - quarter : -1;
            if (__any(at >= 0 && at < kPart)) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (at == (k >> 2) * 16 + (k & 3)) target_logit[j] = z[k];
            }
            float m = z[0];
#pragma unroll
            for (int k = 1; k < 32; ++k) m = fmaxf(m, z[k]);
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const Basis basis = basis_of(m, Kept<T>::kShift);
            if (__any(basis.large)) {
#pragma unroll
                for (int k = 0; k < 32; ++k) z[k] -= basis.from;
            }
            float l = 0.0f;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                z[k] = __builtin_amdgcn_exp2f(fmaf(z[k], kLog2e, basis.r));
                l += z[k];
            }
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            if (j < ny && lane < 16) stats[int64_t(j) * parts + i0 / kPart] = vec<float, 2>{finite_top(m), l};
            if (GRAD) {
                // through LDS, so that a row's 128 values leave as one run; 16-byte
                // chunk c of row j sits in slot c ^ j.  Through the caches, where G's
                // pass finds a small E: past them 2048 x 2048 x 32768 took 712 us
                // instead of 705 and a large one (8192 x 4096 x 131072) as long
                char *line = lds + (lane & 15) * 256 + ((lane >> 4) & 1) * 8;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *(u16x4 *)(line + (((x * 2 + (lane >> 5)) ^ (lane & 15)) << 4)) = Kept<T>::pack(z + 4 * x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = k * 4 + (lane >> 4), chunk = lane & 15;
                    const vec<uint16_t, 8> v = *(const vec<uint16_t, 8> *)(lds + row * 256 + ((chunk ^ row) << 4));
                    const int to = j0 + y * 16 + row;
                    if (to < ny) *(vec<uint16_t, 8> *)(e + to * pitch + i0 + chunk * 8) = v;
                }
            }
        }
    }
};

// The same for the tiles whose products over k are split: a wave joins a row's
// 256 logits of a tile, half a wave for each of its two parts of the vocabulary.
template <class T, bool GRAD>
__global__ __launch_bounds__(256) void join_logits(GemmArgs a, LogitsEpilogue<T, GRAD> e)
{
    const int lane = threadIdx.x & 63, tile = blockIdx.x >> 6;
    const int row = (blockIdx.x & 63) * 4 + (threadIdx.x >> 6);
    int x, y;
    tile_at(a.rounds.full + tile, a.tiles_x, a.tiles_y(a.y.extent), x, y);
    const int64_t j = int64_t(y) * kTile + row;
    if (j >= a.counted()) return;
    const int i = x * kTile + lane * 4;
    const vec<float, 4> v = sum_parts<4>(e.split, a.rounds, tile, row, lane * 4);
    const int at = e.rows.target[e.rows.first + j] - i;
    float z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        z[k] = i + k < a.x.extent ? v[k] : -INFINITY;
        if (at == k) e.target_logit[j] = z[k];
    }
    float m = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const Basis basis = basis_of(m, Kept<T>::kShift);
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        z[k] = __builtin_amdgcn_exp2f(fmaf(z[k] - basis.from, kLog2e, basis.r));
        l += z[k];
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) l += __shfl_xor(l, d);
    if ((lane & 31) == 0) e.stats[j * e.parts + i / kPart] = vec<float, 2>{finite_top(m), l};
    if (GRAD) *(u16x4 *)(e.e + j * e.pitch + i) = Kept<T>::pack(z);
}

// The sum over some parts of exp(z - top), with top their largest logit.
struct Sum {
    float top, sum;

    __device__ void add(float other_top, float other_sum)
    {
        const float most = fmaxf(top, other_top);
        sum = sum * exp2f(float(exponent_below(top, most))) +
              other_sum * exp2f(float(exponent_below(other_top, most)));
        top = most;
    }
};

// lse and loss of a row; one workgroup a row.
template <class T>
__global__ __launch_bounds__(256) void xent_finish(Rows rows, const vec<float, 2> *stats, int parts,
                                                   const float *target_logit, const float *weight, const Unit *unit,
                                                   RowState *state, float *loss, float *lse)
{
    const float in_units = unit != nullptr ? unit->unit : kUnit<T>;
    __shared__ Sum waves[4];
    constexpr float kShift = Kept<T>::kShift;
    const float unshift = exp2f(-kShift);
    const int n = rows.here();
    for (int j = blockIdx.x; j < n; j += gridDim.x) {
        Sum a = {-INFINITY, 0.0f};
        for (int p = threadIdx.x; p < parts; p += 256) {
            const vec<float, 2> s = stats[int64_t(j) * parts + p];
            a.add(s[0], s[1] * unshift * exp2f(float(kShift - unit_exponent(s[0], kShift))));
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const float other_top = __shfl_xor(a.top, d), other_sum = __shfl_xor(a.sum, d);
            a.add(other_top, other_sum);
        }
        if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = a;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w) a.add(waves[w].top, waves[w].sum);
            // dividing by the float kLog2e undoes its own rounding
            const double log2_sum = log2(double(a.sum)), above = log2_sum / kLog2e;  // above: lse - top
            const int row = rows.index[rows.first + j];
            const int t = rows.target[rows.first + j];
            const bool first_copy = rows.copies == 1 || (j & 1) == 0;
            if (lse != nullptr && first_copy) lse[row] = float(double(a.top) + above);
            const float w = weight != nullptr ? weight[row] : 1.0f;
            // the two large terms first: their difference is what counts
            const double below = t >= 0 ? double(target_logit[j]) - double(a.top) - above : __builtin_nan("");
            if (first_copy) loss[row] = float(-w * below);
            RowState s;
            s.log2_sum = log2_sum;
            s.top = a.top;
            s.weight = t >= 0 && log2_sum < INFINITY ? w * in_units : __builtin_nanf("");
            s.target = t;
            s.own = s.weight * expm1f(float(below));
            state[j] = s;
        }
        __syncthreads();
    }
}

// E -> G in place; 8 columns of kGradRows rows a thread.
constexpr int kGradRows = 4;

template <class T>
__global__ __launch_bounds__(256) void xent_grad(Rows rows, const vec<float, 2> *stats, int parts,
                                                 const RowState *state, void *e, int64_t pitch)
{
    const int n = rows.here();
    const int i = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= pitch) return;
    for (int j0 = blockIdx.y * kGradRows; j0 < n; j0 += gridDim.y * kGradRows) {
        vec<uint16_t, 8> v[kGradRows];
        float m[kGradRows];
#pragma unroll
        for (int k = 0; k < kGradRows; ++k) {
            const int64_t j = j0 + k < n ? j0 + k : n - 1;
            v[k] = *(const vec<uint16_t, 8> *)((const uint16_t *)e + j * pitch + i);
            m[k] = stats[j * parts + i / kPart][0];
        }
#pragma unroll
        for (int k = 0; k < kGradRows; ++k) {
            if (j0 + k >= n) break;
            const RowState s = state[j0 + k];
            const float p = s.weight * exp2f(float(exponent_below(m[k], s.top) -
                                                   unit_exponent(m[k], Kept<T>::kShift) - s.log2_sum));
            const bool lost = rows.copies == 2 && ((j0 + k) & 1);  // what the row before rounds away
            vec<T, 8> g;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float f = Kept<T>::unpack(v[k][c]) * p;
                if (s.target == i + c) f = s.own;
                g[c] = T(lost ? f - float(T(f)) : f);
            }
            *(vec<T, 8> *)((T *)e + (j0 + k) * pitch + i) = g;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int64_t kPieceBytes = int64_t(1) << 30;

bool valid(const adam_xent_desc &d)
{
    return d.rows >= 0 && d.rows <= kMaxProductRows && d.hidden >= 1 && d.hidden <= kMaxDirectStride && d.vocab >= 1 &&
           d.vocab <= kMaxDirectStride - kTile && valid_matrix(d.rows, d.hidden, d.h_stride) &&
           valid_matrix(d.vocab, d.hidden, d.w_stride) &&
           (d.dh == nullptr || valid_matrix(d.rows, d.hidden, d.dh_stride)) &&
           (d.dw == nullptr || valid_matrix(d.vocab, d.hidden, d.dw_stride)) &&
           (d.accumulate == 0 || d.accumulate == 1) && d.piece_rows >= 0 && d.piece_rows <= kMaxSize;
}

// Rows held at once; round_up(d.rows) where that is all of them.
int64_t piece_of(const adam_xent_desc &d)
{
    const bool grad = d.dh != nullptr || d.dw != nullptr;
    const int64_t all = std::max<int64_t>(round_up(d.rows, kTile), kTile);
    if (d.piece_rows > 0) return std::min(round_up(d.piece_rows, kTile), all);
    if (!grad) return std::min<int64_t>(all, 16384);
    const int64_t row = round_up(d.vocab, kTile) * 2;
    const int64_t some = std::max<int64_t>(kPieceBytes / row / kTile * kTile, kTile);
    // pieces of a 16-bit dw need its sums in float: where all rows at once
    // take no more memory than that, there is one piece
    const bool sums = d.dw != nullptr && d.dw_type != ADAM_DT_F32;
    if (sums && all * row <= some * row + d.vocab * d.hidden * 4) return all;
    return std::min(some, all);
}

int check(const adam_xent_desc &d)
{
    if (d.type < ADAM_DT_NONE || d.type > ADAM_DT_F16 || d.dw_type < ADAM_DT_NONE || d.dw_type > ADAM_DT_F16)
        return ADAM_EINVAL;
    if (!is_half(d.type) || (d.dw != nullptr && d.dw_type != ADAM_DT_F32 && d.dw_type != d.type)) return ADAM_EDTYPE;
    if (!valid(d)) return ADAM_EINVAL;
    const int64_t piece = piece_of(d);
    return too_many_tiles(d.vocab, piece) || too_many_tiles(d.hidden, piece) || too_many_tiles(d.hidden, d.vocab)
               ? ADAM_EINVAL
               : ADAM_OK;
}

struct XentPlan {
    int64_t piece, pieces, h_pitch, v_pitch, parts, bytes;
    int32_t copies;
    Product dh, dw;
    bool grad, pack_w, sum_w;  // sum_w: dw is summed over the pieces in float
    int32_t *index, *targets, *places, *count;
    uint16_t *h, *w, *e;
    vec<float, 2> *stats;
    RowState *state;
    float *target_logit, *part, *sum;
    Unit *unit;

    XentPlan(const adam_xent_desc &d, void *workspace)
        : piece(piece_of(d)),
          pieces(std::max<int64_t>((d.rows + piece - 1) / piece, 1)), h_pitch(round_up(d.hidden, 8)),
          v_pitch(round_up(d.vocab, kTile)), parts(v_pitch / kPart),
          dh(d.hidden, piece, v_pitch, true),
          dw(d.hidden, d.vocab, d.rows <= kTwiceRows ? 2 * d.rows : std::min(piece, d.rows))
    {
        grad = d.dh != nullptr || d.dw != nullptr;
        copies = grad && d.rows <= kTwiceRows ? 2 : 1;  // then piece is kTile
        pack_w = !direct(d.w, d.w_stride, d.hidden, true);
        sum_w = d.dw != nullptr && d.dw_type != ADAM_DT_F32 && pieces > 1;
        Workspace s{(char *)workspace};
        index = s.take<int32_t>(d.rows * copies);
        targets = s.take<int32_t>(d.rows * copies);
        places = s.take<int32_t>(d.rows);
        count = s.take<int32_t>(1);
        unit = s.take<Unit>(1);
        h = s.take<uint16_t>(piece * h_pitch);
        w = s.take<uint16_t>(pack_w ? d.vocab * h_pitch : 0);
        stats = s.take<vec<float, 2>>(piece * parts);
        target_logit = s.take<float>(piece);
        state = s.take<RowState>(piece);
        e = s.take<uint16_t>(grad ? piece * v_pitch : 0);
        // the products follow each other, so they share the space of their
        // parts; pieces of fewer rows than `piece` have other rounds
        int64_t floats = std::max(d.dh != nullptr ? dh.part_floats() : 0, d.dw != nullptr ? dw.part_floats() : 0);
        for (const int64_t here : {std::min(piece, d.rows * copies), d.rows * copies - (pieces - 1) * piece})
            floats = std::max(floats, Product(d.vocab, here, h_pitch).part_floats());
        part = s.take<float>(floats);
        sum = s.take<float>(sum_w ? d.vocab * h_pitch : 0);
        bytes = s.used;
    }
};

// The logits of a piece: statistics and, for the gradient, E.
template <class T, bool GRAD>
int run_logits(const XentPlan &p, GemmArgs a, const Rows &rows, hipStream_t stream)
{
    const Product product(a.x.extent, a.y.extent, p.h_pitch);
    a.tiles_x = product.tiles_x;
    a.rounds = product.rounds;
    const LogitsEpilogue<T, GRAD> e = {rows, p.target_logit, p.stats, int32_t(p.parts), p.e, p.v_pitch, p.part};
    hipLaunchKernelGGL((gemm_kernel<T, kRows, kRows, LogitsEpilogue<T, GRAD>>), dim3(uint32_t(product.units)),
                       dim3(kThreads), 0, stream, a, e);
    if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
    if (product.split_tiles == 0) return ADAM_OK;
    hipLaunchKernelGGL((join_logits<T, GRAD>), dim3(uint32_t(product.split_tiles * 64)), dim3(256), 0, stream, a, e);
    return launched();
}

template <class T>
int run(const adam_xent_desc &d, const XentPlan &p, hipStream_t stream)
{
    const int rows = int(d.rows), hidden = int(d.hidden), vocab = int(d.vocab);
    const bool at_once = rows > 0 && rows <= kDirectRows && p.pieces == 1;
    // fp16 with weights: G's unit is chosen on the device
    Unit *const unit = p.grad && d.weight != nullptr && d.type == ADAM_DT_F16 ? p.unit : nullptr;
    const float *const scale = unit != nullptr ? &unit->scale : d.d_loss_scale;
    const float factor = unit != nullptr ? 1.0f : 1.0f / kUnit<T>;
    if (at_once)
        hipLaunchKernelGGL(xent_gather_rows, dim3(rows), dim3(256), 0, stream, d.target, d.ignore_index, rows, d.vocab,
                           p.copies, p.index, p.targets, p.count, d.loss, d.lse, (const uint16_t *)d.h, d.h_stride,
                           hidden, p.h, p.h_pitch, (uint16_t *)d.dh, d.dh_stride, d.weight, d.d_loss_scale,
                           unit);
    else
        hipLaunchKernelGGL(xent_gather, dim3(1), dim3(1024), 0, stream, d.target, d.ignore_index, rows, d.vocab,
                           p.index, p.targets, p.places, p.count, d.loss, d.lse, d.weight, d.d_loss_scale, unit);
    if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
    const void *w = d.w;
    int64_t w_stride = d.w_stride;
    if (p.pack_w && rows > 0) {
        const int rc = pack(w, w_stride, vocab, hidden, p.w, p.h_pitch, stream);
        if (rc != ADAM_OK) return rc;
        w = p.w;
        w_stride = p.h_pitch;
    }
    for (int64_t n = 0; n < p.pieces; ++n) {
        const int first = int(n * p.piece);
        const int here = int(std::min(p.piece, d.rows * p.copies - first));  // gathered rows: at most these
        const Rows at = {p.index, p.targets, p.count, first, here, p.copies};
        if (here > 0) {
            if (!at_once) {
                hipLaunchKernelGGL(xent_rows, dim3(std::min(rows, 1 << 20)), dim3(256), 0, stream, p.places, rows,
                                   first, here, (const uint16_t *)d.h, d.h_stride, hidden, p.h, p.h_pitch,
                                   (uint16_t *)(n == 0 ? d.dh : nullptr), d.dh_stride);
                if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            }
            GemmArgs a = {};
            // the gathered rows' padding is 0, so k may run to their pitch
            // where w's does
            a.x = Operand{w, nullptr, w_stride, vocab, p.pack_w ? int32_t(p.h_pitch) : hidden};
            a.y = Operand{p.h, nullptr, p.h_pitch, here, int32_t(p.h_pitch)};
            a.count = p.count;
            a.first = first;
            a.most = here;
            const int rc0 = p.grad ? run_logits<T, true>(p, a, at, stream) : run_logits<T, false>(p, a, at, stream);
            if (rc0 != ADAM_OK) return rc0;
            hipLaunchKernelGGL((xent_finish<T>), dim3(std::min(here, 65536)), dim3(256), 0, stream, at, p.stats,
                               int(p.parts), p.target_logit, d.weight, unit, p.state, d.loss, d.lse);
            if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            if (p.grad) {
                const int64_t columns = (p.v_pitch + 2047) / 2048, groups = (here + kGradRows - 1) / kGradRows;
                hipLaunchKernelGGL((xent_grad<T>),
                                   dim3(uint32_t(columns), uint32_t(std::min({groups, int64_t(32768), (1 << 23) / columns}))),
                                   dim3(256), 0, stream, at, p.stats, int(p.parts), p.state, (void *)p.e, p.v_pitch);
                if (hipGetLastError() != hipSuccess) return ADAM_EHIP;
            }
            if (d.dh != nullptr) {
                GemmArgs g = {};
                g.x = Operand{w, nullptr, w_stride, hidden, vocab};
                g.y = Operand{p.e, nullptr, p.v_pitch, here, int32_t(p.v_pitch)};
                g.count = p.count;
                g.first = first;
                g.most = here;
                StoreEpilogue<T> e = {};
                e.out = (T *)d.dh;
                e.stride = d.dh_stride;
                e.alpha = scale;
                e.factor = factor;
                e.rows = p.index + first;
                e.pairs = p.copies == 2;
                const int rc = run_product<T, kCols, kRows>(p.dh, g, e, p.part, stream);
                if (rc != ADAM_OK) return rc;
            }
        }
        if (d.dw != nullptr) {
            GemmArgs g = {};
            g.x = Operand{p.h, nullptr, p.h_pitch, hidden, here};
            g.y = Operand{p.e, nullptr, p.v_pitch, vocab, here};
            g.count = p.count;
            g.first = first;
            g.most = here;
            g.count_is_depth = 1;
            const bool last = n == p.pieces - 1;
            auto product = [&](auto o, void *out, int64_t stride, const float *add, bool accumulate) {
                using O = decltype(o);
                StoreEpilogue<O> e = {};
                e.out = (O *)out;
                e.stride = stride;
                e.alpha = scale;
                e.factor = factor;
                e.add = add;
                e.add_stride = p.h_pitch;
                e.accumulate = accumulate;
                return run_product<T, kCols, kCols>(p.dw, g, e, p.part, stream);
            };
            int rc;
            if (d.dw_type == ADAM_DT_F32)
                rc = product(float(), d.dw, d.dw_stride, nullptr, d.accumulate || n > 0);
            else if (!last)
                rc = product(float(), p.sum, p.h_pitch, nullptr, n > 0);
            else
                rc = product(T(), d.dw, d.dw_stride, n > 0 ? p.sum : nullptr, d.accumulate);
            if (rc != ADAM_OK) return rc;
        }
    }
    return ADAM_OK;
}

}  // namespace
}  // namespace train

using namespace train;

extern "C" {

int adam_xent_plan(const adam_xent_desc *desc, adam_xent_stats *stats)
{
    if (desc == nullptr || stats == nullptr) return ADAM_EINVAL;
    const int rc = check(*desc);
    if (rc != ADAM_OK) return rc;
    const XentPlan p(*desc, nullptr);
    stats->workspace_bytes = p.bytes;
    stats->piece_rows = p.piece;
    stats->pieces = p.pieces;
    return ADAM_OK;
}

int adam_xent(const adam_xent_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (desc == nullptr) return ADAM_EINVAL;
    const adam_xent_desc &d = *desc;
    int rc = check(d);
    if (rc != ADAM_OK) return rc;
    if (d.rows == 0 && d.dw == nullptr) return ADAM_OK;
    if (d.rows > 0 && (d.h == nullptr || d.w == nullptr || d.target == nullptr || d.loss == nullptr))
        return ADAM_EINVAL;
    const int ob = dtype_bytes(d.dw_type);
    if (!aligned(d.h, 2) || !aligned(d.w, 2) || !aligned(d.target, 8) || !aligned(d.weight, 4) ||
        !aligned(d.loss, 4) || !aligned(d.lse, 4) || !aligned(d.dh, 2) || !aligned(d.d_loss_scale, 4) ||
        (d.dw != nullptr && !aligned(d.dw, ob)))
        return ADAM_EINVAL;
    const XentPlan p(d, workspace);
    if (workspace == nullptr || workspace_bytes < p.bytes || !aligned(workspace, 256)) return ADAM_EINVAL;
    const View in[6] = {matrix(d.h, d.rows, d.hidden, d.h_stride, 2), matrix(d.w, d.vocab, d.hidden, d.w_stride, 2),
                        flat(d.target, d.rows * 8), flat(d.weight, d.rows * 4), flat(d.d_loss_scale, 4), View{}};
    const View out[5] = {flat(d.loss, d.rows * 4), flat(d.lse, d.rows * 4),
                         matrix(d.dh, d.rows, d.hidden, d.dh_stride, 2),
                         matrix(d.dw, d.vocab, d.hidden, d.dw_stride, ob), flat(workspace, p.bytes)};
    for (int i = 0; i < 5; ++i) {
        for (const View &v : in)
            if (overlap(out[i], v)) return ADAM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return ADAM_EINVAL;
    }
    StreamGuard guard(stream);
    if (guard.status != hipSuccess) return ADAM_EHIP;
    return d.type == ADAM_DT_BF16 ? run<bf16>(d, p, stream) : run<f16>(d, p, stream);
}

}  // extern "C"
