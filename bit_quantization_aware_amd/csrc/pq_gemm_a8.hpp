// pq_gemm_a8.hpp -- internal pieces of the packed product of 8-bit activations:
// arguments, the decoding of codes to int8, and the epilogue.  Not part of the
// C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pq_gemm_common.hpp"
#include "pq_row_common.hpp"

namespace pq {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

struct A8Args {
    const int8_t *X;         // [M, K], rows x_st bytes apart
    const float *x_scale;
    const uint8_t *packed;   // export byte order
    const void *alpha, *bias, *other;
    void *Y;
    int32_t *partial;        // split K: [splits, M, p_st]
    int64_t x_st, y_st, o_st, p_st, gstride;
    int M, N, K;
    int alpha_dtype, bias_dtype, y_dtype, act, mul;   // mul: multiply by other
    int splits, nt;          // shares of K; stores past the caches
    float unit;              // level = unit * decoded int8
    uint32_t lut;            // 1, 2 bits: level of code c in byte c
    uint32_t flip, mask;     // 4 bits: code ^ flip, masked, stands in the byte's upper bits
    int up;                  //         shifted left by this
};

// Sixteen consecutive codes of a column to int8, in order.
//
// 2 bits (one word of the export's order: byte j holds codes 2j, 8 + 2j,
// 2j + 1, 9 + 2j): four masks give the even and the odd codes of each half as
// bytes, v_perm puts them in order, and a second v_perm takes each code as the
// index of a byte of the level table -- 15 operations.
// 4 bits: code c of n levels stands for c - n / 2, which is c with its top bit
// flipped, read as a signed number; left in the byte's upper bits it needs no
// sign extension, and the unit takes the factor (2^4 or 2^5) back.
// 1 bit: four codes times 2^0 + 2^7 + 2^14 + 2^21 land in bit 0 of four bytes.
template <int BITS>
struct Words;                // the words that hold sixteen codes
template <>
struct Words<1> { uint32_t w; };         // the low half
template <>
struct Words<2> { uint32_t w; };
template <>
struct Words<4> { uint32_t w, v; };

__device__ __forceinline__ intx4 decode(const A8Args &a, const Words<2> &c)
{
    const uint32_t e = c.w & 0x03030303u, o = (c.w >> 4) & 0x03030303u;
    const uint32_t f = (c.w >> 2) & 0x03030303u, q = (c.w >> 6) & 0x03030303u;
    intx4 r;
    r[0] = __builtin_amdgcn_perm(a.lut, a.lut, __builtin_amdgcn_perm(o, e, 0x05010400));
    r[1] = __builtin_amdgcn_perm(a.lut, a.lut, __builtin_amdgcn_perm(o, e, 0x07030602));
    r[2] = __builtin_amdgcn_perm(a.lut, a.lut, __builtin_amdgcn_perm(q, f, 0x05010400));
    r[3] = __builtin_amdgcn_perm(a.lut, a.lut, __builtin_amdgcn_perm(q, f, 0x07030602));
    return r;
}
__device__ __forceinline__ intx4 decode(const A8Args &a, const Words<4> &c)
{
    intx4 r;
    const uint32_t w[2] = {c.w ^ a.flip, c.v ^ a.flip};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = (w[i] << a.up) & a.mask, e = (w[i] << (a.up + 4)) & a.mask;
        r[2 * i] = __builtin_amdgcn_perm(o, e, 0x05010400);
        r[2 * i + 1] = __builtin_amdgcn_perm(o, e, 0x07030602);
    }
    return r;
}
__device__ __forceinline__ intx4 decode(const A8Args &a, const Words<1> &c)
{
    intx4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __umul24((c.w >> (4 * i)) & 15u, 0x204081u) & 0x01010101u;
        r[i] = __builtin_amdgcn_perm(a.lut, a.lut, b);
    }
    return r;
}

// e^-x by the hardware's exponential, which is within a unit of fp32's last
// place, as its reciprocal is; the rounded product with log2 e is off by up to
// 1.5 |x| units more.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(-1.4426950408889634f * x); }

// The normal distribution's tail erfc(a / sqrt 2) / 2, a >= 0, with a relative
// error like e^(-a^2 / 2)'s: t 2^(P(t) - a^2 log2(e) / 2), t = 1 / (1 + a / sqrt 8).
// P is a Chebyshev fit of degree 9 to log2 of erfc(z) e^(z^2) / 2t over the range
// in which the tail is a normal fp32 number (off by 4.5e-8 at most).  1 + erf
// would cancel on the negative side (4 % of the tail at a = 5) and takes longer
// (8192 x 14336 x 4096 with a second operand 495 us against 446).
__device__ __forceinline__ float normal_tail(float a)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35355339059327379f, 1.f));
    float p = 0.20333263278007507f;
    p = __builtin_fmaf(p, t, -0.9507189989089966f);
    p = __builtin_fmaf(p, t, 1.594277262687683f);
    p = __builtin_fmaf(p, t, -0.9046970009803772f);
    p = __builtin_fmaf(p, t, -0.19887569546699524f);
    p = __builtin_fmaf(p, t, 0.04626460745930672f);
    p = __builtin_fmaf(p, t, 0.034691065549850464f);
    p = __builtin_fmaf(p, t, 0.5610182285308838f);
    p = __builtin_fmaf(p, t, 1.4403448104858398f);
    p = __builtin_fmaf(p, t, -2.825636863708496f);
    return t * __builtin_amdgcn_exp2f(__builtin_fmaf(a * a, -0.72134752044448170f, p));
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act)
{
    if (act == PQ_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];      // NaN stays
    } else if (act == PQ_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= __builtin_amdgcn_rcpf(1.f + exp_neg(v[e]));
    } else if (act == PQ_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float tail = normal_tail(__builtin_fabsf(v[e]));
            v[e] *= v[e] < 0.f ? tail : 1.f - tail;
        }
    } else if (act == PQ_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] *= __builtin_amdgcn_rcpf(1.f + exp_neg(1.5957691216057308f * v[e] * (1.f + 0.044715f * v[e] * v[e])));
    }
}

// Scale (with the levels' unit) and bias of columns 8c .. 8c + 7 (0 past N).
__device__ __forceinline__ void columns8(const A8Args &a, int c, float (&cs)[8], float (&cb)[8])
{
    load_any8(a.alpha, a.alpha_dtype, c, a.N, cs);
    if (a.bias) {
        load_any8(a.bias, a.bias_dtype, c, a.N, cb);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) cb[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] *= a.unit;
}

// Eight outputs of a row: scales, bias, activation, other.
template <typename T>
__device__ __forceinline__ void outputs8(const A8Args &a, float row_scale, const int (&sum)[8], const float (&cs)[8],
                                         const float (&cb)[8], const Raw8<T> &other, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(static_cast<float>(sum[e]), row_scale * cs[e], cb[e]);
    activate(v, a.act);
    if (!a.other) return;
    float o[8];
    raw_to_f32<T>(other, o);
    if (a.mul) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= o[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += o[e];
    }
}

// Eight outputs of row m, columns 8c .. 8c + 7 (those below N), and the store.
template <typename T>
__device__ __forceinline__ void finish8(const A8Args &a, int64_t m, int c, float row_scale, const int (&sum)[8], const float (&cs)[8],
                                        const float (&cb)[8])
{
    float v[8];
    Raw8<T> other;
    if (a.other) other = load_row8(static_cast<const T *>(a.other) + m * a.o_st, c, a.N);
    outputs8<T>(a, row_scale, sum, cs, cb, other, v);
    store_row8<T>(static_cast<T *>(a.Y) + m * a.y_st, c, a.N, v);
}

// f(T{}) for y's type.
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F &&f)
{
    if (dtype == PQ_F32) f(float{});
    else if (dtype == PQ_BF16) f(bf16_t{});
    else f(f16_t{});
}

}  // namespace
}  // namespace pq
