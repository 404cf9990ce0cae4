// pq_gemm_a8.hpp -- internal pieces of the packed product of 8-bit activations:
// arguments, the decoding of codes to int8, and the epilogue.  Not part of the
// C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pq_gemm_common.hpp"
#include "pq_kv_common.hpp"

namespace pq {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

struct A8Args {
    const int8_t *X;         // [M, K], rows x_st bytes apart
    const float *x_scale;
    const uint8_t *packed;   // export byte order
    const void *alpha, *bias, *other;
    void *Y;
    int32_t *partial;        // split K: [splits, M, N]
    int64_t x_st, y_st, o_st, gstride;
    int M, N, K;
    int alpha_dtype, bias_dtype, y_dtype, act, mul;   // mul: multiply by other
    int splits;
    float unit;              // level = unit * decoded int8
    uint32_t lut_lo, lut_hi;             // 1, 2 bits: level of code c in byte c
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
    r[0] = __builtin_amdgcn_perm(a.lut_lo, a.lut_lo, __builtin_amdgcn_perm(o, e, 0x05010400));
    r[1] = __builtin_amdgcn_perm(a.lut_lo, a.lut_lo, __builtin_amdgcn_perm(o, e, 0x07030602));
    r[2] = __builtin_amdgcn_perm(a.lut_lo, a.lut_lo, __builtin_amdgcn_perm(q, f, 0x05010400));
    r[3] = __builtin_amdgcn_perm(a.lut_lo, a.lut_lo, __builtin_amdgcn_perm(q, f, 0x07030602));
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
        r[i] = __builtin_amdgcn_perm(a.lut_lo, a.lut_lo, b);
    }
    return r;
}

__device__ __forceinline__ float any_f32(const void *p, int dtype, int64_t i)
{
    if (dtype == PQ_F32) return static_cast<const float *>(p)[i];
    if (dtype == PQ_BF16) return to_f32(static_cast<const bf16_t *>(p)[i]);
    return to_f32(static_cast<const f16_t *>(p)[i]);
}

// e^-x by the hardware's exponential and a reciprocal: both are off by a unit
// of the last place of fp32, as the products around them.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(-1.4426950408889634f * x); }

__device__ __forceinline__ float activate(float v, int act)
{
    if (act == PQ_ACT_RELU) return v < 0.f ? 0.f : v;        // NaN stays
    if (act == PQ_ACT_SILU) return v / (1.f + exp_neg(v));
    if (act == PQ_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (act == PQ_ACT_GELU_TANH) {
        // 1 + tanh(u) = 2 / (1 + e^-2u)
        const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
        return v / (1.f + exp_neg(2.f * u));
    }
    return v;
}

// One output: row's scale times column's scale, bias, activation, other.
__device__ __forceinline__ float finish(const A8Args &a, int sum, float row_scale, float col_scale, float bias, float other)
{
    const float v = activate(__builtin_fmaf(static_cast<float>(sum), row_scale * col_scale, bias), a.act);
    return a.mul ? v * other : v + other;
}

// Four consecutive columns of a row, n0 .. n0 + 3 (those below N).
__device__ __forceinline__ void store4(const A8Args &a, int m, int n0, const intx4 &sum, const float (&cs)[4], const float (&cb)[4])
{
    const float rs = a.x_scale[m];
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = min(n0 + e, a.N - 1);
        const float other = a.other ? any_f32(a.other, a.y_dtype, m * a.o_st + n) : 0.f;
        y[e] = finish(a, sum[e], rs, cs[e], cb[e], other);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (n0 + e >= a.N) break;
        const int64_t at = m * a.y_st + n0 + e;
        if (a.y_dtype == PQ_F32) static_cast<float *>(a.Y)[at] = y[e];
        else if (a.y_dtype == PQ_BF16) static_cast<bf16_t *>(a.Y)[at] = from_f32<bf16_t>(y[e]);
        else static_cast<f16_t *>(a.Y)[at] = from_f32<f16_t>(y[e]);
    }
}

// Scale (with the levels' unit) and bias of columns n0 .. n0 + 3.
__device__ __forceinline__ void columns4(const A8Args &a, int n0, float (&cs)[4], float (&cb)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = min(n0 + e, a.N - 1);
        cs[e] = any_f32(a.alpha, a.alpha_dtype, n) * a.unit;
        cb[e] = a.bias ? any_f32(a.bias, a.bias_dtype, n) : 0.f;
    }
}

}  // namespace
}  // namespace pq
