// pq_gemm_a8.hip -- the packed product of 8-bit activations (gfx950): codes in
// the export byte order x int8 rows on the int8 matrix unit, with scales,
// bias, activation and a second operand in the epilogue.
//
// Every level is a whole number times a common unit, so codes are decoded to
// int8 and the sum over K is an integer: exact, whatever its order or split.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pq_common.hpp"
#include "pq_gemm_a8.hpp"

namespace pq {
namespace {

constexpr int64_t kMaxA8K = (int64_t(1) << 17) - 64;
constexpr int64_t kMaxA8 = int64_t(1) << 24;

// One 16-column tile by 16 MT rows a block; its four waves take every fourth
// 64-byte group of K and add their sums through LDS.  No activations in LDS:
// a lane reads the sixteen values its codes stand against.
template <int BITS, int MT>
__global__ __launch_bounds__(256) void k_a8_stream(A8Args a)
{
    __shared__ intx4 red[3][MT][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int i16 = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x, m0 = blockIdx.y * (16 * MT);
    constexpr int GK = 512 / BITS;              // k of a 64-byte group
    const int groups = (a.K + GK - 1) / GK;
    intx4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = intx4{0, 0, 0, 0};
    const int8_t *x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = a.X + min(m0 + 16 * t + i16, a.M - 1) * a.x_st;
    for (int q = w; q < groups; q += 4) {
        const u32x4 c = *reinterpret_cast<const u32x4 *>(a.packed + q * a.gstride + static_cast<int64_t>(tile) * 1024 +
                                                          i16 * 64 + g * 16);
#pragma unroll
        for (int j = 0; j < GK / 64; ++j) {
            Words<BITS> wd;
            if constexpr (BITS == 1) wd.w = c[j >> 1] >> (16 * (j & 1));
            if constexpr (BITS == 2) wd.w = c[j];
            if constexpr (BITS == 4) wd = {c[2 * j], c[2 * j + 1]};
            const intx4 b = decode(a, wd);
            const int k = q * GK + g * (GK / 4) + j * 16;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                intx4 v = {0, 0, 0, 0};
                if (k < a.K) v = *reinterpret_cast<const intx4 *>(x[t] + k);
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, v, acc[t], 0, 0, 0);
            }
        }
    }
    if (w > 0) {
#pragma unroll
        for (int t = 0; t < MT; ++t) red[w - 1][t][lane] = acc[t];
    }
    __syncthreads();
    if (w > 0) return;
    const int n0 = tile * 16 + 4 * g;
    if (n0 >= a.N) return;
    float cs[4], cb[4];
    columns4(a, n0, cs, cb);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + i16;
        if (m < a.M) store4(a, m, n0, acc[t] + red[0][t][lane] + red[1][t][lane] + red[2][t][lane], cs, cb);
    }
}

template <int BITS>
pq_status launch_a8(const A8Args &a, hipStream_t s)
{
    const unsigned tiles = static_cast<unsigned>((a.N + 15) / 16);
    if (a.M <= 16) {
        hipLaunchKernelGGL((k_a8_stream<BITS, 1>), dim3(tiles), dim3(256), 0, s, a);
        return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
    }
    A8Args b = a;
    // grid rows are counted in 16 bits: more rows go in several launches
    constexpr int64_t kStep = 65535 * 64;
    for (int64_t m = 0; m < a.M; m += kStep) {
        b.M = static_cast<int>(a.M - m < kStep ? a.M - m : kStep);
        b.X = a.X + m * a.x_st;
        b.x_scale = a.x_scale + m;
        const int size = a.y_dtype == PQ_F32 ? 4 : 2;
        b.Y = static_cast<char *>(a.Y) + m * a.y_st * size;
        b.other = a.other ? static_cast<const char *>(a.other) + m * a.o_st * size : nullptr;
        hipLaunchKernelGGL((k_a8_stream<BITS, 4>), dim3(tiles, static_cast<unsigned>((b.M + 63) / 64)), dim3(256), 0, s, b);
        if (hipGetLastError() != hipSuccess) return PQ_ERR_HIP;
    }
    return PQ_OK;
}

inline bool a8_shape_ok(int mode, int64_t M, int64_t N, int64_t K)
{
    return valid_mode(mode) && M >= 0 && M <= kMaxA8 && N >= 0 && N <= kMaxA8 && K > 0 && K % 64 == 0 && K <= kMaxA8K;
}

// The mode's levels as whole numbers of a unit, and how the kernels decode them.
inline void set_levels(A8Args &a, int mode)
{
    auto lut = [&](int l0, int l1, int l2, int l3, float unit) {
        a.lut_lo = a.lut_hi = (l0 & 255u) | (l1 & 255u) << 8 | (l2 & 255u) << 16 | (l3 & 255u) << 24;
        a.unit = unit;
    };
    switch (mode) {
    case PQ_W1_BINARY: lut(-1, 1, 0, 0, 1.f); break;
    case PQ_W158_SEQ_TERNARY: lut(-1, 0, 1, 2, 2.f / 3.f); break;
    case PQ_W2_SEQ: lut(-3, -1, 1, 3, 0.25f); break;
    case PQ_W2_LSQ: lut(-2, -1, 0, 1, 1.f); break;
    case PQ_W158_LSQ: lut(-1, 0, 1, 2, 1.f); break;
    case PQ_W3_LSQ:
        a.flip = 0x44444444u;
        a.mask = 0xe0e0e0e0u;
        a.up = 1;
        a.unit = 1.f / 32;
        break;
    default:
        a.flip = 0x88888888u;
        a.mask = 0xf0f0f0f0u;
        a.up = 0;
        a.unit = 1.f / 16;
    }
}

}  // namespace
}  // namespace pq

extern "C" {

int64_t pq_gemm_a8_workspace_bytes(int mode, int64_t M, int64_t N, int64_t K)
{
    return pq::a8_shape_ok(mode, M, N, K) ? 0 : -1;
}

pq_status pq_gemm_a8(int mode, int64_t M, int64_t N, int64_t K, const int8_t *X, int64_t x_stride,
                     const float *x_scale, const uint8_t *packed, const void *alpha, int alpha_dtype,
                     const pq_epilogue *epilogue, int y_dtype, void *Y, int64_t y_stride, void *workspace,
                     int64_t workspace_bytes, void *stream)
{
    using namespace pq;
    static const pq_epilogue none = {};
    const pq_epilogue &e = epilogue ? *epilogue : none;
    const int size = dtype_bytes(y_dtype);
    if (!valid_mode(mode) || !size || (alpha_dtype != PQ_BF16 && alpha_dtype != PQ_F32)) return PQ_ERR_MODE;
    if (e.activation < PQ_ACT_NONE || e.activation > PQ_ACT_GELU_TANH || (e.combine != PQ_COMBINE_ADD && e.combine != PQ_COMBINE_MUL))
        return PQ_ERR_MODE;
    if (e.bias && !dtype_bytes(e.bias_dtype)) return PQ_ERR_MODE;
    if (e.reserved != 0) return PQ_ERR_ARG;
    if (!a8_shape_ok(mode, M, N, K) || x_stride < K || x_stride % 16) return PQ_ERR_SHAPE;
    if (M == 0 || N == 0) return PQ_OK;
    const int64_t need = pq_gemm_a8_workspace_bytes(mode, M, N, K);
    if (!X || !x_scale || !packed || !alpha || !Y || (need > 0 && !workspace)) return PQ_ERR_NULL;
    auto off = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(X, 16) || off(x_scale, 4) || off(packed, 16) || off(alpha, dtype_bytes(alpha_dtype)) || off(Y, size) ||
        off(e.other, size) || (e.bias && off(e.bias, dtype_bytes(e.bias_dtype))) || (need > 0 && off(workspace, 16)))
        return PQ_ERR_ALIGN;
    if (workspace_bytes < 0 || (need > 0 && workspace_bytes < need)) return PQ_ERR_ARG;
    if (e.other && e.other == Y && e.other_stride != y_stride) return PQ_ERR_ARG;
    A8Args a = {};
    a.X = X;
    a.x_scale = x_scale;
    a.packed = packed;
    a.alpha = alpha;
    a.bias = e.bias;
    a.other = e.other;
    a.Y = Y;
    a.partial = static_cast<int32_t *>(workspace);
    a.x_st = x_stride;
    a.y_st = y_stride;
    a.o_st = e.other_stride;
    a.gstride = (N + 15) / 16 * 1024;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.alpha_dtype = alpha_dtype;
    a.bias_dtype = e.bias_dtype;
    a.y_dtype = y_dtype;
    a.act = e.activation;
    a.mul = e.other && e.combine == PQ_COMBINE_MUL;
    set_levels(a, mode);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int bits = code_bits(mode);
    return bits == 1 ? launch_a8<1>(a, s) : bits == 2 ? launch_a8<2>(a, s) : launch_a8<4>(a, s);
}

}  // extern "C"
