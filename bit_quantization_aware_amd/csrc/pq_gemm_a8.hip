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
constexpr int64_t kMaxXStride = int64_t(1) << 23;    // a tile's rows are within 32 bits of its first

// One 16-column tile by 16 MT rows a block; its four waves take every fourth
// 64-byte group of K and add their sums through LDS.  No activations in LDS:
// a lane reads the sixteen values its codes stand against.
template <int BITS, int MT>
__global__ __launch_bounds__(256) void k_a8_stream(A8Args a)
{
    __shared__ intx4 red[4][16 * MT * 5];       // rows of 16 sums, 16 bytes apart
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
    // Sums of the four waves; a lane then takes eight columns of a row.
#pragma unroll
    for (int t = 0; t < MT; ++t) red[w][(16 * t + i16) * 5 + g] = acc[t];
    __syncthreads();
    const int c = tile * 2 + (threadIdx.x & 1);
    if (8 * c >= a.N) return;
    float cs[8], cb[8];
    columns8(a, c, cs, cb);
    with_type(a.y_dtype, [&](auto type) __attribute__((always_inline)) {
        for (int r = threadIdx.x >> 1; r < min(16 * MT, a.M - m0); r += 128) {
            int sum[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = r * 5 + 2 * (threadIdx.x & 1) + h;
                const intx4 v = red[0][at] + red[1][at] + red[2][at] + red[3][at];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[4 * h + e] = v[e];
            }
            finish8<decltype(type)>(a, m0 + r, c, a.x_scale[m0 + r], sum, cs, cb);
        }
    });
}

// Output tiles of many rows: WN waves side by side, each 16 MT rows by 16 NT
// columns, over K in stages of 128.  A stage's activations (128 bytes a row,
// 16-byte chunks swizzled as in the bf16 kernels) and code bytes go from memory
// to LDS directly, into a ring of P slots.
template <int BITS, int WN, int MT, int NT, int P>
struct TileCfg {
    static constexpr int BM = 16 * MT, BN = 16 * NT * WN, THREADS = 64 * WN;
    static constexpr int PIECES = BITS == 4 ? 4 : 2;            // 16-byte pieces of a column a stage (1 bit: two stages' worth)
    static constexpr int XB = BM * 128, CB = BN * PIECES * 16, SLOT = XB + CB;
    static constexpr int XI = XB / 1024 / WN, CI = CB / 1024 / WN;   // loads a wave and stage
    static constexpr int EPI = 8 * MT * (BN * 4 + 16);              // the epilogue's half tile
    static constexpr int LDS = P * SLOT > EPI ? P * SLOT : EPI;
    static_assert(XI * WN * 1024 == XB && CI * WN * 1024 == CB, "whole loads");
};

template <int BITS, int WN, int MT, int NT, int P>
__global__ __launch_bounds__(64 * WN, 2) void k_a8_tile(A8Args a, int mtiles, int ntiles)
{
    using C = TileCfg<BITS, WN, MT, NT, P>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int i16 = lane & 15, g = lane >> 4;

    // One XCD's blocks take consecutive tiles, eight row tiles by all columns
    // at a time, so that its L2 serves both operands.
    int t = blockIdx.x;
    const int nb = gridDim.x;
    if ((nb & 7) == 0) t = (t & 7) * (nb >> 3) + (t >> 3);
    const int band = t / (8 * ntiles), rows = min(8, mtiles - 8 * band), in = t - band * 8 * ntiles;
    const int m0 = (8 * band + in % rows) * C::BM, n0 = in / rows * C::BN;

    const uint8_t *xb = reinterpret_cast<const uint8_t *>(a.X) + m0 * a.x_st;
    uint32_t xo[C::XI], xc[C::XI];
#pragma unroll
    for (int q = 0; q < C::XI; ++q) {
        const int r = 8 * (C::XI * w + q) + (lane >> 3);
        xc[q] = ((lane & 7) ^ xswz(r)) * 16;
        xo[q] = static_cast<uint32_t>((min(m0 + r, a.M - 1) - m0) * a.x_st) + xc[q];
    }
    const int last_tile = (a.N - 1) >> 4;
    uint32_t co[C::CI];
#pragma unroll
    for (int q = 0; q < C::CI; ++q) {
        const int at = C::CI * w + q;
        const int tile = BITS == 4 ? at : 2 * at + (lane >> 5), piece = BITS == 4 ? lane >> 4 : (lane >> 4) & 1;
        co[q] = static_cast<uint32_t>(min((n0 >> 4) + tile, last_tile) * 1024 + (lane & 15) * 64 + piece * 16);
    }
    const uint32_t lds_base = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds));
    const int steps = a.K / 64, stages = (steps + 1) / 2;

    // Stage s to its slot; past the last one the last again, so that the
    // number of loads in flight is the same at every wait.  The second half of
    // an odd last stage is not there: its chunks read the first half.
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        s = min(s, stages - 1);
        const uint32_t at = lds_base + slot * C::SLOT;
        const uint32_t cut = (2 * s + 1 < steps) ? 128 : 64;
#pragma unroll
        for (int q = 0; q < C::XI; ++q)
            dma16(xb + s * 128, xc[q] < cut ? xo[q] : xo[q] - 64, at + (C::XI * w + q) * 1024);
        const int group = BITS == 4 ? s : BITS == 2 ? s >> 1 : s >> 2;
        const uint8_t *cb = a.packed + group * a.gstride;
        const uint32_t part = BITS == 4 ? 0 : BITS == 2 ? (s & 1) * 32 : (s & 2) * 16;
#pragma unroll
        for (int q = 0; q < C::CI; ++q) dma16(cb, co[q] + part, at + C::XB + (C::CI * w + q) * 1024);
    };

    intx4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = intx4{0, 0, 0, 0};

    const uint8_t *xr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xr[h] = lds + i16 * 128 + (((4 * h + g) ^ xswz(i16)) << 4);
    const uint8_t *cr = lds + C::XB + w * NT * (C::PIECES * 256) + i16 * 16 +
                        (BITS == 4 ? (g >> 1) * 256 + (g & 1) * 8 : BITS == 2 ? g * 4 : (g >> 1) * 4);

    auto step = [&](auto h_c, int s, int slot) __attribute__((always_inline)) {
        constexpr int H = decltype(h_c)::value;
        const uint8_t *cp = cr + slot * C::SLOT + (BITS == 4 ? H * 512 : BITS == 2 ? H * 256 : H * 8 + (s & 1) * 256);
        Words<BITS> wd[NT];
        intx4 x[MT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if constexpr (BITS == 4) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(cp + j * (C::PIECES * 256));
                wd[j] = {v[0], v[1]};
            } else {
                wd[j].w = *reinterpret_cast<const uint32_t *>(cp + j * (C::PIECES * 256));
                if constexpr (BITS == 1) wd[j].w >>= 16 * (g & 1);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) x[i] = *reinterpret_cast<const intx4 *>(xr[H] + slot * C::SLOT + i * 2048);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const intx4 b = decode(a, wd[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, x[i], acc[i][j], 0, 0, 0);
        }
    };

#pragma unroll
    for (int s = 0; s < P - 1; ++s) issue(s, s);
    int slot = 0;
    for (int s = 0; s < stages; ++s) {
        wait_lgkmcnt0();
        wait_vmcnt<(P - 2) * (C::XI + C::CI)>();
        block_barrier();
        issue(s + P - 1, slot == 0 ? P - 1 : slot - 1);
        step(std::integral_constant<int, 0>{}, s, slot);
        if (2 * s + 1 < steps) step(std::integral_constant<int, 1>{}, s, slot);
        slot = slot == P - 1 ? 0 : slot + 1;
    }
    wait_vmcnt<0>();        // no load is in flight into LDS when the block ends

    // The sums through LDS, so that every output line is written whole: MT / 2
    // row tiles at a time, rows 16 bytes further apart than they are long (the
    // sixteen rows of a write then lie in different banks).
    constexpr int RS = C::BN * 4 + 16;
    const int c = (n0 >> 3) + threadIdx.x % (C::BN / 8);
    float cs[8], cb[8];
    columns8(a, c, cs, cb);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT / 2; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<intx4 *>(lds + (16 * i + i16) * RS + ((w * NT + j) * 16 + 4 * g) * 4) = acc[half * (MT / 2) + i][j];
        __syncthreads();
        const int first = m0 + half * (MT / 2) * 16, rows_left = min(8 * MT, a.M - first);
        if (8 * c < a.N) {
            with_type(a.y_dtype, [&](auto type) __attribute__((always_inline)) {
                for (int r = threadIdx.x / (C::BN / 8); r < rows_left; r += C::THREADS / (C::BN / 8)) {
                    int sum[8];
                    const intx4 *p = reinterpret_cast<const intx4 *>(lds + r * RS + (threadIdx.x % (C::BN / 8)) * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[e] = p[0][e];
                        sum[4 + e] = p[1][e];
                    }
                    finish8<decltype(type)>(a, first + r, c, a.x_scale[first + r], sum, cs, cb);
                }
            });
        }
    }
}

template <int BITS, int WN, int MT, int NT, int P>
pq_status launch_tile(const A8Args &a, hipStream_t s)
{
    using C = TileCfg<BITS, WN, MT, NT, P>;
    const int mtiles = (a.M + C::BM - 1) / C::BM, ntiles = (a.N + C::BN - 1) / C::BN;
    const int64_t blocks = static_cast<int64_t>(mtiles) * ntiles;
    if (blocks > kMaxBlocks) return PQ_ERR_SHAPE;
    hipLaunchKernelGGL((k_a8_tile<BITS, WN, MT, NT, P>), dim3(static_cast<unsigned>(blocks)), dim3(C::THREADS), 0, s, a, mtiles,
                       ntiles);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

template <int BITS>
pq_status launch_a8(const A8Args &a, hipStream_t s)
{
    const unsigned tiles = static_cast<unsigned>((a.N + 15) / 16);
    if (a.M <= 16) {
        hipLaunchKernelGGL((k_a8_stream<BITS, 1>), dim3(tiles), dim3(256), 0, s, a);
        return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
    }
    if (a.M >= 128) return launch_tile<BITS, 4, 8, 4, BITS == 4 ? 2 : 3>(a, s);
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
    if (!a8_shape_ok(mode, M, N, K) || x_stride < K || x_stride % 16 || x_stride > kMaxXStride) return PQ_ERR_SHAPE;
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
