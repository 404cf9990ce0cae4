// pq_norm.hip -- gfx950 kernels and C entry points of the root-mean-square
// norm (with the residual's addition and an output in 8 bits), its gradient,
// and of rows in 8 bits by themselves.
//
// A few operations an element on 2 to 12 bytes of traffic: the memory system
// bounds all of them, so every array is read once and a row stays in registers
// from its loads to its stores.  A team of 64 (four rows a block), 256 or 1024
// threads holds a row, eight consecutive elements a thread and chunk.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pq_row_common.hpp"

namespace pq {
namespace {

constexpr int64_t kMaxNormCols = 32768, kMaxRowCols = 65536;

struct NormArgs {
    const void *x, *residual, *weight;
    void *sum, *y;
    int8_t *q;
    float *scale, *rstd;
    int64_t x_st, r_st, s_st, y_st, q_st;   // elements
    int64_t rows;
    int cols, w_dtype;
    float eps;
};

// Sum or maximum of a team of TEAM threads, the same in all of them.  `lds` has
// a place per wave; a caller that uses it again lets the block meet in between.
template <int TEAM, typename V, typename F>
__device__ __forceinline__ V team_join(V mine, V *lds, F &&join)
{
    if constexpr (TEAM > 64) {
        constexpr int W = TEAM / 64;
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = mine;
        __syncthreads();
        mine = lds[0];
#pragma unroll
        for (int i = 1; i < W; ++i) mine = join(mine, lds[i]);
    }
    return mine;
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float s, float *lds)
{
    return team_join<TEAM>(wave_sum(s), lds, [](float a, float b) { return a + b; });
}
template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t m, uint32_t *lds)
{
    return team_join<TEAM>(wave_max(m), lds, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Eight codes from t c: adding 1.5 2^23 rounds to a whole number (to even) and
// leaves it, in two's complement, in the low byte.
__device__ __forceinline__ u32x2 codes8(const float (&t)[8], float c)
{
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __builtin_bit_cast(uint32_t, t[4 * h + e] * c + 12582912.f);
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0c);
        w[h] = lo | hi;
    }
    return w;
}

// One row per team.  NORM: h, rstd and the weight; otherwise the row as it is.
template <typename T, int TEAM, int NV, bool NORM, bool EIGHT>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm(NormArgs a)
{
    __shared__ float sums[TEAM / 64];
    __shared__ uint32_t tops[TEAM / 64];
    const int tid = TEAM == 64 ? threadIdx.x & 63 : threadIdx.x;
    int64_t row = blockIdx.x;
    if constexpr (TEAM == 64) {
        row = row * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        if (row >= a.rows) return;
    }
    const int cols = a.cols;
    const T *x = static_cast<const T *>(a.x) + row * a.x_st;
    Raw8<T> raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v] = load_row8(x, tid + v * TEAM, cols);
    float t[NV][8], w[NORM ? NV : 1][8];
    if (NORM && a.residual) {
        const T *r = static_cast<const T *>(a.residual) + row * a.r_st;
        T *s = static_cast<T *>(a.sum) + row * a.s_st;
        Raw8<T> more[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) more[v] = load_row8(r, tid + v * TEAM, cols);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float p[8];
            raw_to_f32<T>(raw[v], t[v]);
            raw_to_f32<T>(more[v], p);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[v][e] = to_f32(from_f32<T>(t[v][e] + p[e]));   // h is what is stored
            store_row8<T>(s, tid + v * TEAM, cols, t[v]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) raw_to_f32<T>(raw[v], t[v]);
    }
    if constexpr (NORM) {
#pragma unroll
        for (int v = 0; v < NV; ++v) load_any8(a.weight, a.w_dtype, tid + v * TEAM, cols, w[v]);
    }
    if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(t[v][e], t[v][e], ss);
        ss = team_sum<TEAM>(ss, sums);
        const float rstd = 1.f / __builtin_sqrtf(ss / static_cast<float>(cols) + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) t[v][e] = t[v][e] * rstd * w[v][e];
    }
    if constexpr (!EIGHT) {
        T *y = static_cast<T *>(a.y) + row * a.y_st;
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row8<T>(y, tid + v * TEAM, cols, t[v]);
        return;
    }
    // The scale and the codes are those of y itself, which costs a second
    // reduction.  One for both, of |h weight| with rstd behind it, would take
    // other codes between two of them and overflow where y does not (16384 x 4096
    // in bf16 81.9 us with either, 16384 x 576 16.4 against 15.8).
    uint32_t top = 0;                       // the largest |y|, as its bits: NaN above infinity above all others
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, t[v][e]) & 0x7fffffffu);
    top = team_max<TEAM>(top, tops);
    float scale = fmaxf(__builtin_bit_cast(float, top) * (1.f / 127.f), kMinKvScale);
    if (top >= 0x7f800000u) scale = __builtin_nanf("");
    if (tid == 0) a.scale[row] = scale;
    const float c = 1.f / scale;
    int8_t *q = a.q + row * a.q_st;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int at = tid + v * TEAM;
        const u32x2 w8 = codes8(t[v], c);
        if (8 * at + 8 <= cols) {
            *reinterpret_cast<u32x2_a1 *>(q + 8 * at) = w8;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * at + e < cols) q[8 * at + e] = static_cast<int8_t>(w8[e >> 2] >> (8 * (e & 3)));
        }
    }
}

struct NormBwdArgs {
    const void *h, *weight, *dy, *dsum;
    void *dx;
    const float *rstd;
    float *partial;                         // [blocks, cols], or nullptr: no dweight
    int64_t h_st, dy_st, ds_st, dx_st;
    int64_t rows;
    int cols, w_dtype;
};

// Rows blockIdx, blockIdx + gridDim, ... of a team; the weight's gradient is
// summed in registers over them and left as one row of partial sums a team.
template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm_bwd(NormBwdArgs a)
{
    __shared__ float lds[TEAM / 64];
    const int tid = TEAM == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t teams = static_cast<int64_t>(gridDim.x) * (TEAM == 64 ? 4 : 1);
    int64_t team = blockIdx.x;
    if constexpr (TEAM == 64) team = team * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int cols = a.cols;
    const float inv = 1.f / static_cast<float>(cols);
    // A block of 1024 threads has 128 registers a thread (with four chunks too few:
    // 37 are spilled, 90 in fp32; 2048 x 32768 174 us, in fp32 341): the weight is read
    // again for every row there (from the caches), dsum after the row's sum.
    constexpr bool WIDE = TEAM == 1024;
    float w[WIDE ? 1 : NV][8], dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if constexpr (!WIDE) load_any8(a.weight, a.w_dtype, tid + v * TEAM, cols, w[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
    }
    for (int64_t row = team; row < a.rows; row += teams) {
        const T *h = static_cast<const T *>(a.h) + row * a.h_st, *dy = static_cast<const T *>(a.dy) + row * a.dy_st;
        Raw8<T> rh[NV], rd[NV], rs[WIDE ? 1 : NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            rh[v] = load_row8(h, tid + v * TEAM, cols);
            rd[v] = load_row8(dy, tid + v * TEAM, cols);
        }
        const T *ds = a.dsum ? static_cast<const T *>(a.dsum) + row * a.ds_st : nullptr;
        if (!WIDE && ds) {
#pragma unroll
            for (int v = 0; v < NV; ++v) rs[WIDE ? 0 : v] = load_row8(ds, tid + v * TEAM, cols);
        }
        const float rstd = a.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float n[8], g[8];
            if constexpr (WIDE) {
                __builtin_amdgcn_sched_barrier(0);
                as_read(rh[v]);
                as_read(rd[v]);
            }
            raw_to_f32<T>(rh[v], n);
            raw_to_f32<T>(rd[v], g);
            if constexpr (WIDE) load_any8(a.weight, a.w_dtype, tid + v * TEAM, cols, w[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = g[e] * (n[e] * rstd);
                dw[v][e] += p;
                dot = __builtin_fmaf(p, w[WIDE ? 0 : v][e], dot);
            }
        }
        if constexpr (TEAM > 64) __syncthreads();       // the last row's sums have been read
        const float c = team_sum<TEAM>(dot, lds) * inv;
        T *dx = static_cast<T *>(a.dx) + row * a.dx_st;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float n[8], g[8], s[8] = {};
            if constexpr (WIDE) {
                __builtin_amdgcn_sched_barrier(0);
                as_read(rh[v]);
                as_read(rd[v]);
            }
            raw_to_f32<T>(rh[v], n);
            raw_to_f32<T>(rd[v], g);
            if constexpr (WIDE) load_any8(a.weight, a.w_dtype, tid + v * TEAM, cols, w[0]);
            if (ds) raw_to_f32<T>(WIDE ? load_row8(ds, tid + v * TEAM, cols) : rs[WIDE ? 0 : v], s);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(rstd, g[e] * w[WIDE ? 0 : v][e] - n[e] * rstd * c, s[e]);
            store_row8<T>(dx, tid + v * TEAM, cols, s);
        }
    }
    if (!a.partial) return;
    if constexpr (TEAM == 64) {             // the four waves of a block share a row of partial sums
        __shared__ float rows[4][64 * NV * 8];
        float *mine = rows[threadIdx.x >> 6];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) mine[(tid + v * 64) * 8 + e] = dw[v][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += 256)
            a.partial[static_cast<int64_t>(blockIdx.x) * cols + c] = (rows[0][c] + rows[1][c]) + (rows[2][c] + rows[3][c]);
    } else {
        float *out = a.partial + team * cols;
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row8<float>(out, tid + v * TEAM, cols, dw[v]);
    }
}

// dweight: the partial rows added up, 16 columns a block, 64 strided sums side
// by side, each with eight loads in flight, joined in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_dweight(const float *partial, int64_t parts, int cols, float *dweight)
{
    __shared__ float lds[64][17];
    const int lane = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + lane;
    float s = 0.f;
    if (c < cols)
        for (int64_t p0 = g; p0 < parts; p0 += 64 * 8) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = p0 + 64 * u < parts ? partial[(p0 + 64 * u) * cols + c] : 0.f;
            s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        }
    lds[g][lane] = s;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    // one wave: 4 partial sums of 16 each a column, then two steps over the lanes
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[16 * g + i][lane];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (g == 0 && c < cols) dweight[c] = s;
}

// Team and chunks of a row: one wave up to 1024 columns, then 256 threads up
// to 8192, then 1024.
inline int team_of(int64_t cols) { return cols <= 1024 ? 64 : cols <= 8192 ? 256 : 1024; }

template <typename F>
pq_status with_shape(int64_t cols, F &&f)
{
    using std::integral_constant;
#define PQ_TEAM_CASE(TEAM, NV) \
    if (cols <= TEAM * NV * 8) return f(integral_constant<int, TEAM>{}, integral_constant<int, NV>{});
    PQ_TEAM_CASE(64, 1)
    PQ_TEAM_CASE(64, 2)
    PQ_TEAM_CASE(256, 1)
    PQ_TEAM_CASE(256, 2)
    PQ_TEAM_CASE(256, 3)
    PQ_TEAM_CASE(256, 4)
    PQ_TEAM_CASE(1024, 2)
    PQ_TEAM_CASE(1024, 4)
    PQ_TEAM_CASE(1024, 8)
#undef PQ_TEAM_CASE
    return PQ_ERR_SHAPE;
}

inline unsigned team_blocks(int64_t rows, int team) { return static_cast<unsigned>(team == 64 ? (rows + 3) / 4 : rows); }

template <typename T, bool NORM>
pq_status launch_rows(const NormArgs &a, hipStream_t s)
{
    return with_shape(a.cols, [&](auto team, auto nv) {
        constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
        if constexpr (!NORM || TEAM * NV * 8 <= kMaxNormCols) {
            const dim3 grid(team_blocks(a.rows, TEAM)), block(TEAM < 256 ? 256 : TEAM);
            if constexpr (NORM) {
                if (!a.q) {
                    hipLaunchKernelGGL((k_norm<T, TEAM, NV, NORM, false>), grid, block, 0, s, a);
                    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
                }
            }
            hipLaunchKernelGGL((k_norm<T, TEAM, NV, NORM, true>), grid, block, 0, s, a);
            return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
        } else {
            return PQ_ERR_SHAPE;
        }
    });
}

template <typename T, bool NORM>
pq_status launch_norm(NormArgs a, hipStream_t s)
{
    for (int64_t left = a.rows; left > 0; left -= kLaunchRows) {
        a.rows = left < kLaunchRows ? left : kLaunchRows;
        const pq_status rc = launch_rows<T, NORM>(a, s);
        if (rc != PQ_OK) return rc;
        skip_rows(a.x, a.rows, a.x_st, sizeof(T));
        skip_rows(a.residual, a.rows, a.r_st, sizeof(T));
        skip_rows(a.sum, a.rows, a.s_st, sizeof(T));
        skip_rows(a.y, a.rows, a.y_st, sizeof(T));
        skip_rows(a.q, a.rows, a.q_st, 1);
        skip_rows(a.scale, a.rows, 1, 4);
        skip_rows(a.rstd, a.rows, 1, 4);
    }
    return PQ_OK;
}

// Blocks of the gradient, each with a row of partial sums: two of 256 threads a
// CU and four of waves that take a row each (16384 x 4096 in bf16 with 256, 512,
// 768, 1024 blocks 116, 103, 107, 111 us; 65536 x 576 with 512, 1024, 1792,
// 2048 99, 68, 76, 71), one of 1024 threads (2048 x 16384 with 128, 256, 512 blocks
// 94, 69, 76; 2048 x 32768 245, 174, 201).
inline int64_t bwd_blocks(int64_t rows, int64_t cols)
{
    const int team = team_of(cols);
    const int64_t need = team == 64 ? (rows + 3) / 4 : rows, most = team == 64 ? 1024 : team == 256 ? 512 : 256;
    return need < most ? need : most;
}

template <typename T>
pq_status launch_norm_bwd(const NormBwdArgs &a, hipStream_t s)
{
    return with_shape(a.cols, [&](auto team, auto nv) {
        constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
        if constexpr (TEAM * NV * 8 <= kMaxNormCols) {
            hipLaunchKernelGGL((k_norm_bwd<T, TEAM, NV>), dim3(static_cast<unsigned>(bwd_blocks(a.rows, a.cols))),
                               dim3(TEAM < 256 ? 256 : TEAM), 0, s, a);
            return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
        } else {
            return PQ_ERR_SHAPE;
        }
    });
}

inline bool misaligned(const void *p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

}  // namespace
}  // namespace pq

extern "C" {

pq_status pq_rmsnorm(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, const void *residual,
                     int64_t r_stride, void *sum, int64_t s_stride, const void *weight, int w_dtype, double eps,
                     void *y, int64_t y_stride, int8_t *q, int64_t q_stride, float *scale, float *rstd, void *stream)
{
    using namespace pq;
    const int size = dtype_bytes(dtype), wsize = dtype_bytes(w_dtype);
    if (!size || !wsize) return PQ_ERR_MODE;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxNormCols) return PQ_ERR_SHAPE;
    if (!(eps > 0.0) || !std::isfinite(static_cast<float>(eps)) || !(static_cast<float>(eps) > 0.f)) return PQ_ERR_ARG;
    if (rows == 0) return PQ_OK;
    if (!x || !weight || (residual && !sum) || (q && !scale)) return PQ_ERR_NULL;
    if ((sum && !residual) || !y == !q) return PQ_ERR_ARG;
    if (misaligned(x, size) || misaligned(residual, size) || misaligned(sum, size) || misaligned(y, size) ||
        misaligned(weight, wsize) || misaligned(scale, 4) || misaligned(rstd, 4))
        return PQ_ERR_ALIGN;
    if ((sum == x && s_stride != x_stride) || (sum && sum == residual && s_stride != r_stride) ||
        (y && y == x && y_stride != x_stride) || (y && y == sum))
        return PQ_ERR_ARG;
    if ((sum && rows_overlap(rows, cols, s_stride)) || rows_overlap(rows, cols, y ? y_stride : q_stride)) return PQ_ERR_SHAPE;
    NormArgs a = {};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum = sum;
    a.y = y;
    a.q = q;
    a.scale = scale;
    a.rstd = rstd;
    a.x_st = x_stride;
    a.r_st = r_stride;
    a.s_st = s_stride;
    a.y_st = y_stride;
    a.q_st = q_stride;
    a.rows = rows;
    a.cols = static_cast<int>(cols);
    a.w_dtype = w_dtype;
    a.eps = static_cast<float>(eps);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == PQ_F32    ? launch_norm<float, true>(a, s)
           : dtype == PQ_BF16 ? launch_norm<bf16_t, true>(a, s)
                              : launch_norm<f16_t, true>(a, s);
}

int64_t pq_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    using namespace pq;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxNormCols) return -1;
    return (bwd_blocks(rows, cols) * cols * 4 + 15) / 16 * 16;
}

pq_status pq_rmsnorm_bwd(int dtype, int64_t rows, int64_t cols, const void *h, int64_t h_stride, const void *weight,
                         int w_dtype, const float *rstd, const void *dy, int64_t dy_stride, const void *dsum,
                         int64_t ds_stride, void *dx, int64_t dx_stride, float *dweight, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    using namespace pq;
    const int size = dtype_bytes(dtype), wsize = dtype_bytes(w_dtype);
    if (!size || !wsize) return PQ_ERR_MODE;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxNormCols) return PQ_ERR_SHAPE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows == 0 && !dweight) return PQ_OK;
    if (rows > 0 && (!h || !weight || !rstd || !dy || !dx || (dweight && !workspace))) return PQ_ERR_NULL;
    if (misaligned(h, size) || misaligned(dy, size) || misaligned(dsum, size) || misaligned(dx, size) ||
        misaligned(weight, wsize) || misaligned(rstd, 4) || misaligned(dweight, 4) || !aligned16(workspace))
        return PQ_ERR_ALIGN;
    if (dweight && workspace_bytes < pq_rmsnorm_bwd_workspace_bytes(rows, cols)) return PQ_ERR_ARG;
    if (rows > 0 && ((dx == dy && dx_stride != dy_stride) || (dx == dsum && dx_stride != ds_stride) || dx == h))
        return PQ_ERR_ARG;
    if (rows_overlap(rows, cols, dx_stride)) return PQ_ERR_SHAPE;
    if (rows > 0) {
        NormBwdArgs a = {};
        a.h = h;
        a.weight = weight;
        a.dy = dy;
        a.dsum = dsum;
        a.dx = dx;
        a.rstd = rstd;
        a.partial = dweight ? static_cast<float *>(workspace) : nullptr;
        a.h_st = h_stride;
        a.dy_st = dy_stride;
        a.ds_st = ds_stride;
        a.dx_st = dx_stride;
        a.rows = rows;
        a.cols = static_cast<int>(cols);
        a.w_dtype = w_dtype;
        const pq_status rc = dtype == PQ_F32    ? launch_norm_bwd<float>(a, s)
                             : dtype == PQ_BF16 ? launch_norm_bwd<bf16_t>(a, s)
                                                : launch_norm_bwd<f16_t>(a, s);
        if (rc != PQ_OK) return rc;
    }
    if (dweight) {
        hipLaunchKernelGGL(k_norm_dweight, dim3(static_cast<unsigned>((cols + 15) / 16)), dim3(1024), 0, s,
                           static_cast<const float *>(workspace), bwd_blocks(rows, cols), static_cast<int>(cols), dweight);
        if (hipGetLastError() != hipSuccess) return PQ_ERR_HIP;
    }
    return PQ_OK;
}

pq_status pq_quantize_rows(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, int8_t *q,
                           int64_t q_stride, float *scale, void *stream)
{
    using namespace pq;
    const int size = dtype_bytes(dtype);
    if (!size) return PQ_ERR_MODE;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kMaxRowCols) return PQ_ERR_SHAPE;
    if (rows == 0) return PQ_OK;
    if (!x || !q || !scale) return PQ_ERR_NULL;
    if (misaligned(x, size) || misaligned(scale, 4)) return PQ_ERR_ALIGN;
    if (rows_overlap(rows, cols, q_stride)) return PQ_ERR_SHAPE;
    NormArgs a = {};
    a.x = x;
    a.q = q;
    a.scale = scale;
    a.x_st = x_stride;
    a.q_st = q_stride;
    a.rows = rows;
    a.cols = static_cast<int>(cols);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == PQ_F32    ? launch_norm<float, false>(a, s)
           : dtype == PQ_BF16 ? launch_norm<bf16_t, false>(a, s)
                              : launch_norm<f16_t, false>(a, s);
}

}  // extern "C"
