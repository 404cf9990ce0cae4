// pq_distill.hip -- gfx950 kernels and C entry points of the distillation loss
// from a teacher's top logits, and its gradient.
//
// Per row: q = softmax(z / T) over the vocabulary, p = softmax(t / T) over the
// k entries of the teacher, loss = T^2 sum p (ln p - ln q), dz = T (q - p).
// Two exponentials and a handful of operations a word on 2 to 8 bytes of
// traffic: the memory system bounds it.  One block takes a row.  Each thread
// sums exp against the maximum of its own words and the (maximum, sum) pairs
// are joined once, so there is one reduction a row; rows of up to 131072 words
// of 16 bits (65536 of fp32) stay in registers between the sum and the
// gradient, longer ones are read a second time.
//
// p is 0 for all but k words.  The entries stand in LDS as chains hashed by
// chunks of eight words: a thread looks at one head per chunk and walks a
// chain where there is one, so that every word is written once and finished.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pq_row_common.hpp"

namespace pq {
namespace {

constexpr int kMaxTop = 1024;
constexpr int kHeads = 1024;            // heads of the chains

struct DistillArgs {
    const void *z, *top;
    void *dz;
    const int32_t *index;
    const float *row_weight, *dloss, *stats_in;
    float *loss, *stats;
    int64_t z_st, d_st;
    int rows, vocab, k, top_dtype, segment;
    float temp, inv_temp, c;            // c = log2(e) / T
    double grad;                        // grad_scale T
};

__device__ __forceinline__ float load_any(const void *a, int dtype, int64_t i)
{
    if (dtype == PQ_F32) return static_cast<const float *>(a)[i];
    if (dtype == PQ_BF16) return to_f32(static_cast<const bf16_t *>(a)[i]);
    return to_f32(static_cast<const f16_t *>(a)[i]);
}

__device__ __forceinline__ float wave_fmax(float x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}
__device__ __forceinline__ double wave_sum64(double x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// The teacher's entries of a row in LDS.
struct Entries {
    int32_t word[kMaxTop];              // -1: does not count
    float p[kMaxTop];                   // exp((t - max) / T), not yet divided by its sum
    int16_t next[kMaxTop];
    int head[kHeads];                   // first entry of a chain, -1
    float red[16];
    double red64[16];
};

template <int TEAM>
__device__ __forceinline__ float team_fmax(float x, Entries &l)
{
    x = wave_fmax(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) l.red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = l.red[0];
#pragma unroll
    for (int i = 1; i < TEAM / 64; ++i) x = fmaxf(x, l.red[i]);
    return x;
}
template <int TEAM>
__device__ __forceinline__ double team_sum64(double x, Entries &l)
{
    x = wave_sum64(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) l.red64[threadIdx.x >> 6] = x;
    __syncthreads();
    x = l.red64[0];
#pragma unroll
    for (int i = 1; i < TEAM / 64; ++i) x += l.red64[i];
    return x;
}

// Entries of row r to LDS: words and exp((t - max) / T); max and the sum of p
// come back, sum 0 where no entry counts.  A NaN among the counting logits
// makes the sum NaN.
template <int TEAM>
__device__ __forceinline__ void read_entries(const DistillArgs &a, int64_t r, Entries &l, float &top, double &total)
{
    float most = -INFINITY;
    for (int j = threadIdx.x; j < a.k; j += TEAM) {
        const int w = a.index[r * a.k + j];
        const bool counts = w >= 0 && w < a.vocab;
        const float t = counts ? load_any(a.top, a.top_dtype, r * a.k + j) : -INFINITY;
        l.word[j] = counts ? w : -1;
        l.p[j] = t;
        most = fmaxf(most, t);
    }
    top = team_fmax<TEAM>(most, l);
    const float ref = top == -INFINITY ? 0.f : top;
    double s = 0.0;
    for (int j = threadIdx.x; j < a.k; j += TEAM) {
        const float p = __builtin_amdgcn_exp2f((l.p[j] - ref) * a.c);
        l.p[j] = l.word[j] < 0 ? 0.f : p;
        s += l.p[j];
    }
    total = team_sum64<TEAM>(s, l);
}

// The chains: every word once, with the sum of its entries' p.
template <int TEAM>
__device__ __forceinline__ void chain_entries(const DistillArgs &a, Entries &l)
{
    for (int i = threadIdx.x; i < kHeads; i += TEAM) l.head[i] = -1;
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += TEAM) {
        const int w = l.word[j];
        if (w < 0) continue;
        bool first = true;
        for (int i = 0; i < j && first; ++i) first = l.word[i] != w;
        if (first) l.next[j] = static_cast<int16_t>(atomicExch(&l.head[(w >> 3) & (kHeads - 1)], j));
    }
    __syncthreads();
}

// Sum of p over the entries of a word, in the entries' order.
__device__ __forceinline__ float word_p(const DistillArgs &a, const Entries &l, int j)
{
    float p = l.p[j];
    for (int i = j + 1; i < a.k; ++i)
        if (l.word[i] == l.word[j]) p += l.p[i];
    return p;
}

// Gradient of eight words: g (q - p), q = exp((z - top) / T) inv.
template <typename T>
__device__ __forceinline__ void grad8(const DistillArgs &a, const Entries &l, T *dz, int c, const Raw8<T> &raw, float top,
                                      float gq, float gp)
{
    float x[8];
    raw_to_f32<T>(raw, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f((x[e] - top) * a.c) * gq;
    for (int j = l.head[c & (kHeads - 1)]; j >= 0; j = l.next[j]) {
        if (l.word[j] >> 3 != c) continue;
        const float p = gp * word_p(a, l, j);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] -= (l.word[j] & 7) == e ? p : 0.f;
    }
    store_row8<T>(dz, c, a.vocab, x);
}

template <typename T>
__device__ __forceinline__ void zero_row(T *dz, int vocab, int from, int to, int step)
{
    const float z[8] = {};
    for (int c = from; c < to; c += step) store_row8<T>(dz, c, vocab, z);
}

// Words past a row's end stand as -inf: no part of maximum and sum.
template <typename T>
__device__ __forceinline__ void words8(const Raw8<T> &raw, int c, int vocab, float (&x)[8])
{
    raw_to_f32<T>(raw, x);
    if (8 * c + 8 > vocab) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 8 * c + e < vocab ? x[e] : -INFINITY;
    }
}

// The compiler would keep a row's fp32 values from one use to the next, twice
// the registers of 16-bit words: it is told that they may have changed.
template <typename T>
__device__ __forceinline__ void as_read(Raw8<T> &raw)
{
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) asm volatile("" : "+v"(raw.w[i]));
}

// NV > 0: the row in registers, NV chunks a thread; NV = 0: read twice.
template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(TEAM) void k_distill(DistillArgs a)
{
    __shared__ Entries l;
    const int64_t r = blockIdx.x;
    const int tid = threadIdx.x, chunks = (a.vocab + 7) / 8;
    const T *z = static_cast<const T *>(a.z) + r * a.z_st;
    T *dz = a.dz ? static_cast<T *>(a.dz) + r * a.d_st : nullptr;
    const float weight = a.row_weight ? a.row_weight[r] : 1.f;
    Raw8<T> raw[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
        if (weight != 0.f) {
#pragma unroll
            for (int v = 0; v < NV; ++v) raw[v] = load_row8(z, min(tid + v * TEAM, chunks - 1), a.vocab);
        }
    }
    float t_top;
    double t_sum = 0.0;
    if (weight != 0.f) read_entries<TEAM>(a, r, l, t_top, t_sum);
    if (t_sum == 0.0) {                 // nothing to learn from: the same for the whole block
        if (tid == 0 && a.loss) a.loss[r] = 0.f;
        if (tid < 2 && a.stats) a.stats[2 * r + tid] = static_cast<float>(tid);
        if (dz) zero_row(dz, a.vocab, tid, chunks, TEAM);
        return;
    }
    // the entries' own logits, before any of them may be overwritten
    double dot = 0.0;
    for (int j = tid; j < a.k; j += TEAM) {
        const float p = l.p[j];
        if (p == 0.f) continue;
        // T ln(p / max p): the teacher's logit below its best, from p's own argument
        const float t = load_any(a.top, a.top_dtype, r * a.k + j) - t_top;
        dot += static_cast<double>(p) * (static_cast<double>(t) - static_cast<double>(to_f32(z[l.word[j]])));
    }
    float m = -INFINITY, s = 0.f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[8];
            words8<T>(raw[v], tid + v * TEAM, a.vocab, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, x[e]);
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[8];
            as_read(raw[v]);
            words8<T>(raw[v], tid + v * TEAM, a.vocab, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((x[e] - ref) * a.c);
        }
    } else {
        for (int c = tid; c < chunks; c += TEAM) {
            float x[8], more = m;
            words8<T>(load_row8(z, c, a.vocab), c, a.vocab, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) more = fmaxf(more, x[e]);
            const float ref = more == -INFINITY ? 0.f : more;
            s *= __builtin_amdgcn_exp2f((m - ref) * a.c);
            m = more;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((x[e] - ref) * a.c);
        }
    }
    const float top = team_fmax<TEAM>(m, l), ref = top == -INFINITY ? 0.f : top;
    const double sum = team_sum64<TEAM>(static_cast<double>(s * __builtin_amdgcn_exp2f((m - ref) * a.c)), l);
    dot = team_sum64<TEAM>(dot, l);
    if (tid == 0) {
        if (a.stats) {
            a.stats[2 * r] = top;
            a.stats[2 * r + 1] = static_cast<float>(sum);
        }
        if (a.loss) {
            const double kl = (dot / t_sum + static_cast<double>(top)) * a.inv_temp + log(sum) - log(t_sum);
            a.loss[r] = static_cast<float>(kl * weight * a.temp * a.temp);
        }
    }
    if (!dz) return;
    chain_entries<TEAM>(a, l);
    const double g = a.grad * weight;
    const float gq = static_cast<float>(g / sum), gp = static_cast<float>(g / t_sum);
    if constexpr (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            as_read(raw[v]);
            if (tid + v * TEAM < chunks) grad8<T>(a, l, dz, tid + v * TEAM, raw[v], top, gq, gp);
        }
    } else {
        for (int c = tid; c < chunks; c += TEAM) grad8<T>(a, l, dz, c, load_row8(z, c, a.vocab), top, gq, gp);
    }
}

// The gradient by itself: blocks of `segment` chunks of a row.
template <typename T>
__global__ __launch_bounds__(512) void k_distill_bwd(DistillArgs a)
{
    __shared__ Entries l;
    const int64_t r = blockIdx.x;
    const int chunks = (a.vocab + 7) / 8;
    const int from = static_cast<int>(blockIdx.y) * a.segment, to = min(from + a.segment, chunks);
    const T *z = static_cast<const T *>(a.z) + r * a.z_st;
    T *dz = static_cast<T *>(a.dz) + r * a.d_st;
    const float weight = a.row_weight ? a.row_weight[r] : 1.f;
    float t_top;
    double t_sum = 0.0;
    if (weight != 0.f) read_entries<512>(a, r, l, t_top, t_sum);
    if (t_sum == 0.0) {
        zero_row(dz, a.vocab, from + static_cast<int>(threadIdx.x), to, 512);
        return;
    }
    chain_entries<512>(a, l);
    const double g = a.grad * weight * a.dloss[r];
    const float top = a.stats_in[2 * r];
    const float gq = static_cast<float>(g / a.stats_in[2 * r + 1]), gp = static_cast<float>(g / t_sum);
    for (int c = from + static_cast<int>(threadIdx.x); c < to; c += 512)
        grad8<T>(a, l, dz, c, load_row8(z, c, a.vocab), top, gq, gp);
}

template <typename T>
pq_status launch_distill(const DistillArgs &a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.rows));
    constexpr int WORDS = sizeof(T) == 4 ? 8 : 16;      // most chunks a thread keeps
    if (a.vocab <= 256 * 8 * 4) hipLaunchKernelGGL((k_distill<T, 256, 4>), grid, dim3(256), 0, s, a);
    else if (a.vocab <= 512 * 8 * 8) hipLaunchKernelGGL((k_distill<T, 512, 8>), grid, dim3(512), 0, s, a);
    else if (a.vocab <= 1024 * 8 * 8) hipLaunchKernelGGL((k_distill<T, 1024, 8>), grid, dim3(1024), 0, s, a);
    else if (WORDS > 8 && a.vocab <= 1024 * 8 * WORDS)
        hipLaunchKernelGGL((k_distill<T, 1024, WORDS>), grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((k_distill<T, 1024, 0>), grid, dim3(1024), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

inline bool misaligned(const void *p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

// What both entry points check, and the arguments that they share.
inline pq_status distill_args(DistillArgs &a, int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t l_stride,
                              int64_t k, const int32_t *index, const void *top, int top_dtype, double temperature,
                              const float *row_weight, void *dlogits, int64_t d_stride)
{
    const int size = dtype_bytes(dtype), tsize = dtype_bytes(top_dtype);
    if (!size || !tsize) return PQ_ERR_MODE;
    if (rows < 0 || rows > INT32_MAX || vocab < 1 || vocab > (int64_t(1) << 30) || k < 1 || k > kMaxTop) return PQ_ERR_SHAPE;
    const float temp = static_cast<float>(temperature), inv = static_cast<float>(1.0 / temperature);
    if (!(temperature > 0.0) || !(temp > 0.f) || !(inv > 0.f) || !std::isfinite(temp) || !std::isfinite(inv))
        return PQ_ERR_ARG;
    if (rows == 0) return PQ_OK;
    if (!logits || !index || !top) return PQ_ERR_NULL;
    if (misaligned(logits, size) || misaligned(dlogits, size) || misaligned(index, 4) || misaligned(top, tsize) ||
        misaligned(row_weight, 4))
        return PQ_ERR_ALIGN;
    if (dlogits == logits && d_stride != l_stride) return PQ_ERR_ARG;
    a.z = logits;
    a.top = top;
    a.dz = dlogits;
    a.index = index;
    a.row_weight = row_weight;
    a.z_st = l_stride;
    a.d_st = d_stride;
    a.rows = static_cast<int>(rows);
    a.vocab = static_cast<int>(vocab);
    a.k = static_cast<int>(k);
    a.top_dtype = top_dtype;
    a.temp = temp;
    a.inv_temp = inv;
    a.c = static_cast<float>(1.4426950408889634074 / temperature);
    return PQ_OK;
}

}  // namespace
}  // namespace pq

extern "C" {

pq_status pq_distill(int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t l_stride, int64_t k,
                     const int32_t *index, const void *top, int top_dtype, double temperature,
                     const float *row_weight, float *loss, float *stats, double grad_scale, void *dlogits,
                     int64_t d_stride, void *stream)
{
    using namespace pq;
    DistillArgs a = {};
    const pq_status rc = distill_args(a, dtype, rows, vocab, logits, l_stride, k, index, top, top_dtype, temperature,
                                      row_weight, dlogits, d_stride);
    if (rc != PQ_OK) return rc;
    if (!std::isfinite(grad_scale)) return PQ_ERR_ARG;
    if (rows == 0) return PQ_OK;
    if (!loss && !stats && !dlogits) return PQ_ERR_NULL;
    if (misaligned(loss, 4) || misaligned(stats, 4)) return PQ_ERR_ALIGN;
    a.loss = loss;
    a.stats = stats;
    a.grad = grad_scale * temperature;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == PQ_F32    ? launch_distill<float>(a, s)
           : dtype == PQ_BF16 ? launch_distill<bf16_t>(a, s)
                              : launch_distill<f16_t>(a, s);
}

pq_status pq_distill_bwd(int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t l_stride, int64_t k,
                         const int32_t *index, const void *top, int top_dtype, double temperature,
                         const float *row_weight, const float *stats, const float *dloss, void *dlogits,
                         int64_t d_stride, void *stream)
{
    using namespace pq;
    DistillArgs a = {};
    const pq_status rc = distill_args(a, dtype, rows, vocab, logits, l_stride, k, index, top, top_dtype, temperature,
                                      row_weight, dlogits, d_stride);
    if (rc != PQ_OK) return rc;
    if (rows == 0) return PQ_OK;
    if (!stats || !dloss || !dlogits) return PQ_ERR_NULL;
    if (misaligned(stats, 4) || misaligned(dloss, 4)) return PQ_ERR_ALIGN;
    a.stats_in = stats;
    a.dloss = dloss;
    a.grad = temperature;
    const int64_t chunks = (vocab + 7) / 8;
    // up to 65535 blocks a row, of 4096 words and more
    int64_t segments = (chunks + 4095) / 4096;
    if (segments > 65535) segments = 65535;
    a.segment = static_cast<int>((chunks + segments - 1) / segments);
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(segments));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == PQ_F32) hipLaunchKernelGGL(k_distill_bwd<float>, grid, dim3(512), 0, s, a);
    else if (dtype == PQ_BF16) hipLaunchKernelGGL(k_distill_bwd<bf16_t>, grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL(k_distill_bwd<f16_t>, grid, dim3(512), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

}  // extern "C"
