// pq_distill.hip -- gfx950 kernels and C entry points of the distillation loss
// from a teacher's top logits, and its gradient.
//
// Per row: q = softmax(z / T) over the vocabulary, p = softmax(t / T) over the
// k entries of the teacher, loss = T^2 sum p (ln p - ln q) over the entries, dz =
// T (q - P) with P the entries' p summed by word.
// Two exponentials and a handful of operations a word on 2 to 8 bytes of
// traffic: the memory system bounds it.  One block takes a row.  Each thread
// sums exp against the maximum of its own words and the (maximum, sum) pairs
// are joined once, so there is one reduction a row; rows of up to 131072 words
// of 16 bits (65536 of fp32) stay in registers between the sum and the
// gradient, what longer ones have more is read a second time (1024 rows of 128256
// words in fp32 242 us; 288 with nearly all of it read twice).  One wave reads the
// teacher's list while the others read the row.
// 2048 rows of 128256 words in bf16 take 210 us, 5.0 TB/s, the rate of a copy; the
// loss by itself 112, the gradient 206.
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
constexpr int U = 4;                    // chunks in flight a thread, where a row is not kept

struct DistillArgs {
    const void *z, *top;
    void *dz;
    const int32_t *index;
    const float *row_weight, *dloss, *stats_in;
    float *loss, *stats;
    int64_t z_st, d_st;
    int rows, vocab, k, top_dtype, segment;
    int nt;                             // the gradient is not written into the caches
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

// The teacher's entries of a row in LDS, and what the waves of a block tell
// each other.
struct Entries {
    int32_t word[kMaxTop];              // -1: does not count
    float p[kMaxTop];                   // exp((t - max) / T), not yet divided by its sum
    float all[kMaxTop];                 // a word's p: its first entry's, 0 in the word's others
    int16_t next[kMaxTop];
    int32_t head[kHeads];               // first entry of a chain, -1
    double total, dot;                  // sum of p; sum of p (t - max - z)
    float most[16], sum[16];            // of the waves' words
};

// Between accesses of one wave's lanes to what its other lanes wrote.
__device__ __forceinline__ void lanes_agree() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// One wave's work, while the others read the row: the entries of row r, their
// sum (0 where none counts or all are -inf, NaN where one is NaN), the loss's
// sum with the entries' own logits and, for a gradient, the chains.
template <typename T>
__device__ __forceinline__ void read_entries(const DistillArgs &a, int64_t r, const T *z, bool loss, bool chains, Entries &l)
{
    const int lane = threadIdx.x & 63;
    float most = -INFINITY;
    for (int j = lane; j < a.k; j += 64) {
        const int w = a.index[r * a.k + j];
        const float t = load_any(a.top, a.top_dtype, r * a.k + j);
        const bool counts = w >= 0 && w < a.vocab;
        l.word[j] = counts ? w : -1;
        l.p[j] = t;
        if (counts) most = fmaxf(most, t);
    }
    if (chains)
        for (int i = lane; i < kHeads; i += 64) l.head[i] = -1;
    const float top = wave_fmax(most), ref = top == -INFINITY ? 0.f : top;
    lanes_agree();
    double total = 0.0, dot = 0.0;
    for (int j = lane; j < a.k; j += 64) {
        const int w = l.word[j];
        const float t = l.p[j], p = w < 0 ? 0.f : __builtin_amdgcn_exp2f((t - ref) * a.c);
        l.p[j] = p;
        total += p;
        if (loss && p != 0.f) dot += static_cast<double>(p) * (static_cast<double>(t) - ref - static_cast<double>(to_f32(z[w])));
        // p = 0 needs no place in a chain: lists filled up with one word stay short
        if (chains && p != 0.f) l.next[j] = static_cast<int16_t>(atomicExch(&l.head[(w >> 3) & (kHeads - 1)], j));
    }
    total = wave_sum64(total);
    dot = wave_sum64(dot);
    if (lane == 0) {
        l.total = total;
        l.dot = dot;
    }
    if (!chains) return;
    lanes_agree();
    // A word that is named more than once: its first entry takes the sum.  It
    // is one of whole numbers (of 2^-50 of the word's largest p), so that the
    // chain's order, which is chance, does not show.
    for (int j = lane; j < a.k; j += 64) {
        float p = l.p[j];
        if (p == 0.f) continue;
        const int w = l.word[j];
        bool first = true, more = false;
        float most = p;
        for (int i = l.head[(w >> 3) & (kHeads - 1)]; i >= 0; i = l.next[i]) {
            if (l.word[i] != w) continue;
            first = first && i >= j;
            more = more || i != j;
            most = fmaxf(most, l.p[i]);
        }
        if (more && first) {
            const int e = __builtin_amdgcn_frexp_expf(most);        // most < 2^e: 1024 terms stay below 2^60
            uint64_t sum = 0;
            for (int i = l.head[(w >> 3) & (kHeads - 1)]; i >= 0; i = l.next[i])
                if (l.word[i] == w) sum += static_cast<uint64_t>(ldexp(static_cast<double>(l.p[i]), 50 - e));
            p = static_cast<float>(ldexp(static_cast<double>(sum), e - 50));
        }
        l.all[j] = first ? p : 0.f;
    }
}

// Gradient of the eight words of chunk c: g (q - p), q = exp((z - top) / T) / sum.
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
        const float p = gp * l.all[j];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] -= (l.word[j] & 7) == e ? p : 0.f;
    }
    if (a.nt) store_whole8<true>(dz + 8 * static_cast<int64_t>(c), x);
    else store_whole8(dz + 8 * static_cast<int64_t>(c), x);
}

// Gradient of one word, of those behind the last whole chunk.
template <typename T>
__device__ __forceinline__ void grad1(const DistillArgs &a, const Entries &l, T *dz, int w, float z, float top, float gq, float gp)
{
    float x = __builtin_amdgcn_exp2f((z - top) * a.c) * gq;
    for (int j = l.head[(w >> 3) & (kHeads - 1)]; j >= 0; j = l.next[j])
        if (l.word[j] == w) x -= gp * l.all[j];
    dz[w] = from_f32<T>(x);
}

// Words 8 from .. of a row to 0, and those behind the last whole chunk where
// `rest` is theirs.
template <typename T>
__device__ __forceinline__ void zero_words(T *dz, int from, int to, int step, int rest, int vocab)
{
    const float z[8] = {};
    for (int c = from; c < to; c += step) store_whole8(dz + 8 * static_cast<int64_t>(c), z);
    if (rest >= 0 && rest < vocab) dz[rest] = from_f32<T>(0.f);
}

// NV chunks a thread in registers; the words behind the last whole chunk go to
// the first threads, one each.
template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(TEAM) void k_distill(DistillArgs a)
{
    __shared__ Entries l;
    const int64_t r = blockIdx.x;
    const int tid = threadIdx.x, chunks = a.vocab / 8, rest = 8 * chunks + tid;
    const T *z = static_cast<const T *>(a.z) + r * a.z_st;
    T *dz = a.dz ? static_cast<T *>(a.dz) + r * a.d_st : nullptr;
    const float weight = a.row_weight ? a.row_weight[r] : 1.f;
    Raw8<T> raw[NV];
    float z_rest = -INFINITY;
    if (weight != 0.f) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (tid + v * TEAM < chunks) raw[v] = load_whole8(z + 8 * static_cast<int64_t>(tid + v * TEAM));
        if (rest < a.vocab) z_rest = to_f32(z[rest]);
    }
    if (tid < 64 && weight != 0.f) read_entries<T>(a, r, z, a.loss != nullptr, dz != nullptr, l);
    float m = z_rest, s = 0.f;
    if (weight != 0.f) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            __builtin_amdgcn_sched_barrier(0);
            if (tid + v * TEAM >= chunks) continue;
            float x[8];
            as_read(raw[v]);
            raw_to_f32<T>(raw[v], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, x[e]);
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            __builtin_amdgcn_sched_barrier(0);
            if (tid + v * TEAM >= chunks) continue;
            float x[8];
            as_read(raw[v]);
            raw_to_f32<T>(raw[v], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((x[e] - ref) * a.c);
        }
        s += __builtin_amdgcn_exp2f((z_rest - ref) * a.c);
        // what the registers do not hold
        for (int c = tid + NV * TEAM; c < chunks; c += U * TEAM) {
            Raw8<T> q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = load_whole8(z + 8 * static_cast<int64_t>(min(c + u * TEAM, chunks - 1)));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * TEAM >= chunks) break;
                float x[8], more = m;
                raw_to_f32<T>(q[u], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) more = fmaxf(more, x[e]);
                const float ref = more == -INFINITY ? 0.f : more;
                s *= __builtin_amdgcn_exp2f((m - ref) * a.c);
                m = more;
#pragma unroll
                for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((x[e] - ref) * a.c);
            }
        }
    }
    // the pairs (maximum, sum) of the lanes, then of the waves
    float top = wave_fmax(m), ref = top == -INFINITY ? 0.f : top;
    s = wave_sum(s * __builtin_amdgcn_exp2f((m - ref) * a.c));
    if ((tid & 63) == 0) {
        l.most[tid >> 6] = top;
        l.sum[tid >> 6] = s;
    }
    __syncthreads();
    const double t_sum = weight != 0.f ? l.total : 0.0;
    if (t_sum == 0.0) {                 // nothing to learn from: the same for the whole block
        if (tid == 0 && a.loss) a.loss[r] = 0.f;
        if (tid < 2 && a.stats) a.stats[2 * r + tid] = static_cast<float>(tid);
        if (dz) zero_words(dz, tid, chunks, TEAM, rest, a.vocab);
        return;
    }
    top = l.most[0];
#pragma unroll
    for (int i = 1; i < TEAM / 64; ++i) top = fmaxf(top, l.most[i]);
    ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < TEAM / 64; ++i) sum += l.sum[i] * __builtin_amdgcn_exp2f((l.most[i] - ref) * a.c);
    if (tid == 0) {
        if (a.stats) {
            a.stats[2 * r] = top;
            a.stats[2 * r + 1] = sum;
        }
        if (a.loss) {
            const double kl = (l.dot / t_sum + static_cast<double>(top)) * a.inv_temp + log(static_cast<double>(sum)) - log(t_sum);
            a.loss[r] = static_cast<float>(kl * weight * a.temp * a.temp);
        }
    }
    if (!dz) return;
    const double g = a.grad * weight;
    const float gq = static_cast<float>(g / static_cast<double>(sum)), gp = static_cast<float>(g / t_sum);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        __builtin_amdgcn_sched_barrier(0);
        if (tid + v * TEAM >= chunks) continue;
        as_read(raw[v]);
        grad8<T>(a, l, dz, tid + v * TEAM, raw[v], top, gq, gp);
    }
    for (int c = tid + NV * TEAM; c < chunks; c += U * TEAM) {
        Raw8<T> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = load_whole8(z + 8 * static_cast<int64_t>(min(c + u * TEAM, chunks - 1)));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * TEAM < chunks) grad8<T>(a, l, dz, c + u * TEAM, q[u], top, gq, gp);
    }
    if (rest < a.vocab) grad1<T>(a, l, dz, rest, z_rest, top, gq, gp);
}

// The gradient by itself: blocks of `segment` chunks of a row.
template <typename T>
__global__ __launch_bounds__(512) void k_distill_bwd(DistillArgs a)
{
    __shared__ Entries l;
    const int64_t r = blockIdx.x;
    const int chunks = a.vocab / 8;
    const int from = static_cast<int>(blockIdx.y) * a.segment, to = min(from + a.segment, chunks);
    const int rest = to == chunks ? 8 * chunks + static_cast<int>(threadIdx.x) : -1;
    const T *z = static_cast<const T *>(a.z) + r * a.z_st;
    T *dz = static_cast<T *>(a.dz) + r * a.d_st;
    const float weight = a.row_weight ? a.row_weight[r] : 1.f;
    if (threadIdx.x < 64 && weight != 0.f) read_entries<T>(a, r, z, false, true, l);
    __syncthreads();
    const double t_sum = weight != 0.f ? l.total : 0.0;
    if (t_sum == 0.0) {
        zero_words(dz, from + static_cast<int>(threadIdx.x), to, 512, rest, a.vocab);
        return;
    }
    const double g = a.grad * weight * a.dloss[r];
    const float top = a.stats_in[2 * r];
    const float gq = static_cast<float>(g / a.stats_in[2 * r + 1]), gp = static_cast<float>(g / t_sum);
    for (int c = from + static_cast<int>(threadIdx.x); c < to; c += U * 512) {
        Raw8<T> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = load_whole8(z + 8 * static_cast<int64_t>(min(c + u * 512, to - 1)));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * 512 < to) grad8<T>(a, l, dz, c + u * 512, q[u], top, gq, gp);
    }
    if (rest >= 0 && rest < a.vocab) grad1<T>(a, l, dz, rest, to_f32(z[rest]), top, gq, gp);
}

// Threads and chunks by the row.  (With eight chunks for rows over 65536 words, two
// blocks a CU in place of one, and the rest of the row read twice, 2048 rows of
// 128256 words in bf16 take 210 us with a gradient that goes past the caches, as
// with sixteen, 235 against 218 with one that does not, and 94 against 112 for the
// loss alone.  One form for all gives one loss, bit for bit.)
template <typename T>
pq_status launch_rows(const DistillArgs &a, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.rows));
    if (a.vocab <= 256 * 8 * 4) hipLaunchKernelGGL((k_distill<T, 256, 4>), grid, dim3(256), 0, s, a);
    else if (a.vocab <= 512 * 8 * 8) hipLaunchKernelGGL((k_distill<T, 512, 8>), grid, dim3(512), 0, s, a);
    else if (sizeof(T) == 4 || a.vocab <= 1024 * 8 * 8) hipLaunchKernelGGL((k_distill<T, 1024, 8>), grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((k_distill<T, 1024, sizeof(T) == 2 ? 16 : 8>), grid, dim3(1024), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

template <typename T>
pq_status launch_bwd_rows(const DistillArgs &a, hipStream_t s)
{
    const int64_t chunks = a.vocab / 8 > 0 ? a.vocab / 8 : 1;
    hipLaunchKernelGGL(k_distill_bwd<T>, dim3(static_cast<unsigned>(a.rows), static_cast<unsigned>((chunks + a.segment - 1) / a.segment)),
                       dim3(512), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

template <typename T, typename F>
pq_status launch_distill(DistillArgs a, F &&launch)
{
    const int tsize = dtype_bytes(a.top_dtype);
    for (int64_t left = a.rows; left > 0; left -= kLaunchRows) {
        a.rows = static_cast<int>(left < kLaunchRows ? left : kLaunchRows);
        const pq_status rc = launch(a);
        if (rc != PQ_OK) return rc;
        skip_rows(a.z, a.rows, a.z_st, sizeof(T));
        skip_rows(a.dz, a.rows, a.d_st, sizeof(T));
        skip_rows(a.index, a.rows, a.k, 4);
        skip_rows(a.top, a.rows, a.k, tsize);
        skip_rows(a.row_weight, a.rows, 1, 4);
        skip_rows(a.dloss, a.rows, 1, 4);
        skip_rows(a.stats_in, a.rows, 2, 4);
        skip_rows(a.loss, a.rows, 1, 4);
        skip_rows(a.stats, a.rows, 2, 4);
    }
    return PQ_OK;
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
    const float c = static_cast<float>(1.4426950408889634074 / temperature);
    if (!(temperature > 0.0) || !(temp > 0.f) || !(inv > 0.f) || !std::isfinite(temp) || !std::isfinite(c))
        return PQ_ERR_ARG;
    if (rows == 0) return PQ_OK;
    if (!logits || !index || !top) return PQ_ERR_NULL;
    if (misaligned(logits, size) || misaligned(dlogits, size) || misaligned(index, 4) || misaligned(top, tsize) ||
        misaligned(row_weight, 4))
        return PQ_ERR_ALIGN;
    if (dlogits == logits && d_stride != l_stride) return PQ_ERR_ARG;
    if (dlogits && rows_overlap(rows, vocab, d_stride)) return PQ_ERR_SHAPE;
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
    a.c = c;
    // Over half the memory-side cache's size is written past the caches (2048 x
    // 128256 in bf16 209 us against 220, 512 x 200000 95 against 109); less may be
    // found there by its reader.  Not where a store is part of a piece of memory:
    // fp32, whose eight words take two (1024 x 128256 280 against 242), and rows at
    // odd addresses (2048 x 128257 264 against 261, the gradient alone 243 against
    // 229).
    a.nt = size == 2 && rows * vocab * size > (int64_t(1) << 27) && aligned16(dlogits) && d_stride % 8 == 0;
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
    auto with = [&](auto type) {
        using T = decltype(type);
        return launch_distill<T>(a, [&](const DistillArgs &b) { return launch_rows<T>(b, s); });
    };
    return dtype == PQ_F32 ? with(float{}) : dtype == PQ_BF16 ? with(bf16_t{}) : with(f16_t{});
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
    const int64_t chunks = vocab / 8 > 0 ? vocab / 8 : 1;
    // equal parts of up to 32768 words, at most 32768 of them a row
    const int64_t segments = (chunks + 4095) / 4096;
    a.segment = static_cast<int>((chunks + segments - 1) / segments);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto with = [&](auto type) {
        using T = decltype(type);
        return launch_distill<T>(a, [&](const DistillArgs &b) { return launch_bwd_rows<T>(b, s); });
    };
    return dtype == PQ_F32 ? with(float{}) : dtype == PQ_BF16 ? with(bf16_t{}) : with(f16_t{});
}

}  // extern "C"
