// pq_kv_common.hpp -- internal pieces shared by the serving sources: element
// loads and stores, the cache descriptor's checks and addressing.  Not part of
// the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pq_common.hpp"

namespace pq {

// Accesses whose address is a multiple of 8 bytes only (caller's strides): the
// hardware needs dword alignment.
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));

struct bf16_t { uint16_t bits; };
struct f16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16_t x) { return bf16_to_f32(x.bits); }
__device__ __forceinline__ float to_f32(f16_t x) { return static_cast<float>(__builtin_bit_cast(_Float16, x.bits)); }

template <typename T>
__device__ __forceinline__ T from_f32(float x)
{
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (__is_same(T, bf16_t)) return bf16_t{__builtin_bit_cast(uint16_t, static_cast<__bf16>(x))};
    else return f16_t{__builtin_bit_cast(uint16_t, static_cast<_Float16>(x))};
}

// The two 16-bit values of a word, in fp32.
template <typename T>
__device__ __forceinline__ void unpack16(uint32_t w, float &lo, float &hi)
{
    if constexpr (__is_same(T, bf16_t)) {
        lo = __builtin_bit_cast(float, w << 16);
        hi = __builtin_bit_cast(float, w & 0xFFFF0000u);
    } else {
        lo = to_f32(f16_t{static_cast<uint16_t>(w)});
        hi = to_f32(f16_t{static_cast<uint16_t>(w >> 16)});
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if constexpr (__is_same(T, bf16_t)) return pack_bf16x2(lo, hi);
    else
        return static_cast<uint32_t>(from_f32<f16_t>(lo).bits) | (static_cast<uint32_t>(from_f32<f16_t>(hi).bits) << 16);
}

// N consecutive elements to fp32 and back; N = 4 or 8 with addresses aligned
// to min(16, N * sizeof(T)) bytes, or N = 1.  The cache kernels' vector stores
// are non-temporal whatever their size: rows need not be whole lines, and a
// plain store of part of a line waits for the rest of it in L2 (rows of 80
// channels read back from 4 bits: 63 us against 85; prompts appended 44
// against 58).
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T *p, float (&x)[N])
{
    if constexpr (N == 1) {
        x[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f32x4 v = reinterpret_cast<const f32x4 *>(p)[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
        }
    } else if constexpr (N == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack16<T>(v[e], x[2 * e], x[2 * e + 1]);
    } else {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
        for (int e = 0; e < 2; ++e) unpack16<T>(v[e], x[2 * e], x[2 * e + 1]);
    }
}

// Eight consecutive elements as they lie in memory (a load that does not look
// at its value yet), and their fp32 values.
template <typename T>
struct Raw8 {
    u32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const u32x4 *>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void raw_to_f32(const Raw8<T> &r, float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = __builtin_bit_cast(f32x4, r.w[0]), b = __builtin_bit_cast(f32x4, r.w[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = a[e];
            x[4 + e] = b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack16<T>(r.w[0][e], x[2 * e], x[2 * e + 1]);
    }
}

// A vector store, past the caches (NT) or not.
template <bool NT, typename V>
__device__ __forceinline__ void store_vec(V *p, V v)
{
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

template <typename T, int N, bool NT = true>
__device__ __forceinline__ void store_f32(T *p, const float (&x)[N])
{
    if constexpr (N == 1) {
        *p = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            store_vec<NT>(reinterpret_cast<f32x4 *>(p) + i, f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]});
    } else if constexpr (N == 8) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pack16<T>(x[2 * e], x[2 * e + 1]);
        store_vec<NT>(reinterpret_cast<u32x4 *>(p), v);
    } else {
        u32x2 v;
#pragma unroll
        for (int e = 0; e < 2; ++e) v[e] = pack16<T>(x[2 * e], x[2 * e + 1]);
        store_vec<NT>(reinterpret_cast<u32x2 *>(p), v);
    }
}

// Blocks of 256 threads of one launch: a grid's threads are counted in 32 bits.
constexpr int64_t kMaxBlocks = ((int64_t(1) << 32) - 1) / 256;

// Smallest scale of a quantised row, 2^-60: a constant row then has a scale
// whose reciprocal and whose logarithm are finite.
constexpr float kMinKvScale = 0x1p-60f;

inline int dtype_bytes(int dtype) { return dtype == PQ_F32 ? 4 : dtype == PQ_BF16 || dtype == PQ_F16 ? 2 : 0; }

inline int64_t kv_row_bytes(int format, int64_t dim)
{
    if (dim < 16 || dim > 256 || dim % 16) return -1;
    switch (format) {
    case PQ_KV_16: return 2 * dim;
    case PQ_KV_8: return dim;
    case PQ_KV_4: return dim / 2;
    default: return -1;
    }
}

inline int log2_of(int v) { return __builtin_ctz(static_cast<unsigned>(v)); }

// The descriptor by itself (no pointer is followed).
inline pq_status kv_cache_status(const pq_kv_cache *c)
{
    if (!c) return PQ_ERR_NULL;
    if (c->format < PQ_KV_16 || c->format > PQ_KV_4) return PQ_ERR_MODE;
    if (c->format == PQ_KV_16 && c->dtype != PQ_BF16 && c->dtype != PQ_F16) return PQ_ERR_MODE;
    if (c->reserved != 0) return PQ_ERR_ARG;
    const int64_t rb = kv_row_bytes(c->format, c->dim);
    if (rb < 0 || c->heads < 1 || c->heads > 65535) return PQ_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 32768 || (c->page_size & (c->page_size - 1))) return PQ_ERR_SHAPE;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX) return PQ_ERR_SHAPE;
    const int64_t st[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (int64_t s : st)
        if (s < 0 || s % 8) return PQ_ERR_SHAPE;
    // a token's offset inside a page is 32-bit in the kernels
    if (c->token_stride < rb || c->token_stride > (INT32_MAX - rb) / c->page_size) return PQ_ERR_SHAPE;
    if (!c->k || !c->v) return PQ_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v)) return PQ_ERR_ALIGN;
    if (c->format != PQ_KV_16) {
        if (!c->k_param || !c->v_param) return PQ_ERR_NULL;
        if (!aligned16(c->k_param) || !aligned16(c->v_param)) return PQ_ERR_ALIGN;
    }
    return PQ_OK;
}

}  // namespace pq
