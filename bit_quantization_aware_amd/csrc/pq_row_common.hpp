// pq_row_common.hpp -- internal pieces shared by the kernels that hold rows in
// registers (normalisation, rows in 8 bits, distillation): access to eight
// consecutive elements of any alignment, and sums over a team of threads.  Not
// part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pq_kv_common.hpp"

namespace pq {
namespace {

// Rows need not begin at a multiple of 16 bytes (odd widths, views).  Global
// memory takes a vector at any address, so that one form of access serves them
// all: lines that are cut in two cost the memory system twice, the issue once.
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

template <typename T>
__device__ __forceinline__ Raw8<T> load_whole8(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const u32x4_a1 *>(p)[i];
    return r;
}

// The compiler would keep a row's fp32 values from one use to the next, twice
// the registers of 16-bit words: it is told that they may have changed.
template <typename T>
__device__ __forceinline__ void as_read(Raw8<T> &raw)
{
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) asm volatile("" : "+v"(raw.w[i]));
}

// Elements 8c .. 8c + 7 of a row of `cols`, as they lie in memory; those past
// its end are zero.
template <typename T>
__device__ __forceinline__ Raw8<T> load_row8(const T *row, int c, int cols)
{
    Raw8<T> r;
    const T *p = row + 8 * static_cast<int64_t>(c);
    if (8 * c + 8 <= cols) return load_whole8(p);
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) r.w[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (8 * c + e >= cols) break;
        if constexpr (sizeof(T) == 4) {
            r.w[e >> 2][e & 3] = __builtin_bit_cast(uint32_t, p[e]);
        } else {
            r.w[0][e >> 1] |= static_cast<uint32_t>(p[e].bits) << (16 * (e & 1));
        }
    }
    return r;
}

// NT: past the caches.  Where a branch has this store on one side and an
// ordinary one on the other, the compiler would make one of the two and drop the
// hint; it cannot join what lies between statements of its own.
template <bool NT = false, typename T>
__device__ __forceinline__ void store_whole8(T *p, const float (&x)[8])
{
    if constexpr (NT) asm volatile("");
    if constexpr (sizeof(T) == 4) {
        const f32x4 v[2] = {{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}};
        f32x4_a4 *to = reinterpret_cast<f32x4_a4 *>(p);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (NT) __builtin_nontemporal_store(v[i], to + i);
            else to[i] = v[i];
        }
    } else {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pack16<T>(x[2 * e], x[2 * e + 1]);
        u32x4_a1 *to = reinterpret_cast<u32x4_a1 *>(p);
        if constexpr (NT) __builtin_nontemporal_store(v, to);
        else *to = v;
    }
    if constexpr (NT) asm volatile("");
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_row8(T *row, int c, int cols, const float (&x)[8])
{
    T *p = row + 8 * static_cast<int64_t>(c);
    if (8 * c + 8 <= cols) {
        store_whole8<NT>(p, x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (8 * c + e < cols) p[e] = from_f32<T>(x[e]);
}

// Rows of one launch, a block of up to 1024 threads each: a grid's threads are
// counted in 32 bits.  More rows go in several launches.
constexpr int64_t kLaunchRows = int64_t(1) << 21;

// Moves a pointer that may be NULL by `rows` rows of `stride` elements.
template <typename P>
inline void skip_rows(P *&p, int64_t rows, int64_t stride, int size)
{
    if (p) p = reinterpret_cast<P *>(reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(rows * stride * size));
}

// Whether the rows of an output would lie over each other.
inline bool rows_overlap(int64_t rows, int64_t cols, int64_t stride) { return rows > 1 && stride < cols && stride > -cols; }

// Eight values of an array of any element type (a run-time choice that is the
// same for all threads).
__device__ __forceinline__ void load_any8(const void *a, int dtype, int c, int cols, float (&x)[8])
{
    if (dtype == PQ_F32) raw_to_f32<float>(load_row8(static_cast<const float *>(a), c, cols), x);
    else if (dtype == PQ_BF16) raw_to_f32<bf16_t>(load_row8(static_cast<const bf16_t *>(a), c, cols), x);
    else raw_to_f32<f16_t>(load_row8(static_cast<const f16_t *>(a), c, cols), x);
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), m)));
    return x;
}

}  // namespace
}  // namespace pq
