// pq_kv.hip -- gfx950 kernels and C entry points of the key-value cache: new
// tokens rotated, quantised and written (pq_kv_append), and tokens read back
// into dense arrays (pq_kv_load).
//
// A quantised row (one token and head of K or V) is held as x^ = z + s n with
// n in 0 .. Q and one bf16 pair (s, z) per row.  One pair per row and not per
// group of channels, because of what the attention kernel can do with it: the
// pair leaves both products as a factor and a constant per token (q . k^ =
// s (q . n) + z sum q, and sum p v^ = sum (p s) n + sum p z), so that the
// matrix unit multiplies the bare codes.  Both kernels move 2 to 4 bytes a
// channel for about ten operations: the memory system bounds them.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pq_kv_common.hpp"

namespace pq {
namespace {

// ------------------------------------------------------------------ append

struct AppendArgs {
    uint8_t *k, *v;
    uint32_t *kp, *vp;
    int64_t page_stride, head_stride, num_slots;
    int token_stride, page_log2, heads, dim;
    const void *xk, *xv, *q;
    void *qo;
    int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;   // elements
    const int64_t *slots;
    const int32_t *positions;
    const float *table;             // NULL: no rotation
    int64_t tokens;
    int max_pos, rot, half, q_heads;
    int lanes_log2;                 // log2 of the lanes of a row (8 channels each)
    int rows, slices;               // rows of a token (2 heads + q_heads); waves per token
};

// The rotation of one lane's 8 channels d0 .. d0 + 7: y = x c + partner s per
// channel, with s carrying the sign of the channel's half; `on` has a bit per
// rotated channel.
struct Turn {
    float c[8], s[8];
    int partner;                    // half layout: channel of element 0's partner
    unsigned on;
};

__device__ __forceinline__ void load_turn(const AppendArgs &a, int d0, int pos, Turn &t)
{
    t.on = 0;
    t.partner = d0;
    if (!a.table || pos < 0 || d0 >= a.rot) return;
    const int hr = a.rot / 2;
    const bool known = pos < a.max_pos;
    const float *row = a.table + static_cast<int64_t>(known ? pos : 0) * a.rot;
    const bool whole = a.rot % 16 == 0;             // a lane's channels and their partners are whole 8-channel runs
    t.partner = d0 < hr ? d0 + hr : d0 - hr;
    if (whole) {
        float cs[16];
        const int first = a.half ? (d0 < hr ? d0 : d0 - hr) : d0 / 2;
        if (a.max_pos > 0) {
            if (a.half) load_f32<float, 16>(row + 2 * first, cs);
            else {
                float c8[8];
                load_f32<float, 8>(row + 2 * first, c8);
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] = c8[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = a.half ? cs[2 * e] : cs[e & ~1], s = a.half ? cs[2 * e + 1] : cs[e | 1];
            const bool second = a.half ? d0 >= hr : e & 1;
            t.c[e] = known ? c : __builtin_nanf("");
            t.s[e] = second ? s : -s;
        }
        t.on = 0xFF;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            if (d >= a.rot) continue;
            const int i = a.half ? (d < hr ? d : d - hr) : d / 2;
            const bool second = a.half ? d >= hr : d & 1;
            const float c = known ? row[2 * i] : __builtin_nanf(""), s = known ? row[2 * i + 1] : 0.f;
            t.c[e] = c;
            t.s[e] = second ? s : -s;
            t.on |= 1u << e;
        }
    }
}

// x: the lane's channels of a row, already loaded; `row` points at the row.
template <typename T>
__device__ __forceinline__ void apply_turn(const AppendArgs &a, const Turn &t, const T *row, int d0, float (&x)[8])
{
    if (!t.on) return;
    float y[8];
    if (!a.half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
    } else if (a.rot % 16 == 0) {
        load_f32<T, 8>(row + t.partner, y);
    } else {
        const int hr = a.rot / 2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            y[e] = d < a.rot ? to_f32(row[d < hr ? d + hr : d - hr]) : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (t.on >> e & 1) x[e] = x[e] * t.c[e] + y[e] * t.s[e];
}

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// One wave per token and slice of its rows: 2 heads rows of K and V, then the
// query heads.  2^lanes_log2 lanes hold a row, 8 channels each, so the row's
// minimum and maximum are a butterfly inside them and a wave takes several
// rows at once; the rotation's table values stay in registers over the rows.
template <typename T, int FMT, typename CT>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a)
{
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int64_t token = wave / a.slices;
    if (token >= a.tokens) return;
    const int lane = threadIdx.x & 63;
    const int row_lanes = 1 << a.lanes_log2, side = 64 >> a.lanes_log2;
    const int d0 = (lane & (row_lanes - 1)) * 8;
    const bool mine = d0 < a.dim;
    const int64_t slot = a.slots[token];
    const bool stored = slot >= 0 && slot < a.num_slots;
    const int64_t page = stored ? slot >> a.page_log2 : 0;
    const int off = static_cast<int>(slot & ((1 << a.page_log2) - 1));
    Turn turn;
    turn.on = 0;
    turn.partner = d0;
    if (mine) load_turn(a, d0, a.table ? a.positions[token] : 0, turn);

    const int step = side * a.slices;
    for (int base = side * static_cast<int>(wave - token * a.slices); base < a.rows; base += step) {
        const int r = base + (lane >> a.lanes_log2);
        const bool live = mine && r < a.rows;
        const int kind = r < a.heads ? 0 : r < 2 * a.heads ? 1 : 2;
        const int h = kind == 0 ? r : kind == 1 ? r - a.heads : r - 2 * a.heads;
        float x[8] = {};
        if (live) {
            const T *src = kind == 0   ? static_cast<const T *>(a.xk) + token * a.k_ts + h * a.k_hs
                           : kind == 1 ? static_cast<const T *>(a.xv) + token * a.v_ts + h * a.v_hs
                                       : static_cast<const T *>(a.q) + token * a.q_ts + h * a.q_hs;
            load_f32<T, 8>(src + d0, x);
            if (kind != 1) apply_turn<T>(a, turn, src, d0, x);
            // q_out may be q: every lane's loads of a row come before its
            // store, and the lanes of a row are in one wave
            if (kind == 2) store_f32<T, 8>(static_cast<T *>(a.qo) + token * a.qo_ts + h * a.qo_hs + d0, x);
        }
        if constexpr (FMT == PQ_KV_16) {
            if (live && kind < 2 && stored) {
                uint8_t *dst = (kind ? a.v : a.k) + page * a.page_stride + h * a.head_stride +
                               static_cast<int64_t>(off) * a.token_stride + 2 * d0;
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack16<CT>(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<u32x4_a8 *>(dst) = w;
            }
        } else {
            constexpr float top = FMT == PQ_KV_8 ? 255.f : 15.f;
            float mn = __builtin_inff(), mx = -__builtin_inff();
            if (live) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mn = min_nan(mn, x[e]);
                    mx = max_nan(mx, x[e]);
                }
            }
            for (int o = 1; o < row_lanes; o <<= 1) {
                mn = min_nan(mn, __shfl_xor(mn, o));
                mx = max_nan(mx, __shfl_xor(mx, o));
            }
            if (live && kind < 2 && stored) {
                const uint32_t sb = pack_bf16x2((mx - mn) * (1.f / top), mn);
                const float s = fmaxf(bf16_to_f32(sb & 0xFFFFu), kMinKvScale), z = bf16_to_f32(sb >> 16);
                const float inv = 1.f / s;
                uint32_t n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // clamped, then rounded to even by the addition of 2^23
                    const float v = fminf(fmaxf((x[e] - z) * inv, 0.f), top) + 8388608.f;
                    n[e] = __builtin_bit_cast(uint32_t, v) & 0xFFu;
                }
                const int64_t rowoff = page * a.page_stride + h * a.head_stride + static_cast<int64_t>(off) * a.token_stride;
                uint8_t *dst = (kind ? a.v : a.k) + rowoff;
                if constexpr (FMT == PQ_KV_8) {
                    u32x2 w;
                    w[0] = n[0] | n[1] << 8 | n[2] << 16 | n[3] << 24;
                    w[1] = n[4] | n[5] << 8 | n[6] << 16 | n[7] << 24;
                    *reinterpret_cast<u32x2 *>(dst + d0) = w;
                } else {
                    uint32_t w = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w |= n[e] << (4 * e);
                    *reinterpret_cast<uint32_t *>(dst + d0 / 2) = w;
                }
                if (d0 == 0) {
                    const uint32_t pair = (__builtin_bit_cast(uint32_t, s) >> 16) | (sb & 0xFFFF0000u);
                    (kind ? a.vp : a.kp)[((page * a.heads + h) << a.page_log2) + off] = pair;
                }
            }
        }
    }
}

template <typename T>
pq_status launch_append(const pq_kv_cache &c, const AppendArgs &a, hipStream_t s)
{
    const int64_t blocks = (a.tokens * a.slices + 3) / 4;
    if (blocks > INT32_MAX) return PQ_ERR_SHAPE;
    const dim3 g(static_cast<unsigned>(blocks)), b(256);
    if (c.format == PQ_KV_8) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_8, bf16_t>), g, b, 0, s, a);
    else if (c.format == PQ_KV_4) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_4, bf16_t>), g, b, 0, s, a);
    else if (c.dtype == PQ_BF16) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_16, bf16_t>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_kv_append<T, PQ_KV_16, f16_t>), g, b, 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

// -------------------------------------------------------------------- load

constexpr int kLoadTokens = 16;     // output tokens of a block

struct LoadArgs {
    const uint8_t *k, *v;
    const uint32_t *kp, *vp;
    int64_t page_stride, head_stride, num_pages;
    int token_stride, page_log2, heads, dim;
    const int32_t *table;
    int64_t table_stride, max_pages;
    const int32_t *starts, *cu;
    int batch;
    int64_t tokens;
    void *ko, *vo;
    int64_t ko_ts, ko_hs, vo_ts, vo_hs;
    int lanes_log2, slices;         // lanes of a row (8 channels each); blocks per token tile
};

// A block takes 16 consecutive output tokens: 16 lanes find their pages (the
// sequence by a binary search of cu), then the waves walk (head, K or V).  For
// one head the 16 tokens' rows lie together in a page, so a wave reads whole
// lines of codes and writes whole rows.
template <typename T, int FMT, typename CT>
__global__ __launch_bounds__(256) void k_kv_load(LoadArgs a)
{
    __shared__ int s_page[kLoadTokens], s_off[kLoadTokens];
    const int64_t tile = blockIdx.x / a.slices;
    const int slice = static_cast<int>(blockIdx.x - tile * a.slices);
    const int64_t t0 = tile * kLoadTokens;
    if (threadIdx.x < kLoadTokens) {
        const int64_t i = t0 + threadIdx.x;
        int page = -1, off = 0;
        if (i < a.tokens && i < a.cu[a.batch]) {
            int lo = 0, hi = a.batch - 1;           // last b with cu[b] <= i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.cu[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const int64_t t = i - a.cu[lo] + (a.starts ? a.starts[lo] : 0);
            if (t >= 0 && (t >> a.page_log2) < a.max_pages) {
                const int p = a.table[lo * a.table_stride + (t >> a.page_log2)];
                if (p >= 0 && p < a.num_pages) page = p;
                off = static_cast<int>(t & ((1 << a.page_log2) - 1));
            }
        }
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = off;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row_lanes = 1 << a.lanes_log2, side = 64 >> a.lanes_log2;
    const int d0 = (lane & (row_lanes - 1)) * 8;
    if (d0 >= a.dim) return;
    for (int r = slice * 4 + wave; r < 2 * a.heads; r += 4 * a.slices) {
        const bool is_v = r >= a.heads;
        const int h = is_v ? r - a.heads : r;
        const uint8_t *src = (is_v ? a.v : a.k) + h * a.head_stride;
        const uint32_t *par = is_v ? a.vp : a.kp;
        T *out = static_cast<T *>(is_v ? a.vo : a.ko) + (is_v ? a.vo_hs : a.ko_hs) * h + d0;
        const int64_t ts = is_v ? a.vo_ts : a.ko_ts;
#pragma unroll 4
        for (int j = lane >> a.lanes_log2; j < kLoadTokens; j += side) {
            if (t0 + j >= a.tokens) break;
            const int page = s_page[j], off = s_off[j];
            float x[8] = {};
            if (page >= 0) {
                const uint8_t *p = src + page * a.page_stride + static_cast<int64_t>(off) * a.token_stride;
                if constexpr (FMT == PQ_KV_16) {
                    const u32x4 w = *reinterpret_cast<const u32x4_a8 *>(p + 2 * d0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) unpack16<CT>(w[e], x[2 * e], x[2 * e + 1]);
                } else {
                    const uint32_t pair = par[((static_cast<int64_t>(page) * a.heads + h) << a.page_log2) + off];
                    const float s = bf16_to_f32(pair & 0xFFFFu), z = bf16_to_f32(pair >> 16);
                    if constexpr (FMT == PQ_KV_8) {
                        const u32x2 w = *reinterpret_cast<const u32x2 *>(p + d0);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = z + s * static_cast<float>(w[e >> 2] >> (8 * (e & 3)) & 0xFFu);
                    } else {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(p + d0 / 2);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = z + s * static_cast<float>(w >> (4 * e) & 0xFu);
                    }
                }
            }
            store_f32<T, 8>(out + (t0 + j) * ts, x);
        }
    }
}

template <typename T>
pq_status launch_load(const pq_kv_cache &c, const LoadArgs &a, unsigned blocks, hipStream_t s)
{
    const dim3 g(blocks), b(256);
    if (c.format == PQ_KV_8) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_8, bf16_t>), g, b, 0, s, a);
    else if (c.format == PQ_KV_4) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_4, bf16_t>), g, b, 0, s, a);
    else if (c.dtype == PQ_BF16) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_16, bf16_t>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_kv_load<T, PQ_KV_16, f16_t>), g, b, 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

// log2 of the lanes that hold a row, 8 channels each.
int row_lanes_log2(int dim)
{
    int l = 1;
    while ((8 << l) < dim) ++l;
    return l;
}

bool strides8(const int64_t *s, int n)
{
    for (int i = 0; i < n; ++i)
        if (s[i] % 8) return false;
    return true;
}

}  // namespace
}  // namespace pq

extern "C" {

int64_t pq_kv_row_bytes(int format, int64_t dim) { return pq::kv_row_bytes(format, dim); }

pq_status pq_kv_append(const pq_kv_cache *cache, int dtype, int64_t tokens, const void *k, int64_t k_token_stride,
                       int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                       const int64_t *slots, const int32_t *positions, const float *table, int64_t max_pos,
                       int64_t rot, int layout, const void *q, int64_t q_heads, int64_t q_token_stride,
                       int64_t q_head_stride, void *q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                       void *stream)
{
    using namespace pq;
    const pq_status st = kv_cache_status(cache);
    if (st != PQ_OK) return st;
    const pq_kv_cache &c = *cache;
    if (!dtype_bytes(dtype)) return PQ_ERR_MODE;
    if (table && layout != PQ_ROPE_HALF && layout != PQ_ROPE_INTERLEAVED) return PQ_ERR_MODE;
    if (tokens < 0 || q_heads < 0 || q_heads > 65535) return PQ_ERR_SHAPE;
    if (table && (rot < 0 || rot > c.dim || rot % 2 || max_pos < 0 || max_pos > INT32_MAX)) return PQ_ERR_SHAPE;
    const int64_t strides[8] = {k_token_stride, k_head_stride, v_token_stride,  v_head_stride,
                                q_token_stride, q_head_stride, qo_token_stride, qo_head_stride};
    if (!strides8(strides, q_heads ? 8 : 4)) return PQ_ERR_SHAPE;
    if (q_heads && !table) return PQ_ERR_ARG;
    if (tokens == 0) return PQ_OK;
    if (!k || !v || !slots || (table && !positions) || (q_heads && (!q || !q_out))) return PQ_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (q_heads && (!aligned16(q) || !aligned16(q_out)))) return PQ_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(slots) % 8 || reinterpret_cast<uintptr_t>(positions) % 4 || !aligned16(table))
        return PQ_ERR_ALIGN;
    if (q_heads && q == q_out && (q_token_stride != qo_token_stride || q_head_stride != qo_head_stride))
        return PQ_ERR_ARG;
    AppendArgs a = {};
    a.k = static_cast<uint8_t *>(c.k);
    a.v = static_cast<uint8_t *>(c.v);
    a.kp = static_cast<uint32_t *>(c.k_param);
    a.vp = static_cast<uint32_t *>(c.v_param);
    a.page_stride = c.page_stride;
    a.head_stride = c.head_stride;
    a.token_stride = static_cast<int>(c.token_stride);
    a.page_log2 = log2_of(c.page_size);
    a.num_slots = c.num_pages << a.page_log2;
    a.heads = c.heads;
    a.dim = c.dim;
    a.xk = k;
    a.xv = v;
    a.q = q;
    a.qo = q_out;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.qo_ts = qo_token_stride;
    a.qo_hs = qo_head_stride;
    a.slots = slots;
    a.positions = positions;
    a.table = rot > 0 ? table : nullptr;
    a.tokens = tokens;
    a.max_pos = static_cast<int>(max_pos);
    a.rot = static_cast<int>(rot);
    a.half = layout == PQ_ROPE_HALF;
    a.q_heads = static_cast<int>(q_heads);
    a.lanes_log2 = row_lanes_log2(c.dim);
    a.rows = 2 * c.heads + a.q_heads;
    // Few tokens: a token's rows go to several waves, as in the rotation.
    const int side = 64 >> a.lanes_log2;
    const int64_t rounds = (a.rows + side - 1) / side;
    int64_t slices = (2048 + tokens - 1) / tokens;
    if (slices > rounds) slices = rounds;
    a.slices = static_cast<int>(slices);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == PQ_F32) return launch_append<float>(c, a, s);
    return dtype == PQ_BF16 ? launch_append<bf16_t>(c, a, s) : launch_append<f16_t>(c, a, s);
}

pq_status pq_kv_load(const pq_kv_cache *cache, int dtype, int64_t batch, int64_t tokens, const int32_t *block_table,
                     int64_t table_stride, int64_t max_pages, const int32_t *starts, const int32_t *cu, void *k_out,
                     int64_t ko_token_stride, int64_t ko_head_stride, void *v_out, int64_t vo_token_stride,
                     int64_t vo_head_stride, void *stream)
{
    using namespace pq;
    const pq_status st = kv_cache_status(cache);
    if (st != PQ_OK) return st;
    const pq_kv_cache &c = *cache;
    if (!dtype_bytes(dtype)) return PQ_ERR_MODE;
    if (batch < 0 || batch > INT32_MAX - 1 || tokens < 0 || max_pages < 0 || table_stride < 0) return PQ_ERR_SHAPE;
    const int64_t strides[4] = {ko_token_stride, ko_head_stride, vo_token_stride, vo_head_stride};
    if (!strides8(strides, 4)) return PQ_ERR_SHAPE;
    if (tokens == 0) return PQ_OK;
    if (batch == 0) return PQ_ERR_ARG;              // rows without a sequence
    if ((!block_table && max_pages > 0) || !cu || !k_out || !v_out) return PQ_ERR_NULL;
    if (!aligned16(k_out) || !aligned16(v_out)) return PQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(cu)) % 4)
        return PQ_ERR_ALIGN;
    LoadArgs a = {};
    a.k = static_cast<const uint8_t *>(c.k);
    a.v = static_cast<const uint8_t *>(c.v);
    a.kp = static_cast<const uint32_t *>(c.k_param);
    a.vp = static_cast<const uint32_t *>(c.v_param);
    a.page_stride = c.page_stride;
    a.head_stride = c.head_stride;
    a.num_pages = c.num_pages;
    a.token_stride = static_cast<int>(c.token_stride);
    a.page_log2 = log2_of(c.page_size);
    a.heads = c.heads;
    a.dim = c.dim;
    a.table = block_table;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.starts = starts;
    a.cu = cu;
    a.batch = static_cast<int>(batch);
    a.tokens = tokens;
    a.ko = k_out;
    a.vo = v_out;
    a.ko_ts = ko_token_stride;
    a.ko_hs = ko_head_stride;
    a.vo_ts = vo_token_stride;
    a.vo_hs = vo_head_stride;
    a.lanes_log2 = row_lanes_log2(c.dim);
    // Few tokens: the heads of a token tile go to several blocks.
    const int64_t tiles = (tokens + kLoadTokens - 1) / kLoadTokens;
    const int64_t rounds = (2 * c.heads + 3) / 4;
    int64_t slices = (1024 + tiles - 1) / tiles;
    if (slices > rounds) slices = rounds;
    a.slices = static_cast<int>(slices);
    if (tiles * slices > INT32_MAX) return PQ_ERR_SHAPE;
    const unsigned blocks = static_cast<unsigned>(tiles * slices);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == PQ_F32) return launch_load<float>(c, a, blocks, s);
    return dtype == PQ_BF16 ? launch_load<bf16_t>(c, a, blocks, s) : launch_load<f16_t>(c, a, blocks, s);
}

}  // extern "C"
