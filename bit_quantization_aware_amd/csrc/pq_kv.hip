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

// The lanes of a row, 8 channels each (an even number: dim is a multiple of
// 16), rows side by side without a gap.
struct RowLanes {
    int n, inverse;                 // 2^16 / n, rounded up: lane / n = lane * inverse >> 16 for lanes below 256
    int side;                       // rows of a wave
    RowLanes() = default;
    explicit RowLanes(int dim) : n(dim / 8), inverse((65536 + n - 1) / n), side(64 / n) {}
    __device__ __forceinline__ int row(int lane) const { return lane * inverse >> 16; }
};

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
    RowLanes lanes;
    int kv_groups, groups, slices;  // row groups of a token: of K and of V each, of K, V and Q; waves per token
};

// The rotation of one lane's 8 channels d0 .. d0 + 7: y = x c + partner s per
// channel, with s carrying the sign of the channel's half; `on` has a bit per
// rotated channel.
struct Turn {
    float c[8], s[8];
    unsigned on;
};

__device__ __forceinline__ void load_turn(const AppendArgs &a, int d0, int pos, Turn &t)
{
    t.on = 0;
    if (!a.table || pos < 0 || d0 >= a.rot) return;
    const int hr = a.rot / 2;
    const bool known = pos < a.max_pos;
    const float *row = a.table + static_cast<int64_t>(known ? pos : 0) * a.rot;
    const bool whole = a.rot % 16 == 0;             // a lane's channels and their partners are whole 8-channel runs
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

// x: the lane's channels of a row; `other`: its partner's run (half layout,
// whole runs); `row` points at the row.
template <typename T>
__device__ __forceinline__ void apply_turn(const AppendArgs &a, const Turn &t, const Raw8<T> &other, const T *row, int d0,
                                           float (&x)[8])
{
    if (!t.on) return;
    float y[8];
    if (!a.half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
    } else if (a.rot % 16 == 0) {
        raw_to_f32<T>(other, y);
    } else {
        const int hr = a.rot / 2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            y[e] = d < a.rot ? to_f32(row[d < hr ? d + hr : d - hr]) : 0.f;
        }
    }
    if (t.on == 0xFF) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * t.c[e] + y[e] * t.s[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (t.on >> e & 1) x[e] = x[e] * t.c[e] + y[e] * t.s[e];
    }
}

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Minimum and maximum over the n lanes of a row.  Powers of two: neighbours,
// pairs, quads and eights exchange by DPP (mirrors serve, since the lanes of a
// half agree).  Others: the row's n / 2 pairs as a ring, each looking ahead
// over what it has covered so far, and no further than around; `ring` holds
// the steps' source lanes, four bytes a lane.
template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float from_lane(int at, float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(at, __builtin_bit_cast(int, x)));
}
constexpr int kRingSteps = 4;       // up to 16 pairs
__device__ __forceinline__ void set_ring(int n, int lane, int in_row, int (&ring)[kRingSteps])
{
    int covered = 1;
#pragma unroll
    for (int i = 0; i < kRingSteps; ++i) {
        const int ahead = min(covered, n / 2 - covered), to = in_row + 2 * ahead;
        ring[i] = 4 * (lane - in_row + (to < n ? to : to - n));
        covered += ahead;
    }
}
__device__ __forceinline__ void row_range(int n, const int (&ring)[kRingSteps], float &mn, float &mx)
{
    constexpr int kPairs = 0xB1, kQuads = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;   // quad_perm 1 0 3 2; 2 3 0 1
    mn = min_nan(mn, dpp<kPairs>(mn));
    mx = max_nan(mx, dpp<kPairs>(mx));
    if (n & (n - 1)) {
        int covered = 1;
#pragma unroll
        for (int i = 0; i < kRingSteps; ++i) {
            if (covered >= n / 2) break;
            mn = min_nan(mn, from_lane(ring[i], mn));
            mx = max_nan(mx, from_lane(ring[i], mx));
            covered *= 2;
        }
        return;
    }
    if (n >= 4) {
        mn = min_nan(mn, dpp<kQuads>(mn));
        mx = max_nan(mx, dpp<kQuads>(mx));
    }
    if (n >= 8) {
        mn = min_nan(mn, dpp<kHalfMirror>(mn));
        mx = max_nan(mx, dpp<kHalfMirror>(mx));
    }
    if (n >= 16) {
        mn = min_nan(mn, dpp<kMirror>(mn));
        mx = max_nan(mx, dpp<kMirror>(mx));
    }
    if (n >= 32) {
        mn = min_nan(mn, __shfl_xor(mn, 16));
        mx = max_nan(mx, __shfl_xor(mx, 16));
    }
}

// Codes of a lane's 8 channels, as they lie in the row: whole numbers in fp32,
// put together two or four at a time by exact multiply-adds.
template <int FMT>
__device__ __forceinline__ u32x2 pack_codes(const float (&n)[8])
{
    u32x2 w;
    if constexpr (FMT == PQ_KV_8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = static_cast<uint32_t>(__builtin_fmaf(n[4 * i + 1], 256.f, n[4 * i]));
            const uint32_t hi = static_cast<uint32_t>(__builtin_fmaf(n[4 * i + 3], 256.f, n[4 * i + 2]));
            w[i] = hi << 16 | lo;
        }
    } else {
        uint32_t h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float lo = __builtin_fmaf(n[4 * i + 1], 16.f, n[4 * i]), hi = __builtin_fmaf(n[4 * i + 3], 16.f, n[4 * i + 2]);
            h[i] = static_cast<uint32_t>(__builtin_fmaf(hi, 256.f, lo));
        }
        w[0] = h[1] << 16 | h[0];
        w[1] = 0;
    }
    return w;
}

// One wave per token and slice of its rows.  dim / 8 lanes hold a row, 8
// channels each, and a wave takes a group of as many heads of K, V or Q as fit
// at once (rows of 80 channels in 16 lanes each, with a butterfly in them,
// waste six: 14 Ki tokens of 30 heads 38 us against 30); what kind of rows a
// group holds is the same for the whole wave.  One group is in flight a wave (two
// change little: 30 heads of 80 channels 30.0 us against 29.5, 48 of 128 70.2
// against 72.3), and the rotation's table values stay in registers over all of
// them.
// What bounds it is vector instructions (some 600 a token at 30 heads of 80
// channels), then the bytes.
template <typename T, int FMT, typename CT>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a)
{
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t token = static_cast<int64_t>(blockIdx.x) * 4 + wave;
    if (token >= a.tokens) return;
    const int slice = blockIdx.y;
    const int lane = threadIdx.x & 63, sub = a.lanes.row(lane), in_row = lane - sub * a.lanes.n, d0 = 8 * in_row;
    const bool mine = sub < a.lanes.side;
    int ring[kRingSteps];
    if constexpr (FMT != PQ_KV_16) set_ring(a.lanes.n, lane, in_row, ring);
    const int64_t slot = a.slots[token];
    const bool stored = slot >= 0 && slot < a.num_slots;
    const int64_t page = stored ? slot >> a.page_log2 : 0;
    const int off = static_cast<int>(slot & ((1 << a.page_log2) - 1));
    const int64_t in_page = page * a.page_stride + static_cast<int64_t>(off) * a.token_stride;
    const T *xk = static_cast<const T *>(a.xk) + token * a.k_ts, *xv = static_cast<const T *>(a.xv) + token * a.v_ts;
    const T *xq = static_cast<const T *>(a.q) + token * a.q_ts;
    T *qo = static_cast<T *>(a.qo) + token * a.qo_ts;
    Turn turn;
    turn.on = 0;
    if (mine) load_turn(a, d0, a.table ? a.positions[token] : 0, turn);
    // half layout, whole runs: the partners come from memory
    const bool fetch = turn.on && a.half && a.rot % 16 == 0;
    const int partner = d0 < a.rot / 2 ? d0 + a.rot / 2 : d0 - a.rot / 2;

    const int kv_groups = a.kv_groups;
    for (int g = slice; g < a.groups; g += a.slices) {
        const int kind = g < kv_groups ? 0 : g < 2 * kv_groups ? 1 : 2;
        const int limit = kind == 2 ? a.q_heads : a.heads;
        const int h = (g - kind * kv_groups) * a.lanes.side + sub, head = min(h, limit - 1);
        const bool live = mine && h < limit;
        const T *src = (kind == 0 ? xk : kind == 1 ? xv : xq) + head * (kind == 0 ? a.k_hs : kind == 1 ? a.v_hs : a.q_hs);
        const Raw8<T> own = load_raw(src + d0);
        Raw8<T> other = own;
        if (fetch && kind != 1) other = load_raw(src + partner);
        float x[8];
        raw_to_f32<T>(own, x);
        if (kind != 1) apply_turn<T>(a, turn, other, src, d0, x);
        if (kind == 2) {
            // q_out may be q: a row is read and written by lanes of one wave,
            // which has all it needs of it by now
            if (live) store_f32<T, 8>(qo + head * a.qo_hs + d0, x);
            continue;
        }
        uint8_t *dst = (kind ? a.v : a.k) + in_page + head * a.head_stride;
        if constexpr (FMT == PQ_KV_16) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack16<CT>(x[2 * e], x[2 * e + 1]);
            if (live && stored) *reinterpret_cast<u32x4_a8 *>(dst + 2 * d0) = w;
        } else {
            constexpr float top = FMT == PQ_KV_8 ? 255.f : 15.f;
            float mn = x[0], mx = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) {
                mn = min_nan(mn, x[e]);
                mx = max_nan(mx, x[e]);
            }
            row_range(a.lanes.n, ring, mn, mx);
            const uint32_t sb = pack_bf16x2((mx - mn) * (1.f / top), mn);
            const float s = fmaxf(bf16_to_f32(sb & 0xFFFFu), kMinKvScale), z = bf16_to_f32(sb >> 16);
            const float inv = 1.f / s;
            float n[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = __builtin_rintf(__builtin_amdgcn_fmed3f((x[e] - z) * inv, 0.f, top));
            const u32x2 w = pack_codes<FMT>(n);
            if (live && stored) {
                if constexpr (FMT == PQ_KV_8) *reinterpret_cast<u32x2 *>(dst + d0) = w;
                else *reinterpret_cast<uint32_t *>(dst + d0 / 2) = w[0];
                if (d0 == 0)
                    (kind ? a.vp : a.kp)[((page * a.heads + head) << a.page_log2) + off] =
                        (__builtin_bit_cast(uint32_t, s) >> 16) | (sb & 0xFFFF0000u);
            }
        }
    }
}

template <typename T>
pq_status launch_append(const pq_kv_cache &c, const AppendArgs &a, hipStream_t s)
{
    const int64_t blocks = (a.tokens + 3) / 4;
    if (blocks > kMaxBlocks) return PQ_ERR_SHAPE;
    const dim3 g(static_cast<unsigned>(blocks), static_cast<unsigned>(a.slices)), b(256);
    if (c.format == PQ_KV_8) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_8, bf16_t>), g, b, 0, s, a);
    else if (c.format == PQ_KV_4) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_4, bf16_t>), g, b, 0, s, a);
    else if (c.dtype == PQ_BF16) hipLaunchKernelGGL((k_kv_append<T, PQ_KV_16, bf16_t>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_kv_append<T, PQ_KV_16, f16_t>), g, b, 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

// -------------------------------------------------------------------- load

// Output tokens of a block, and rows a thread has in flight.  Four contexts of
// 32 Ki tokens, 4 bits to bf16, 8 heads of 128 channels 139 us, 5 heads of 80
// 46 us; with 8 / 32 tokens 144 / 146 and 49 / 46; with 2 / 8 rows 154 / 137
// and 46 / 46, but 511 tokens of 3 heads 4.0 us with four rows, 4.6 with eight.
// The stores bound it: 537 MB of 651.
constexpr int kLoadTokens = 16, kLoadRows = 4;

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
    RowLanes lanes;
    int slices;                     // blocks per token tile
};

// A block takes 16 consecutive output tokens: 16 lanes find their pages (the
// sequence by a binary search of cu), then the block walks the tokens' rows.
template <typename T, int FMT, typename CT>
__global__ __launch_bounds__(256) void k_kv_load(LoadArgs a)
{
    __shared__ int s_page[kLoadTokens], s_off[kLoadTokens];
    const int slice = blockIdx.y;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kLoadTokens;
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
    const int sub = a.lanes.row(threadIdx.x), d0 = 8 * (static_cast<int>(threadIdx.x) - sub * a.lanes.n);
    const int side = 256 / a.lanes.n;               // rows the block takes at a time
    const bool mine = sub < side;
    const int n = static_cast<int>(a.tokens - t0 < kLoadTokens ? a.tokens - t0 : kLoadTokens) * a.heads;
    // K and V one after the other, each as one run of (token, head) rows:
    // side by side in the output, so that the block writes whole stretches.
    for (int base = slice * side * kLoadRows; base < 2 * n; base += a.slices * side * kLoadRows) {
        int64_t to[kLoadRows];
        bool v[kLoadRows], live[kLoadRows];
        u32x4 w[kLoadRows];
        uint32_t pair[kLoadRows];
#pragma unroll
        for (int k = 0; k < kLoadRows; ++k) {
            const int r = base + k * side + sub;
            live[k] = mine && r < 2 * n;
            v[k] = r >= n;
            const int rr = live[k] ? (v[k] ? r - n : r) : 0;
            const int j = rr / a.heads, h = rr - j * a.heads;
            const int page = s_page[j], off = s_off[j];
            w[k] = u32x4{0, 0, 0, 0};
            pair[k] = 0;                            // no source: z = s = 0
            to[k] = (t0 + j) * (v[k] ? a.vo_ts : a.ko_ts) + h * (v[k] ? a.vo_hs : a.ko_hs) + d0;
            if (live[k] && page >= 0) {
                const uint8_t *p = (v[k] ? a.v : a.k) + page * a.page_stride + h * a.head_stride +
                                   static_cast<int64_t>(off) * a.token_stride;
                if constexpr (FMT == PQ_KV_16) {
                    w[k] = *reinterpret_cast<const u32x4_a8 *>(p + 2 * d0);
                } else {
                    pair[k] = (v[k] ? a.vp : a.kp)[((static_cast<int64_t>(page) * a.heads + h) << a.page_log2) + off];
                    if constexpr (FMT == PQ_KV_8) {
                        const u32x2 x = *reinterpret_cast<const u32x2 *>(p + d0);
                        w[k][0] = x[0];
                        w[k][1] = x[1];
                    } else {
                        w[k][0] = *reinterpret_cast<const uint32_t *>(p + d0 / 2);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kLoadRows; ++k) {
            if (!live[k]) continue;
            float x[8];
            const float s = bf16_to_f32(pair[k] & 0xFFFFu), z = bf16_to_f32(pair[k] >> 16);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (FMT == PQ_KV_8) x[e] = z + s * static_cast<float>(w[k][e >> 2] >> (8 * (e & 3)) & 0xFFu);
                if constexpr (FMT == PQ_KV_4) x[e] = z + s * static_cast<float>(w[k][0] >> (4 * e) & 0xFu);
            }
            if constexpr (FMT == PQ_KV_16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack16<CT>(w[k][e], x[2 * e], x[2 * e + 1]);
            }
            store_f32<T, 8>(static_cast<T *>(v[k] ? a.vo : a.ko) + to[k], x);
        }
    }
}

template <typename T>
pq_status launch_load(const pq_kv_cache &c, const LoadArgs &a, dim3 g, hipStream_t s)
{
    const dim3 b(256);
    if (c.format == PQ_KV_8) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_8, bf16_t>), g, b, 0, s, a);
    else if (c.format == PQ_KV_4) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_4, bf16_t>), g, b, 0, s, a);
    else if (c.dtype == PQ_BF16) hipLaunchKernelGGL((k_kv_load<T, PQ_KV_16, bf16_t>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_kv_load<T, PQ_KV_16, f16_t>), g, b, 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
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
    a.lanes = RowLanes(c.dim);
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
    // Few tokens: a token's row groups go to several waves, as in the rotation
    // (16 tokens of 8 + 32 heads of 128 in 8 bits 4.1 us, unsliced 9.9).
    const int side = a.lanes.side;
    a.kv_groups = (c.heads + side - 1) / side;
    a.groups = 2 * a.kv_groups + (a.q_heads + side - 1) / side;
    int64_t slices = (2048 + tokens - 1) / tokens;
    if (slices > a.groups) slices = a.groups;
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
    a.lanes = RowLanes(c.dim);
    // Few tokens: the heads of a token tile go to several blocks (16 tokens of
    // 8 heads of 128 in 8 bits 4.4 us, unsliced 9.4).
    const int64_t tiles = (tokens + kLoadTokens - 1) / kLoadTokens;
    const int64_t per_round = kLoadRows * (256 / a.lanes.n);
    const int64_t rounds = (2 * kLoadTokens * static_cast<int64_t>(c.heads) + per_round - 1) / per_round;
    int64_t slices = (1024 + tiles - 1) / tiles;
    if (slices > rounds) slices = rounds;
    a.slices = static_cast<int>(slices);
    if (tiles > kMaxBlocks) return PQ_ERR_SHAPE;
    const dim3 blocks(static_cast<unsigned>(tiles), static_cast<unsigned>(slices));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == PQ_F32) return launch_load<float>(c, a, blocks, s);
    return dtype == PQ_BF16 ? launch_load<bf16_t>(c, a, blocks, s) : launch_load<f16_t>(c, a, blocks, s);
}

}  // extern "C"
