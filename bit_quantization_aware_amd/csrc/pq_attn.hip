// pq_attn.hip -- gfx950 kernels and C entry point of pq_attn_decode: attention
// of one new token per sequence over a paged key-value cache of 16-, 8- or
// 4-bit rows.
//
// Per query head, with x_t = scale log2(e) q . k^_t and a running reference m
// (one pass over the cache):
//   p_t = 2^(x_t - m),  l = sum p_t,  o = sum p_t v^_t,  out = o / l,
// and whenever m grows by d, l and o are multiplied by 2^-d.
//
// Affine rows k^ = z + s n leave the products as scalars of a token,
//   q . k^ = s (q . n) + z sum q,      sum p v^ = sum (p s) n + sum p z,
// so the matrix unit works on the bare codes: a code byte, zero-extended to
// 16 bits, is the f16 subnormal n 2^-24, which the f16 MFMA multiplies
// exactly.  One byte permute places two codes; nothing is converted.
//
// Layout.  A wave takes 32 tokens at a time.  S^T = K Q^T (rows: tokens,
// columns: the heads of a group, up to 16) leaves lane (head = lane % 16,
// kb = lane / 16) with the scores of tokens 4 kb + i of two 16-token tiles.
// Those eight are, in that order, the k-index run 8 kb .. 8 kb + 7 of the
// second product O^T = V^T P^T, for any order of tokens that P and V share:
// the probabilities go from accumulator to operand in their own registers.
// V^T needs eight tokens of one channel per lane; a lane loads 16 / 8 / 4-bit
// runs of the same channels of its eight tokens and transposes them with byte
// permutes.  No LDS and no cross-lane traffic in the loop but a maximum.
//
// Work split.  The cache is read once and every byte costs the same, so the
// 128-token tiles of all (sequence, head) rows are laid end to end and cut
// into equal shares, one per block, whatever the lengths are.  A row that lies
// in one share is written directly; the others leave (m, l, o) per share in
// the workspace and a second kernel joins them in order.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pq_kv_common.hpp"

namespace pq {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int kTile = 128;          // tokens of a scheduling unit: 32 per wave
constexpr int kMaxBatch = 1024;     // sequences of one launch (their tile counts sit in LDS)
constexpr int kMaxShares = 512;     // blocks of one launch

struct AttnArgs {
    const uint8_t *k, *v;
    const uint32_t *kp, *vp;
    int64_t page_stride, head_stride, num_pages;
    int token_stride, page_log2, heads, dim;
    const uint16_t *q;
    int64_t q_bs, q_hs;
    const int32_t *table;
    int64_t table_stride;
    int64_t max_tokens;             // max_pages * page_size
    const int32_t *lens;
    int batch, group, gtiles;       // query heads per cache head; 16-head tiles of a group
    int group_rows;                 // rows of a partial: min(group, 16)
    int64_t window;
    float scale_log2;               // scale * log2(e)
    uint16_t *out;
    int64_t out_bs, out_hs;
    float *lse;
    int q_heads;
    float *part_o;                  // [2 shares][group_rows][dim]
    float *part_ml;                 // [2 shares][group_rows][2]
    int shares;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Attended range of a sequence, its first token rounded down to a 16-token
// tile: pages are whole numbers of those.
struct Range {
    int64_t first, len, base;       // base = first & ~15
    __device__ __forceinline__ int64_t tiles() const { return len > first ? (len - base + kTile - 1) / kTile : 0; }
};

__device__ __forceinline__ Range range_of(const AttnArgs &a, int b)
{
    Range r;
    int64_t n = a.lens[b];
    n = n < 0 ? 0 : n;
    r.len = n < a.max_tokens ? n : a.max_tokens;
    r.first = a.window > 0 && r.len > a.window ? r.len - a.window : 0;
    r.base = r.first & ~static_cast<int64_t>(15);
    return r;
}

// pre[i] = tiles of sequences before i, pre[batch] their sum; 256 threads.
__device__ __forceinline__ void tile_prefix(const AttnArgs &a, int64_t *pre, int64_t *wave_sum)
{
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 256) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const int64_t n = b < a.batch ? range_of(a, b).tiles() : 0;
        int64_t s = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t up = __shfl_up(s, o);
            if ((threadIdx.x & 63) >= static_cast<unsigned>(o)) s += up;
        }
        if ((threadIdx.x & 63) == 63) wave_sum[threadIdx.x >> 6] = s;
        __syncthreads();
        int64_t at = before;
        for (int w = 0; w < 4; ++w) {
            if (w < static_cast<int>(threadIdx.x >> 6)) at += wave_sum[w];
            before += wave_sum[w];
        }
        if (b < a.batch) pre[b] = at + s - n;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[a.batch] = before;
    __syncthreads();
}

// Which partial a share writes for a row whose first tile is `row0`: the one
// for the row it starts inside (or at), or the one for the row it ends in.
__device__ __forceinline__ int64_t part_slot(int64_t share, int64_t row0, int64_t per_share)
{
    return 2 * share + (row0 > share * per_share ? 1 : 0);
}

// max / sum over the lanes that hold the same head (lane % 16).
__device__ __forceinline__ float head_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float head_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// QT: type of q and out (and of a 16-bit cache).  FMT: cache format.  DP: dim
// rounded up to 64, 128 or 256.
template <typename QT, int FMT, int DP>
struct Attn {
    static constexpr bool kRaw = FMT == PQ_KV_16;
    static constexpr bool kF16 = !kRaw || __is_same(QT, f16_t);   // operand type of both products
    using OT = typename std::conditional<kF16, f16_t, bf16_t>::type;
    static constexpr int KS = DP / 32;      // k steps of the first product
    static constexpr int E = DP / 16;       // channels of a lane in the second
    // Operand order of the channels of step s in lane group kb.  16-bit rows:
    // 32 s + 8 kb + j.  Codes: steps 2c, 2c + 1 share the 16-channel run
    // 64 c + 16 kb (16 or 8 bytes, one load).
    // The probabilities are scaled by 2^kShift, so that an f16 keeps 24 bits
    // of range below the largest before it becomes subnormal.
    static constexpr float kShift = kF16 ? 7.f : 0.f;
    static constexpr float kSlack = 8.f;    // m may lag behind the maximum by this much

    u32x4 q[KS];
    f32x4 o[E];
    float m, l, zsum;
    float c1, c2;                   // x = s_k (acc c1) + z_k c2   (raw: x = acc c1)

    __device__ __forceinline__ void load_q(const AttnArgs &a, int b, int kvh, int gt)
    {
        const int lane = threadIdx.x & 63, head = lane & 15, kb = lane >> 4;
        const int g = gt * 16 + head;
        const bool on = g < a.group;
        const uint16_t *row = a.q + b * a.q_bs + static_cast<int64_t>(kvh * a.group + (on ? g : 0)) * a.q_hs;
        float f[KS][8];
        float amax = 0.f, sum = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = kRaw ? 32 * s + 8 * kb : 64 * (s >> 1) + 16 * kb + 8 * (s & 1);
            u32x4 w = {0, 0, 0, 0};
            if (on && d < a.dim) w = *reinterpret_cast<const u32x4 *>(row + d);
            if constexpr (kRaw) {
                q[s] = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack16<QT>(w[e], f[s][2 * e], f[s][2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    amax = fmaxf(amax, fabsf(f[s][e]));
                    sum += f[s][e];
                }
            }
        }
        c1 = a.scale_log2;
        c2 = 0.f;
        if constexpr (!kRaw) {
            // q goes to f16 multiplied by the power of two that brings its
            // largest channel to [2^13, 2^14): exact for the channels of a
            // bf16 q down to 2^-26 of it, and off by 2^-33 of it below.
            amax = head_max(amax);
            sum = head_sum(sum);
            const int ex = static_cast<int>(__builtin_bit_cast(uint32_t, amax) >> 23) - 127;   // floor(log2 amax)
            const int up = amax > 0.f && ex < 128 ? 13 - ex : 0;
            // 2^up in two factors: up reaches 139
            const float u1 = __builtin_ldexpf(1.f, up / 2), u2 = __builtin_ldexpf(1.f, up - up / 2);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                float g8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) g8[e] = f[s][e] * u1 * u2;
                if constexpr (FMT == PQ_KV_8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[s][e] = pack16<f16_t>(g8[2 * e], g8[2 * e + 1]);
                } else {
                    // the order in which nibbles leave a word (k_operands): 0, 4, then
                    // 1, 5 sixteen times too large, then 2, 6 and 3, 7 likewise
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f16th = e & 1 ? 0.0625f : 1.f;
                        q[s][e] = pack16<f16_t>(g8[e] * f16th, g8[e + 4] * f16th);
                    }
                }
            }
            c1 = a.scale_log2 * __builtin_ldexpf(1.f, 24) / u1 / u2;
            c2 = a.scale_log2 * sum;
        }
    }

    __device__ __forceinline__ void clear()
    {
        m = -__builtin_inff();
        l = 0.f;
        zsum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // What a lane loads of 16 tokens for the first product.
    static constexpr int KC = kRaw ? KS : KS / 2;
    struct KTile {
        u32x4 w[KC];
        u32x4 par;                  // pairs of tokens 4 kb .. 4 kb + 3
    };
    struct VTile {
        uint32_t w[4][E / (kRaw ? 2 : FMT == PQ_KV_8 ? 4 : 8) ? E / (kRaw ? 2 : FMT == PQ_KV_8 ? 4 : 8) : 1];   // tokens 4 kb + j
        u32x4 par;
    };
    static constexpr int VW = sizeof(VTile::w[0]) / 4;

    // `row`: the page's first row of this head plus t0's offset (wave-uniform)
    static __device__ __forceinline__ void load_k(const AttnArgs &a, const uint8_t *row, const uint32_t *par, KTile &t)
    {
        const int lane = threadIdx.x & 63, kb = lane >> 4;
        const uint8_t *p = row + (lane & 15) * a.token_stride;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            if constexpr (kRaw) {
                const int d = min(32 * c + 8 * kb, a.dim - 8);          // past dim: any channel, q is 0 there
                t.w[c] = *reinterpret_cast<const u32x4_a8 *>(p + 2 * d);
            } else {
                const int d = min(64 * c + 16 * kb, a.dim - 16);
                if constexpr (FMT == PQ_KV_8) {
                    t.w[c] = *reinterpret_cast<const u32x4_a8 *>(p + d);
                } else {
                    const u32x2 w = *reinterpret_cast<const u32x2 *>(p + d / 2);
                    t.w[c] = u32x4{w[0], w[1], 0, 0};
                }
            }
        }
        if constexpr (!kRaw) t.par = *reinterpret_cast<const u32x4 *>(par + 4 * kb);
    }

    static __device__ __forceinline__ void load_v(const AttnArgs &a, const uint8_t *row, const uint32_t *par, VTile &t)
    {
        const int lane = threadIdx.x & 63, kb = lane >> 4;
        const int d = min((lane & 15) * E, a.dim - E);
        const uint8_t *p = row + 4 * kb * a.token_stride + (kRaw ? 2 * d : FMT == PQ_KV_8 ? d : d / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *r = p + j * a.token_stride;
            if constexpr (FMT == PQ_KV_4 && E == 4) {
                t.w[j][0] = *reinterpret_cast<const uint16_t *>(r);
            } else if constexpr (VW == 1) {
                t.w[j][0] = *reinterpret_cast<const uint32_t *>(r);
            } else if constexpr (VW == 2) {
                const u32x2 w = *reinterpret_cast<const u32x2_a4 *>(r);
                t.w[j][0] = w[0];
                t.w[j][1] = w[1];
            } else {
#pragma unroll
                for (int i = 0; i < VW / 4; ++i) {
                    const u32x4 w = reinterpret_cast<const u32x4_a8 *>(r)[i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) t.w[j][4 * i + e] = w[e];
                }
            }
        }
        if constexpr (!kRaw) t.par = *reinterpret_cast<const u32x4 *>(par + 4 * kb);
    }

    __device__ __forceinline__ f32x4 scores(const KTile &t) const
    {
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            if constexpr (kRaw) {
                c = mfma16<kF16>(t.w[i], q[i], c);
            } else if constexpr (FMT == PQ_KV_8) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    u32x4 f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = __builtin_amdgcn_perm(0, t.w[i][2 * s + (e >> 1)], e & 1 ? 0x0c030c02u : 0x0c010c00u);
                    c = mfma16<kF16>(f, q[2 * i + s], c);
                }
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t w = t.w[i][s], w8 = w >> 8;
                    const u32x4 f = {w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u};
                    c = mfma16<kF16>(f, q[2 * i + s], c);
                }
            }
        }
        return c;
    }

    // Operand of channel E * (lane % 16) + e: tokens 4 kb + j of tile a, then of b.
    static __device__ __forceinline__ u32x4 v_operand(const VTile &ta, const VTile &tb, int e)
    {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const VTile &t = i < 2 ? ta : tb;
            const int j = 2 * (i & 1);
            if constexpr (kRaw) {
                f[i] = __builtin_amdgcn_perm(t.w[j + 1][e >> 1], t.w[j][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
            } else if constexpr (FMT == PQ_KV_8) {
                const uint32_t b = e & 3;
                f[i] = __builtin_amdgcn_perm(t.w[j + 1][e >> 2], t.w[j][e >> 2], 0x0c000c00u | b | (b + 4) << 16);
            } else {
                const uint32_t b = (e >> 1) & 3, mask = e & 1 ? 0xF0F0F0F0u : 0x0F0F0F0Fu;   // odd channels: 16 n
                f[i] = __builtin_amdgcn_perm(t.w[j + 1][e >> 3] & mask, t.w[j][e >> 3] & mask, 0x0c000c00u | b | (b + 4) << 16);
            }
        }
        return f;
    }

    // 32 tokens.  `seen`: bit i for token 4 kb + i of tile a, bit 4 + i of b.
    __device__ __forceinline__ void step(const KTile &ka, const KTile &kb_, VTile &va, VTile &vb, unsigned seen, bool masked)
    {
        const f32x4 sa = scores(ka), sb = scores(kb_);
        float x[8], y[8];           // y = x + log2 s_v: the exponent of the weight of the codes
        float sv[8], zv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float acc = i < 4 ? sa[i & 3] : sb[i & 3];
            if constexpr (kRaw) {
                x[i] = y[i] = acc * c1;
            } else {
                const uint32_t kp = i < 4 ? ka.par[i & 3] : kb_.par[i & 3], vp = i < 4 ? va.par[i & 3] : vb.par[i & 3];
                sv[i] = __builtin_bit_cast(float, vp << 16);
                zv[i] = __builtin_bit_cast(float, vp & 0xFFFF0000u);
                x[i] = __builtin_fmaf(__builtin_bit_cast(float, kp << 16), acc * c1,
                                      __builtin_bit_cast(float, kp & 0xFFFF0000u) * c2);
                y[i] = x[i] + __builtin_amdgcn_logf(sv[i]);
            }
        }
        if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool on = seen >> i & 1;
                x[i] = on ? x[i] : -__builtin_inff();
                y[i] = on ? y[i] : -__builtin_inff();
                if constexpr (!kRaw) {
                    sv[i] = on ? sv[i] : 1.f;
                    zv[i] = on ? zv[i] : 0.f;
                } else {
                    // 0 times what lies there must be 0
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t &r = i < 4 ? va.w[i & 3][w] : vb.w[i & 3][w];
                        r = on ? r : 0u;
                    }
                }
            }
        }
        float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
        if (__ballot(top > m + kSlack)) {           // also the first tile: m is -inf
            const float mn = fmaxf(m, head_max(top));
            const float f = m == mn ? 1.f : exp2_fast(m - mn);
            m = mn;
            l *= f;
            zsum *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= f;
        }
        const float ref = (m == -__builtin_inff() ? 0.f : m) - kShift;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = exp2_fast(x[i] - ref);
            l += p;
            if constexpr (kRaw) {
                w[i] = p;
            } else {
                w[i] = p * sv[i];   // at most 2^(kShift + kSlack) by the choice of m
                zsum = __builtin_fmaf(p, zv[i], zsum);
            }
        }
        // The weights as the sum of two 16-bit values: rounded to one, each
        // token's share would be off by 2^-9 (bf16) and the output by as much
        // as its own rounding again.
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = pack16<OT>(w[2 * i], w[2 * i + 1]);
            float h0, h1;
            unpack16<OT>(hi[i], h0, h1);
            lo[i] = pack16<OT>(w[2 * i] - h0, w[2 * i + 1] - h1);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const u32x4 f = v_operand(va, vb, e);
            o[e] = mfma16<kF16>(f, hi, o[e]);
            o[e] = mfma16<kF16>(f, lo, o[e]);
        }
    }

    // What a unit of o[e] stands for.
    static __device__ __forceinline__ float o_unit(int e)
    {
        if constexpr (kRaw) return 1.f;
        else return FMT == PQ_KV_4 && (e & 1) ? 0x1p20f : 0x1p24f;
    }
};

template <typename QT, int FMT, int DP>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void k_attn_decode(AttnArgs a)
{
    using A = Attn<QT, FMT, DP>;
    constexpr int E = A::E;
    constexpr int kPad = DP + 4;
    __shared__ int64_t s_pre[kMaxBatch + 1];
    __shared__ int64_t s_wsum[4];
    __shared__ float s_m[4][16], s_l[4][16], s_z[4][16];
    __shared__ __align__(16) float s_o[4 * 16 * kPad];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, kb = lane >> 4, head = lane & 15;
    tile_prefix(a, s_pre, s_wsum);
    const int vheads = a.heads * a.gtiles;
    const int64_t total = s_pre[a.batch] * vheads;
    const int64_t per = (total + a.shares - 1) / a.shares;
    const int64_t begin = blockIdx.x * per, end = begin + per < total ? begin + per : total;
    if (begin >= end) return;
    int b = 0;
    {
        int hi = a.batch - 1;                       // last b whose rows start at or before `begin`
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (s_pre[mid] * vheads <= begin) b = mid;
            else hi = mid - 1;
        }
    }
    A st;
    for (int64_t at = begin; at < end;) {
        while (s_pre[b + 1] * vheads <= at) ++b;    // also past sequences without tiles
        const int64_t n = s_pre[b + 1] - s_pre[b];
        const int vh = static_cast<int>((at - s_pre[b] * vheads) / n);
        const int64_t row0 = s_pre[b] * vheads + vh * n;
        const int kvh = vh / a.gtiles, gt = vh - kvh * a.gtiles;
        const int64_t stop = row0 + n < end ? row0 + n : end;
        const Range r = range_of(a, b);
        const int32_t *pages = a.table + b * a.table_stride;
        st.load_q(a, b, kvh, gt);
        st.clear();
        // 64 pages' ids at a time, one a lane: 32 tiles of two 16-token halves
        for (int64_t j0 = at - row0; j0 < stop - row0; j0 += 32) {
            const int count = static_cast<int>(stop - row0 - j0 < 32 ? stop - row0 - j0 : 32);
            const int64_t t_lane = r.base + (j0 + (lane >> 1)) * kTile + wave * 32 + (lane & 1) * 16;
            int id = -1;
            if ((lane >> 1) < count && t_lane < r.len) {
                id = pages[t_lane >> a.page_log2];
                if (id < 0 || id >= a.num_pages) id = -1;
            }
            for (int j = 0; j < count; ++j) {
                const int64_t t = r.base + (j0 + j) * kTile + wave * 32;
                if (t >= r.len) break;
                typename A::KTile ka, kc;
                typename A::VTile va, vc;
                const int pa = __builtin_amdgcn_readlane(id, 2 * j), pb = __builtin_amdgcn_readlane(id, 2 * j + 1);
                const bool masked = pa < 0 || pb < 0 || t < r.first || t + 32 > r.len;
                const int in_page = (1 << a.page_log2) - 1;
                const int oa = static_cast<int>(t) & in_page, ob = static_cast<int>(t + 16) & in_page;
                const int64_t page_a = pa < 0 ? 0 : pa, page_b = pb < 0 ? 0 : pb;
                const int64_t ra = page_a * a.page_stride + kvh * a.head_stride + static_cast<int64_t>(oa) * a.token_stride;
                const int64_t rb = page_b * a.page_stride + kvh * a.head_stride + static_cast<int64_t>(ob) * a.token_stride;
                const int64_t qa = ((page_a * a.heads + kvh) << a.page_log2) + oa;
                const int64_t qb = ((page_b * a.heads + kvh) << a.page_log2) + ob;
                A::load_k(a, a.k + ra, a.kp + qa, ka);
                A::load_k(a, a.k + rb, a.kp + qb, kc);
                A::load_v(a, a.v + ra, a.vp + qa, va);
                A::load_v(a, a.v + rb, a.vp + qb, vc);
                unsigned seen = 0xFF;
                if (masked) {
                    seen = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t u = t + (i >> 2) * 16 + 4 * kb + (i & 3);
                        if ((i < 4 ? pa : pb) >= 0 && u >= r.first && u < r.len) seen |= 1u << i;
                    }
                }
                st.step(ka, kc, va, vc, seen, masked);
            }
        }
        // join the four waves
        __syncthreads();                            // the last row's s_o has been read
        const float l_all = head_sum(st.l), z_all = head_sum(st.zsum);
        if (kb == 0) {
            s_m[wave][head] = st.m;
            s_l[wave][head] = l_all;
            s_z[wave][head] = z_all;
        }
        __syncthreads();
        const float mx = fmaxf(fmaxf(s_m[0][head], s_m[1][head]), fmaxf(s_m[2][head], s_m[3][head]));
        const float f = st.m == mx ? 1.f : exp2_fast(st.m - mx);
        const int rows = min(16, a.group - gt * 16);
        if (head < rows) {
            float *so = s_o + (wave * 16 + head) * kPad;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<f32x4 *>(so + E * (4 * kb + i) + e) =
                        f32x4{st.o[e][i] * (f * A::o_unit(0)), st.o[e + 1][i] * (f * A::o_unit(1)),
                              st.o[e + 2][i] * (f * A::o_unit(0)), st.o[e + 3][i] * (f * A::o_unit(1))};
        }
        __syncthreads();
        const bool whole = row0 >= begin && row0 + n <= end;
        const int64_t slot = part_slot(blockIdx.x, row0, per);
        for (int i = tid * 4; i < rows * DP; i += 1024) {
            const int g = i / DP, d = i - g * DP;
            if (d >= a.dim) continue;
            const float M = fmaxf(fmaxf(s_m[0][g], s_m[1][g]), fmaxf(s_m[2][g], s_m[3][g]));
            float L = 0.f, Z = 0.f;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < 4; ++w) {
                const float fw = s_m[w][g] == M ? 1.f : exp2_fast(s_m[w][g] - M);
                L += s_l[w][g] * fw;
                Z += s_z[w][g] * fw;
                v += *reinterpret_cast<const f32x4 *>(s_o + (w * 16 + g) * kPad + d);
            }
            v += Z;
            if (whole) {
                // L is 0 only if every token lies in a hidden page
                const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
                const int64_t hq = static_cast<int64_t>(kvh) * a.group + gt * 16 + g;
                u32x2 w2 = {pack16<QT>(v[0] * inv, v[1] * inv), pack16<QT>(v[2] * inv, v[3] * inv)};
                *reinterpret_cast<u32x2 *>(a.out + b * a.out_bs + hq * a.out_hs + d) = w2;
                if (d == 0 && a.lse)
                    a.lse[static_cast<int64_t>(b) * a.q_heads + hq] =
                        L == 0.f ? -__builtin_inff() : (M - A::kShift + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
            } else {
                *reinterpret_cast<f32x4 *>(a.part_o + (slot * a.group_rows + g) * a.dim + d) = v;
                if (d == 0) {
                    a.part_ml[(slot * a.group_rows + g) * 2] = M - A::kShift;
                    a.part_ml[(slot * a.group_rows + g) * 2 + 1] = L;
                }
            }
        }
        at = stop;
    }
}

// Joins the shares of the rows that span several, in order, and writes the
// rows without a token.  One block per (sequence, cache head, head tile).
template <typename QT>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a)
{
    __shared__ int64_t s_pre[kMaxBatch + 1];
    __shared__ int64_t s_wsum[4];
    tile_prefix(a, s_pre, s_wsum);
    const int vheads = a.heads * a.gtiles;
    const int64_t total = s_pre[a.batch] * vheads;
    const int64_t per = (total + a.shares - 1) / a.shares;
    const int b = blockIdx.x / vheads, vh = blockIdx.x - b * vheads;
    const int kvh = vh / a.gtiles, gt = vh - kvh * a.gtiles;
    const int rows = min(16, a.group - gt * 16);
    const int64_t n = s_pre[b + 1] - s_pre[b];
    const int64_t row0 = s_pre[b] * vheads + vh * n;
    const int64_t first = n ? row0 / per : 0, last = n ? (row0 + n - 1) / per : -1;
    if (first == last) return;
    for (int i = threadIdx.x * 4; i < rows * a.dim; i += 1024) {
        const int g = i / a.dim, d = i - g * a.dim;
        float M = -__builtin_inff(), L = 0.f;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int64_t s = first; s <= last; ++s)
            M = fmaxf(M, a.part_ml[(part_slot(s, row0, per) * a.group_rows + g) * 2]);
        for (int64_t s = first; s <= last; ++s) {
            const int64_t at = part_slot(s, row0, per) * a.group_rows + g;
            const float ms = a.part_ml[at * 2];
            const float f = ms == M ? 1.f : exp2_fast(ms - M);
            L = __builtin_fmaf(a.part_ml[at * 2 + 1], f, L);
            const f32x4 p = *reinterpret_cast<const f32x4 *>(a.part_o + at * a.dim + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(p[e], f, v[e]);
        }
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
        const int64_t hq = static_cast<int64_t>(kvh) * a.group + gt * 16 + g;
        u32x2 w2 = {pack16<QT>(v[0] * inv, v[1] * inv), pack16<QT>(v[2] * inv, v[3] * inv)};
        *reinterpret_cast<u32x2 *>(a.out + b * a.out_bs + hq * a.out_hs + d) = w2;
        if (d == 0 && a.lse)
            a.lse[static_cast<int64_t>(b) * a.q_heads + hq] =
                L == 0.f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
    }
}

template <typename QT, int FMT>
void launch_dim(const AttnArgs &a, hipStream_t s)
{
    const dim3 g(static_cast<unsigned>(a.shares)), t(256);
    if (a.dim <= 64) hipLaunchKernelGGL((k_attn_decode<QT, FMT, 64>), g, t, 0, s, a);
    else if (a.dim <= 128) hipLaunchKernelGGL((k_attn_decode<QT, FMT, 128>), g, t, 0, s, a);
    else hipLaunchKernelGGL((k_attn_decode<QT, FMT, 256>), g, t, 0, s, a);
}

template <typename QT>
pq_status launch_attn(int format, const AttnArgs &a, hipStream_t s)
{
    if (format == PQ_KV_16) launch_dim<QT, PQ_KV_16>(a, s);
    else if (format == PQ_KV_8) launch_dim<QT, PQ_KV_8>(a, s);
    else launch_dim<QT, PQ_KV_4>(a, s);
    if (hipGetLastError() != hipSuccess) return PQ_ERR_HIP;
    hipLaunchKernelGGL(k_attn_join<QT>, dim3(static_cast<unsigned>(a.batch * a.heads * a.gtiles)), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

int64_t attn_workspace(int dim, int group)
{
    const int64_t rows = group < 16 ? group : 16;
    return 2 * kMaxShares * rows * (dim + 4) * 4;   // o, then m and l (padded to 16 bytes)
}

}  // namespace
}  // namespace pq

extern "C" {

int64_t pq_attn_decode_workspace_bytes(const pq_kv_cache *cache, int64_t batch, int64_t q_heads)
{
    using namespace pq;
    if (kv_cache_status(cache) != PQ_OK || batch < 0 || q_heads < 1 || q_heads % cache->heads) return -1;
    if (batch == 0) return 0;
    return attn_workspace(cache->dim, static_cast<int>(q_heads / cache->heads));
}

pq_status pq_attn_decode(const pq_kv_cache *cache, int q_dtype, int64_t batch, int64_t q_heads, const void *q,
                         int64_t q_batch_stride, int64_t q_head_stride, const int32_t *block_table,
                         int64_t table_stride, int64_t max_pages, const int32_t *lens, double scale, int64_t window,
                         int64_t max_len, void *out, int64_t out_batch_stride, int64_t out_head_stride, float *lse,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace pq;
    const pq_status st = kv_cache_status(cache);
    if (st != PQ_OK) return st;
    const pq_kv_cache &c = *cache;
    if (q_dtype != PQ_BF16 && q_dtype != PQ_F16) return PQ_ERR_MODE;
    if (c.format == PQ_KV_16 && c.dtype != q_dtype) return PQ_ERR_MODE;
    if (batch < 0 || batch > INT32_MAX || q_heads < 1 || q_heads > 65535 || q_heads % c.heads) return PQ_ERR_SHAPE;
    if (max_pages < 0 || max_pages > (int64_t(1) << 31) / c.page_size || table_stride < 0) return PQ_ERR_SHAPE;
    if (((q_batch_stride | q_head_stride | out_batch_stride | out_head_stride) & 7) != 0) return PQ_ERR_SHAPE;
    if (!std::isfinite(scale) || window < 0 || max_len < 0) return PQ_ERR_ARG;
    if (batch == 0) return PQ_OK;
    if (!q || !out || !lens || (!block_table && max_pages > 0) || !workspace) return PQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return PQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(lse)) % 4)
        return PQ_ERR_ALIGN;
    const int group = static_cast<int>(q_heads / c.heads);
    if (workspace_bytes < attn_workspace(c.dim, group)) return PQ_ERR_ARG;
    AttnArgs a = {};
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
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride;
    a.q_hs = q_head_stride;
    a.table = block_table;
    a.table_stride = table_stride;
    a.max_tokens = max_pages * c.page_size;
    a.lens = lens;
    a.group = group;
    a.gtiles = (group + 15) / 16;
    a.group_rows = group < 16 ? group : 16;
    a.window = window;
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634074);
    a.out = static_cast<uint16_t *>(out);
    a.out_bs = out_batch_stride;
    a.out_hs = out_head_stride;
    a.lse = lse;
    a.q_heads = static_cast<int>(q_heads);
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + static_cast<int64_t>(2) * kMaxShares * a.group_rows * c.dim;
    int64_t longest = max_len > 0 && max_len < a.max_tokens ? max_len : a.max_tokens;
    if (window > 0 && longest > window + 15) longest = window + 15;   // its first tile may start 15 tokens early
    const int64_t tiles = (longest + kTile - 1) / kTile;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    for (int64_t b0 = 0; b0 < batch; b0 += kMaxBatch) {
        AttnArgs x = a;
        x.batch = static_cast<int>(batch - b0 < kMaxBatch ? batch - b0 : kMaxBatch);
        x.q += b0 * q_batch_stride;
        x.out += b0 * out_batch_stride;
        if (x.lse) x.lse += b0 * q_heads;
        if (x.table) x.table += b0 * table_stride;
        x.lens += b0;
        int64_t shares = static_cast<int64_t>(x.batch) * c.heads * a.gtiles * tiles;
        x.shares = static_cast<int>(shares < 1 ? 1 : shares > kMaxShares ? kMaxShares : shares);
        const pq_status r = q_dtype == PQ_BF16 ? launch_attn<bf16_t>(c.format, x, s) : launch_attn<f16_t>(c.format, x, s);
        if (r != PQ_OK) return r;
    }
    return PQ_OK;
}

}  // extern "C"
