// pq_attn.hip -- gfx950 kernels and C entry point of pq_attn_decode: attention
// of one new token per sequence over a paged key-value cache of 16-, 8- or
// 4-bit rows.
//
// Per query head, with x_t = scale log2(e) q . k^_t and a running whole-numbered reference m
// (one pass over the cache):
//   p_t = 2^(x_t - m),  l = sum p_t,  o = sum p_t v^_t,  out = o / l,
// and whenever m grows by d, l and o are multiplied by 2^-d.
//
// Affine rows k^ = z + s n leave the products as scalars of a token; with the
// middle code c,
//   q . k^ = s (q . (n - c)) + (z + s c) sum q,
//   sum p v^ = sum (p s) n + sum p z,
// so the matrix unit works on the bare codes: a code byte, zero-extended to
// 16 bits, is the f16 subnormal n 2^-24, which the f16 MFMA multiplies
// exactly.  One byte permute places two codes; nothing is converted.  4-bit
// codes stand as 16 n: the matrix unit lines the terms of a sum up by their
// exponents, a subnormal's counts as the smallest normal's, and what bare
// nibbles leave below is cut off, always downwards (lse off by 3e-6 of its
// size instead of 1e-7, at 2 % less time over 64 ragged contexts).
//
// The first product starts from -c sum q, so that only the small difference
// is rounded afterwards.  In the second every other token is taken from the
// other end, v^ = (z + s Q) - s (Q - n): both sums then stay near the size of
// the result, where sums of n and of z alone would grow with the number of
// tokens and leave the output as a small difference (f16 output over some
// 10^4 tokens off by 1e-3 instead of 2e-4).
//
// Layout.  S^T = K Q^T (rows: 16 tokens, columns: 16 heads) leaves lane
// (column = lane % 16, kb = lane / 16) with the scores of tokens 4 kb + i.
// Those of two tiles are, in that order, the k-index run 8 kb .. 8 kb + 7 of
// the second product O^T = V^T P^T, for any order of tokens that P and V
// share: the probabilities go from accumulator to operand in their own
// registers.  V^T needs eight tokens of one channel per lane; a lane loads
// runs of the same channels of its eight tokens and transposes them with byte
// permutes.  No LDS and no cross-lane traffic in the loop but a maximum.
//
// Groups of few heads would leave most columns, and with them most lanes of
// the softmax, without work.  With R = 2 (4 bits) the columns hold R copies of
// the group's heads; a wave takes R blocks of 32 tokens at a time and copy r
// of the columns keeps block r only (its own m, l and o), so that every lane
// works on tokens of its own: the softmax costs 1 / R.
//
// Work split.  The cache is read once and every byte costs the same, so the
// steps of all (sequence, head) rows, each row with kRowCost more for its
// beginning and end, are laid end to end and cut into equal shares, one per
// block, whatever the lengths are.  A row that lies in one
// share is written directly; of the others each share leaves (m, l, o) in the
// workspace, and a second kernel joins them, in order.  Short rows are not
// split: one block each and no second kernel.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "pq_kv_common.hpp"

namespace pq {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxBatch = 1024;     // sequences of one launch (their step counts sit in LDS)
// Blocks of one launch: two per CU.  (Of over 128 channels in 16 or 8 bits the
// registers let a CU take one; it then takes its two one after the other.)
constexpr int kMaxShares = 512;
constexpr int kWaves = 4;
// What a row costs a share beyond its steps (first loads, joining the waves,
// a last round with idle waves), in steps of one wave.  64 ragged contexts of
// 80 channels in 4 bits take 37.6 us with 8, 39.3 with 4, 38.0 with 12.
constexpr int kRowCost = 8;

struct AttnArgs {
    const uint8_t *k, *v;
    const uint32_t *kp, *vp;
    int64_t page_stride, head_stride, num_pages;
    int token_stride, page_log2, heads, dim;
    const uint16_t *q;
    int64_t q_bs, q_hs;
    const int32_t *table;
    int64_t table_stride;
    int max_tokens;                 // most that max_pages and max_len allow, at most 2^30
    const int32_t *lens;
    int batch, group, gtiles;       // query heads per cache head; 16-head tiles of a group
    int group_rows;                 // rows of a partial: min(group, 16)
    int window;                     // 0: everything
    float scale_log2;               // scale * log2(e)
    uint16_t *out;
    int64_t out_bs, out_hs;
    float *lse;
    int q_heads;
    float *part_o;                  // [2 kMaxShares][group_rows][dim]
    f32x2 *part_ml;                 // [2 kMaxShares][group_rows] (m, l)
    int2 *spans;                    // [batch][heads][gtiles]: a row's first partial and last share
    int shares;                     // 0: one block per row
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// What sums with the reference `from` are multiplied by to have the reference
// `to`; not 0, so that an infinite sum stays one.
__device__ __forceinline__ float rescale(float from, float to)
{
    return from == to ? 1.f : __builtin_elementwise_maximum(exp2_fast(from - to), 0x1p-126f);
}

// Attended range of a sequence, its first token rounded down to a 16-token
// tile: pages are whole numbers of those.
struct Range {
    int first, len, base;           // base = first & ~15
    __device__ __forceinline__ int steps(int unit) const { return len > first ? (len - base + unit - 1) / unit : 0; }
};

__device__ __forceinline__ Range range_of(const AttnArgs &a, int len)
{
    Range r;
    r.len = min(max(len, 0), a.max_tokens);
    r.first = a.window > 0 && r.len > a.window ? r.len - a.window : 0;
    r.base = r.first & ~15;
    return r;
}

// lens[i] = clamped lengths; pre[i] = steps and row costs of one head of the
// sequences before i, pre[batch] their sum; 256 threads.
__device__ __forceinline__ void step_prefix(const AttnArgs &a, int unit, int *lens, int *pre, int *wave_sum)
{
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 256) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const Range r = range_of(a, b < a.batch ? a.lens[b] : 0);
        const int n = r.len > r.first ? r.steps(unit) + kRowCost : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(s, o);
            if ((threadIdx.x & 63) >= static_cast<unsigned>(o)) s += up;
        }
        if ((threadIdx.x & 63) == 63) wave_sum[threadIdx.x >> 6] = s;
        __syncthreads();
        int at = before;
        for (int w = 0; w < kWaves; ++w) {
            if (w < static_cast<int>(threadIdx.x >> 6)) at += wave_sum[w];
            before += wave_sum[w];
        }
        if (b < a.batch) {
            pre[b] = at + s - n;
            lens[b] = r.len;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[a.batch] = before;
    __syncthreads();
}

// The cut of the line of steps and row costs into shares: the first `more`
// have `each` + 1 of them, the others `each`.
struct Cut {
    int each, more;
    __device__ __forceinline__ int begin(int share) const { return share * each + min(share, more); }
    __device__ __forceinline__ int share_of(int step) const
    {
        const int wide = more * (each + 1);
        return step < wide ? step / (each + 1) : more + (step - wide) / each;
    }
    // Which partial a share writes for the row that starts at `row0`: that of
    // the row it begins in, or that of the row it ends in.
    __device__ __forceinline__ int slot(int share, int row0) const { return 2 * share + (row0 > begin(share) ? 1 : 0); }
};

// max / sum over the lanes of a column (lane % 16).
__device__ __forceinline__ float column_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float column_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Loads at a 32-bit offset of the lane from a wave-uniform address: buffer
// loads, whose resource is made from the address in scalar registers.  From a
// pointer the compiler adds the two in every lane, 64 bits wide, 24 times a
// step (the offsets' extensions leave the loop, and with them the proof that
// they are 32-bit ones).  `bytes`: what may be read there.
struct Resource {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ Resource(const uint8_t *p, int bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, bytes, 0x00027000)) {}     // raw, 32-bit data
    template <bool NT>
    __device__ __forceinline__ u32x4 load16(uint32_t at) const
    {
        return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, NT ? 2 : 0);     // 2: non-temporal
    }
    template <bool NT>
    __device__ __forceinline__ u32x2 load8(uint32_t at) const
    {
        return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, NT ? 2 : 0);
    }
    __device__ __forceinline__ uint32_t load4(uint32_t at) const { return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0); }
    __device__ __forceinline__ uint32_t load2(uint32_t at) const
    {
        return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
    }
};

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// QT: type of q and out (and of a 16-bit cache).  FMT: cache format.  DP: dim
// rounded up to 64, 96 (4 bits), 128 or 256.  R: copies of the heads in the columns.  NT:
// the cache is read past the caches (launch_one).
template <typename QT, int FMT, int DP, int R, bool NT>
struct Attn {
    static constexpr bool kRaw = FMT == PQ_KV_16;
    static constexpr bool kF16 = !kRaw || __is_same(QT, f16_t);   // operand type of both products
    // The weights p (or p s) enter the second product as several 16-bit values,
    // each carrying the remainder of the one before: rounded to one (2^-9 off
    // in bf16, 2^-12 in f16) they would add as much to the output's error as
    // its own rounding.  Two hold 22 bits in f16, three hold all 24 in bf16.
    // The matrix unit has the room.  Of 16-bit rows they are cut off, never
    // rounded up, and not 0 where the weight is not: an infinite value then
    // meets no 0 and no negative remainder, and the sum is infinite too.  (An
    // f16 weight below 2^-24 has no such value: infinity by 0 is NaN there.)
    static constexpr int kPieces = kF16 ? 2 : 3;
    static constexpr int kUnit = 32 * R;    // tokens of a step
    static constexpr int kCols = 16 / R;    // heads of a tile
    static constexpr int KS = DP / 32;      // k steps of the first product
    static constexpr int VD = DP == 96 ? 128 : DP;  // channels of the second: a lane's E are whole words of codes
    static constexpr int E = VD / 16;       // in runs of kRun
    static constexpr int kRun = kRaw && E == 16 ? 8 : E;    // (one 16-byte load each, side by side over the lanes)
    // Words of a lane per 16 tokens: K in KC runs of KW words (16-bit rows: 8
    // channels of step s at 32 s + 8 kb; codes: 16 channels at 64 c + 16 kb,
    // which are steps 2c and 2c + 1; of 96 the last 32: 8 at 64 + 8 kb), V in
    // VW words per token.
    static constexpr int KC = kRaw ? KS : (KS + 1) / 2, KW = FMT == PQ_KV_4 ? 2 : 4;
    static constexpr int VW = kRaw ? E / 2 : FMT == PQ_KV_8 ? E / 4 : E >= 8 ? E / 8 : 1;
    // The weights are scaled by 2^kShift, so that an f16 keeps 22 octaves
    // below the largest before it becomes subnormal; m may lag behind the
    // maximum by kSlack, so that it seldom moves.
    static constexpr float kShift = kF16 ? 7.f : 0.f, kUnscale = kF16 ? 0x1p-7f : 1.f, kSlack = 8.f;

    u32x4 q[KS];
    f32x4 o[E];
    float m, l, zsum;
    float ref, limit;               // m - kShift; the y that moves m
    float c1, c2;                   // x = s_k (acc c1) + (z_k + s_k c) c2   (16-bit rows: x = acc c1)
    f32x4 acc0;                     // start of the first product
    uint32_t k[R][2][KC][KW], v[R][2][4][VW];   // two 16-token tiles per block; V: tokens 4 kb + j
    u32x4 kpar[2], vpar[2];         // pairs of tokens 4 kb + i of the lane's own block

    static __device__ __forceinline__ int column() { return threadIdx.x & 15; }
    static __device__ __forceinline__ int kb() { return (threadIdx.x & 63) >> 4; }
    static __device__ __forceinline__ int copy() { return column() / kCols; }

    // The heads' channels as they lie in memory (set_q turns them into operands).
    __device__ __forceinline__ void load_q(const AttnArgs &a, int b, int kvh, int gt)
    {
        const int g = gt * 16 + column() % kCols;
        const bool on = g < a.group;
        const uint16_t *row = a.q + b * a.q_bs + static_cast<int64_t>(kvh * a.group + (on ? g : 0)) * a.q_hs;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const bool single = kRaw || (KS % 2 && s == KS - 1);     // a step of its own, not half of a 64-channel run
            const int d = single ? 32 * s + 8 * kb() : 64 * (s >> 1) + 16 * kb() + 8 * (s & 1);
            q[s] = u32x4{0, 0, 0, 0};
            if (on && d < a.dim) q[s] = *reinterpret_cast<const u32x4 *>(row + d);
        }
    }

    __device__ __forceinline__ void set_q(const AttnArgs &a)
    {
        c1 = a.scale_log2;
        c2 = 0.f;
        acc0 = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (!kRaw) {
            float amax = 0.f, sum = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x, y;
                    unpack16<QT>(q[s][e], x, y);
                    amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
                    sum += x + y;
                }
            sum = column_sum(sum);
            // q goes to f16 multiplied by the power of two that brings its
            // largest channel to [2^13, 2^14): exact for the channels of a
            // bf16 q down to 2^-26 of it, and off by 2^-33 of it below.
            amax = column_max(amax);
            const int ex = static_cast<int>(__builtin_bit_cast(uint32_t, amax) >> 23) - 127;   // floor(log2 amax)
            const int up = amax > 0.f && ex < 128 ? 13 - ex : 0;
            // 2^up in two factors: up reaches 139
            const float u1 = __builtin_ldexpf(1.f, up / 2), u2 = __builtin_ldexpf(1.f, up - up / 2);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                float g8[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack16<QT>(q[s][e], g8[2 * e], g8[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) g8[e] = g8[e] * u1 * u2;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (FMT == PQ_KV_8) {
                        q[s][e] = pack16<f16_t>(g8[2 * e], g8[2 * e + 1]);
                    } else {
                        // the order in which nibbles leave a word (scores): 0, 4, then 1, 5, ...
                        q[s][e] = pack16<f16_t>(g8[e], g8[e + 4]);
                    }
                }
            }
            const float start = -128.f * 0x1p-24f * (sum * u1 * u2);    // nibbles stand as 16 n
            acc0 = f32x4{start, start, start, start};
            c1 = a.scale_log2 * (FMT == PQ_KV_8 ? 0x1p24f : 0x1p20f) / u1 / u2;
            c2 = a.scale_log2 * sum;
        }
    }

    __device__ __forceinline__ void clear()
    {
        m = limit = -__builtin_inff();
        ref = -kShift;
        l = 0.f;
        zsum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // Byte offsets of the lane's loads from a 16-token tile's first row, and
    // the tile's bytes.  Channels past dim meet a q of 0: any codes do there,
    // but 16-bit values may be infinite, so those come as 0, from an offset
    // that lies behind every tile (a buffer load gives 0 there).
    static constexpr uint32_t kNowhere = 0x80000000u;
    uint32_t k_off, k_last, k_half, v_off, v_step, v_second;
    int tile_bytes;

    __device__ __forceinline__ void set_offsets(const AttnArgs &a)
    {
        const uint32_t row = column() * a.token_stride;
        // run c of K lies 16 * 4 (4-bit: 8 * 4) bytes after run c - 1, the last one inside the row
        const uint32_t run = KW * 4, row_bytes = kRaw ? 2 * a.dim : FMT == PQ_KV_8 ? a.dim : a.dim / 2;
        k_off = row + kb() * run;
        k_last = row + row_bytes - run;
        k_half = row + min(32 + 4 * kb(), static_cast<int>(row_bytes) - 4);      // 4 bits: 8 channels at 64 + 8 kb
        const uint32_t d = min(column() * kRun, a.dim - kRun);
        v_second = 2 * (min(128u + column() * kRun, static_cast<uint32_t>(a.dim - kRun)) - d);
        v_off = 4 * kb() * a.token_stride + (kRaw ? 2 * d : FMT == PQ_KV_8 ? d : d / 2);
        v_step = a.token_stride;
        tile_bytes = 15 * a.token_stride + row_bytes;
    }

    __device__ __forceinline__ void load_k(int r, int tile, const uint8_t *tile_row)
    {
        const Resource rows(tile_row, tile_bytes);
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t at = k_off + c * (KW * 16);
            if constexpr (!kRaw) at = min(at, k_last);
            else if (DP == 64 || c >= KC / 2) at = at <= k_last ? at : kNowhere;    // dim > DP / 2 but for DP = 64
            if constexpr (DP == 96) {
                if (c == KC - 1) {
                    k[r][tile][c][0] = rows.load4(k_half);
                    break;
                }
            }
            if constexpr (KW == 2) {
                const u32x2 w = rows.template load8<NT>(at);
                k[r][tile][c][0] = w[0];
                k[r][tile][c][1] = w[1];
            } else {
                const u32x4 w = rows.template load16<NT>(at);
#pragma unroll
                for (int e = 0; e < 4; ++e) k[r][tile][c][e] = w[e];
            }
        }
    }

    __device__ __forceinline__ void load_v(int r, int tile, const uint8_t *tile_row)
    {
        const Resource rows(tile_row, tile_bytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t t = v_off + j * v_step;
            uint32_t(&w)[VW] = v[r][tile][j];
            if constexpr (FMT == PQ_KV_4 && E == 4) {
                w[0] = rows.load2(t);
            } else if constexpr (VW == 1) {
                w[0] = rows.load4(t);
            } else if constexpr (VW == 2) {
                const u32x2 x = rows.template load8<NT>(t);
                w[0] = x[0];
                w[1] = x[1];
            } else {
#pragma unroll
                for (int i = 0; i < VW / 4; ++i) {
                    // a second run (16-bit rows of over 128 channels) lies 128 channels on
                    const u32x4 x = rows.template load16<NT>(i ? t + v_second : t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[4 * i + e] = x[e];
                }
            }
        }
    }

    __device__ __forceinline__ f32x4 scores(int r, int tile) const
    {
        f32x4 sum = acc0;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const uint32_t(&w)[KW] = k[r][tile][i];
            if constexpr (kRaw) {
                sum = mfma16<kF16>(u32x4{w[0], w[1], w[2], w[3]}, q[i], sum);
            } else {
#pragma unroll
                for (int s = 0; s < 2 && 2 * i + s < KS; ++s) {
                    u32x4 f;
                    if constexpr (FMT == PQ_KV_8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[e] = __builtin_amdgcn_perm(0, w[2 * s + (e >> 1)], e & 1 ? 0x0c030c02u : 0x0c010c00u);
                    } else {
                        const uint32_t w0 = w[s];
                        f = u32x4{w0 << 4 & 0x00F000F0u, w0 & 0x00F000F0u, w0 >> 4 & 0x00F000F0u, w0 >> 8 & 0x00F000F0u};
                    }
                    sum = mfma16<kF16>(f, q[2 * i + s], sum);
                }
            }
        }
        return sum;
    }

    // Operand of channel(column, e): tokens 4 kb + j of the block's first tile,
    // then of its second; of the odd ones Q - n.
    __device__ __forceinline__ u32x4 v_operand(int r, int e) const
    {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t *w0 = v[r][i >> 1][2 * (i & 1)], *w1 = v[r][i >> 1][2 * (i & 1) + 1];
            if constexpr (kRaw) {
                f[i] = __builtin_amdgcn_perm(w1[e >> 1], w0[e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
            } else if constexpr (FMT == PQ_KV_8) {
                const uint32_t b = e & 3;
                f[i] = __builtin_amdgcn_perm(~w1[e >> 2], w0[e >> 2], 0x0c000c00u | b | (b + 4) << 16);
            } else {
                const uint32_t b = (e >> 1) & 3, up = e & 1 ? 0 : 4, nibble = 0xF0F0F0F0u;
                const uint32_t n1 = __builtin_amdgcn_bitop3_b32(w1[e >> 3] << up, nibble, 0, 0x0C);    // ~a & b
                f[i] = __builtin_amdgcn_perm(n1, w0[e >> 3] << up & nibble, 0x0c000c00u | b | (b + 4) << 16);
            }
        }
        return f;
    }

    // First product of all blocks; the lane keeps the scores of its own.
    __device__ __forceinline__ void first_product(float (&x)[8]) const
    {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const f32x4 sa = scores(r, 0), sb = scores(r, 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = i < 4 ? sa[i & 3] : sb[i & 3];
                x[i] = r == 0 || copy() == r ? s : x[i];
            }
        }
    }

    // Scores to weights, as operands.  `seen`: bit i for token 4 kb + i of the
    // own block's first tile, bit 4 + i of its second.  Everything is relative
    // to `ref` = m - kShift, which goes in with the constant of a token's row.
    __device__ __forceinline__ void softmax(float (&x)[8], unsigned seen, bool masked, u32x4 (&weights)[kPieces])
    {
        float y[8];                 // x + log2 of s_v's size (+ kBias): the exponent of the weight of the codes
        float sv[8], zv[8];
        constexpr float kBias = kRaw ? 0.f : 127.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kRaw) {
                y[i] = x[i] = __builtin_fmaf(x[i], c1, -ref);
            } else {
                constexpr float mid = FMT == PQ_KV_8 ? 128.f : 8.f;
                const uint32_t kw = kpar[i >> 2][i & 3], vw = vpar[i >> 2][i & 3];
                const float sk = __builtin_bit_cast(float, kw << 16), zk = __builtin_bit_cast(float, kw & 0xFFFF0000u);
                sv[i] = __builtin_bit_cast(float, vw << 16);
                zv[i] = __builtin_bit_cast(float, vw & 0xFFFF0000u);
                x[i] = __builtin_fmaf(sk, x[i] * c1, __builtin_fmaf(__builtin_fmaf(sk, mid, zk), c2, -ref));
                // How large the row's values count: its scale; at least 2^-60,
                // also where the row was never written and its scale is 0, and
                // 2^-40 of its zero, so that neither p nor p z overflows.  (The
                // elementwise maximum is one operation for three values; fmaxf
                // brings its operands into canonical form first.)
                const float size = __builtin_elementwise_maximum(
                    __builtin_elementwise_maximum(fabsf(sv[i]), fabsf(zv[i]) * 0x1p-40f), kMinKvScale);
                // the bits of a positive float are 2^23 (127 + log2) to within 0.09 octaves
                y[i] = __builtin_fmaf(static_cast<float>(__builtin_bit_cast(uint32_t, size)), 0x1p-23f, x[i]);
            }
        }
        if (masked) {
            asm volatile("");                       // a branch: not selects in every step
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
                    for (int w = 0; w < VW; ++w) v[0][i >> 2][i & 3][w] = on ? v[0][i >> 2][i & 3][w] : 0u;
                }
            }
        }
        const float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
        if (__ballot(top > limit)) {                // also the first step: limit is -inf
            // A whole number, so that the shift and the factors of l and o are
            // exact, however far below 0 rows of the smallest scale bring it.
            const float mn = floorf(fmaxf(m, column_max(top) + (ref - kBias)));
            const float f = rescale(m, mn);
            const float next = mn == -__builtin_inff() ? ref : mn - kShift, by = ref - next;
            m = mn;
            ref = next;
            limit = mn == -__builtin_inff() ? -__builtin_inff() : kShift + kSlack + kBias;
            l *= f;
            zsum *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += by;
        }
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = exp2_fast(x[i]);
            l += p;
            if constexpr (kRaw) {
                w[i] = p;
            } else {
                // at most 2^(kShift + kSlack) by the choice of m; odd tokens hold Q - n
                constexpr float top = FMT == PQ_KV_8 ? 255.f : 15.f;
                w[i] = i & 1 ? -(p * sv[i]) : p * sv[i];
                zsum = __builtin_fmaf(p, i & 1 ? __builtin_fmaf(sv[i], top, zv[i]) : zv[i], zsum);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF16) {
                // the first is cut off, in one operation for both; the second has what is left
                const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(w[2 * i], w[2 * i + 1]));
                float h0, h1;
                unpack16<f16_t>(hi, h0, h1);
                // written as multiply-adds: one operation takes the f16, subtracts and rounds to f16
                const f16x2_t r = {static_cast<_Float16>(__builtin_fmaf(-h0, 1.f, w[2 * i])),
                                   static_cast<_Float16>(__builtin_fmaf(-h1, 1.f, w[2 * i + 1]))};
                u16x2_t lo = __builtin_bit_cast(u16x2_t, r);
                if constexpr (kRaw)                 // at least 2^-24 beside a first that is not 0
                    lo = __builtin_elementwise_max(lo, __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, hi), u16x2_t{1, 1}));
                weights[0][i] = hi;
                weights[1][i] = __builtin_bit_cast(uint32_t, lo);
            } else {
                float a = w[2 * i], b = w[2 * i + 1];
#pragma unroll
                for (int n = 0; n < kPieces; ++n) {
                    a = __builtin_elementwise_maximum(a, 0x1p-126f);
                    b = __builtin_elementwise_maximum(b, 0x1p-126f);
                    const uint32_t ab = __builtin_bit_cast(uint32_t, a), bb = __builtin_bit_cast(uint32_t, b);
                    weights[n][i] = __builtin_amdgcn_perm(bb, ab, 0x07060302u);
                    a -= __builtin_bit_cast(float, ab & 0xFFFF0000u);
                    b -= __builtin_bit_cast(float, bb & 0xFFFF0000u);
                }
            }
        }
    }

    __device__ __forceinline__ void second_product(const u32x4 (&weights)[kPieces])
    {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            u32x4 w[kPieces];
            const bool own = R == 1 || copy() == r;
#pragma unroll
            for (int n = 0; n < kPieces; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[n][i] = own ? weights[n][i] : 0u;
            // four channels at a time, so that no product waits for the one before
#pragma unroll
            for (int e0 = 0; e0 < E; e0 += 4) {
                u32x4 f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[e] = v_operand(r, e0 + e);
                    o[e0 + e] = mfma16<kF16>(f[e], w[0], o[e0 + e]);
                }
#pragma unroll
                for (int n = 1; n < kPieces; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e0 + e] = mfma16<kF16>(f[e], w[n], o[e0 + e]);
            }
        }
    }

    // The channel that element e of a lane in row n (column n of V) stands for.
    static __device__ __forceinline__ int channel(int n, int e) { return e / kRun * 128 + kRun * n + e % kRun; }

    // What a unit of o stands for, the weights' scale taken out.
    static constexpr float kOUnit = (kRaw ? 1.f : FMT == PQ_KV_8 ? 0x1p24f : 0x1p20f) * kUnscale;
};

// out and lse of 4 channels of a row from its sums.
template <typename QT>
__device__ __forceinline__ void write_out(const AttnArgs &a, int b, int hq, int d, float M, float L, f32x4 v)
{
    // L is 0 only where every token lies in a hidden page
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    *reinterpret_cast<u32x2 *>(a.out + b * a.out_bs + hq * a.out_hs + d) =
        u32x2{pack16<QT>(v[0] * inv, v[1] * inv), pack16<QT>(v[2] * inv, v[3] * inv)};
    // M is a whole number, the exponent of L joins it exactly
    if (d == 0 && a.lse)
        a.lse[static_cast<int64_t>(b) * a.q_heads + hq] =
            L == 0.f ? -__builtin_inff()
                     : (M + static_cast<float>(__builtin_amdgcn_frexp_expf(L)) +
                        __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(L))) * 0.69314718055994531f;
}

// A row (sequence, cache head, head tile) of a share, as its waves see it.
struct Row {
    int b, kvh, gt;
    int row0, n;                    // its beginning on the line, and its length there: kRowCost, then its steps
    int step0, stop;                // the share's part: its first step; where it ends on the line
    Range r;
    int t0, count;                  // the wave's first token; its steps (every kWaves-th)
};

template <typename QT, int FMT, int DP, int R, bool NT>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void k_attn_decode(AttnArgs a)
{
    using A = Attn<QT, FMT, DP, R, NT>;
    constexpr int E = A::E, kUnit = A::kUnit, kCols = A::kCols;
    constexpr int kPad = A::VD + 4;
    constexpr int kIds = 2 * R, kBatch = 64 / kIds;         // page ids of a step; steps whose ids a wave holds
    __shared__ int s_pre[kMaxBatch + 1], s_len[kMaxBatch];
    __shared__ int s_wsum[kWaves];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16], s_z[kWaves][16];
    __shared__ __align__(16) float s_o[kWaves * 16 * kPad];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kb = A::kb(), column = A::column();
    const int vheads = a.heads * a.gtiles;
    Cut cut = {};
    int begin = 0, end = 0;
    if (a.shares) {
        step_prefix(a, kUnit, s_len, s_pre, s_wsum);
        const int total = s_pre[a.batch] * vheads;
        cut = Cut{total / a.shares, total % a.shares};
        begin = cut.begin(blockIdx.x);
        end = cut.begin(blockIdx.x + 1);
        if (begin >= end) return;
    }
    const int in_page = (1 << a.page_log2) - 1;

    auto row_of = [&](int at, int b) {              // the row at `at`, in sequence b or later
        Row w;
        while (s_pre[b + 1] * vheads <= at) ++b;    // also past sequences without steps
        w.b = __builtin_amdgcn_readfirstlane(b);
        const int p0 = __builtin_amdgcn_readfirstlane(s_pre[w.b]);
        w.n = __builtin_amdgcn_readfirstlane(s_pre[w.b + 1]) - p0;
        const int vh = (at - p0 * vheads) / w.n;
        w.row0 = p0 * vheads + vh * w.n;
        w.kvh = vh / a.gtiles;
        w.gt = vh - w.kvh * a.gtiles;
        w.stop = min(w.row0 + w.n, end);
        w.r = range_of(a, __builtin_amdgcn_readfirstlane(s_len[w.b]));
        w.step0 = max(at - w.row0 - kRowCost, 0);
        w.t0 = w.r.base + (w.step0 + wave) * kUnit;
        w.count = max(w.stop - w.row0 - kRowCost - w.step0 - wave + kWaves - 1, 0) / kWaves;
        return w;
    };
    // Page ids of steps i0 .. i0 + kBatch - 1, one a lane; -1 where there is
    // none.  Nothing looks at the loaded value here, so that the wave does not
    // wait for it.
    auto load_ids = [&](const Row &w, int i0) {
        const int i = i0 + lane / kIds;
        const int t = w.t0 + i * (kWaves * kUnit) + lane % kIds * 16;
        int id = -1;
        if (i < w.count && t < w.r.len) id = a.table[w.b * a.table_stride + (t >> a.page_log2)];
        return id;
    };
    // A step whose loads are under way or wanted: its tiles' page ids, in
    // scalar registers.
    struct Step {
        int id[kIds], t;            // t: the wave's first token in it
    };
    auto step_at = [&](const Row &w, int held, int i) {
        Step f;
#pragma unroll
        for (int k = 0; k < kIds; ++k) f.id[k] = __builtin_amdgcn_readlane(held, (i % kBatch) * kIds + k);
        f.t = w.t0 + i * (kWaves * kUnit);
        return f;
    };
    const int pages = static_cast<int>(a.num_pages);
    auto valid = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(pages); };
    A st;
    st.set_offsets(a);
    int64_t tile_at[kIds];                          // byte offsets of a step's tiles in k and v
    // hidden tiles are read from page 0 and masked
    auto load_keys = [&](int kvh, const Step &f) {
#pragma unroll
        for (int t = 0; t < kIds; ++t) {
            const int off = (f.t + t * 16) & in_page;
            tile_at[t] = (valid(f.id[t]) ? f.id[t] : 0) * a.page_stride + kvh * a.head_stride +
                         static_cast<int64_t>(off) * a.token_stride;
            st.load_k(t >> 1, t & 1, a.k + tile_at[t]);
        }
    };
    auto load_values = [&]() {                      // of the step whose keys were loaded last
#pragma unroll
        for (int t = 0; t < kIds; ++t) st.load_v(t >> 1, t & 1, a.v + tile_at[t]);
    };
    const uint64_t v_from_k = reinterpret_cast<uint64_t>(a.vp) - reinterpret_cast<uint64_t>(a.kp);
    auto load_pairs = [&](int kvh, const Step &f) {
        if constexpr (!A::kRaw) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint64_t at[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int id = f.id[2 * r + t];
                    at[r] = reinterpret_cast<uint64_t>(
                        a.kp + ((static_cast<int64_t>(valid(id) ? id : 0) * a.heads + kvh) << a.page_log2) +
                        ((f.t + (2 * r + t) * 16) & in_page));
                }
                uint64_t p = at[0];
#pragma unroll
                for (int r = 1; r < R; ++r) p = A::copy() == r ? at[r] : p;
                p += 16 * kb;
                st.kpar[t] = *reinterpret_cast<const PQ_GLOBAL u32x4 *>(p);
                st.vpar[t] = *reinterpret_cast<const PQ_GLOBAL u32x4 *>(p + v_from_k);
            }
        }
    };

    Row w;
    if (a.shares) {
        int b0 = 0, hi = a.batch - 1;               // last sequence whose rows start at or before `begin`
        while (b0 < hi) {
            const int mid = (b0 + hi + 1) >> 1;
            if (s_pre[mid] * vheads <= begin) b0 = mid;
            else hi = mid - 1;
        }
        w = row_of(begin, b0);
        if (w.stop <= w.row0 + kRowCost) return;    // none of its steps
    } else {                                        // the block's own row
        w.b = blockIdx.x / vheads;
        const int vh = blockIdx.x - w.b * vheads;
        w.kvh = vh / a.gtiles;
        w.gt = vh - w.kvh * a.gtiles;
        w.r = range_of(a, a.lens[w.b]);
        w.row0 = w.step0 = 0;
        w.n = w.stop = end = w.r.steps(kUnit) + kRowCost;
        w.t0 = w.r.base + wave * kUnit;
        w.count = max(w.n - kRowCost - wave + kWaves - 1, 0) / kWaves;
    }
    // Loads run one step ahead: a step's keys, pairs and values are asked for as
    // soon as the step before has used its own, the first ones of a row during
    // the last step of the row before.  They are never under a branch inside a
    // step (a step without a successor asks for its own data again): with one
    // the compiler can only wait for all of them.
    bool ready = false;                             // the row's first loads are under way
    int held = load_ids(w, 0);
    for (;;) {
        const bool follows = w.stop + kRowCost < end;       // with a step of it at least
        Row next = w;
        int next_held = -1;
        if (follows) {
            next = row_of(w.stop, w.b);
            next_held = load_ids(next, 0);
        }
        Step now = step_at(w, held, 0);
        if (!ready) {
            st.load_q(a, w.b, w.kvh, w.gt);
            if (w.count > 0) {
                load_keys(w.kvh, now);
                load_values();
                load_pairs(w.kvh, now);
            }
        }
        asm volatile("" : "+v"(next_held));         // arrived before the steps begin
        st.set_q(a);
        st.clear();
        int held_after = -1;
        // Two blocks share a CU (with the exception at kMaxShares), and its
        // older waves go first: a priority that falls with each quarter of the
        // share keeps the two level (4 % of 64 ragged 4-bit contexts).
        const int quarter = (end - begin + 3) >> 2;
        for (int i = 0; i < w.count; ++i) {
            const int done = w.row0 + kRowCost + w.step0 + i * kWaves - begin;
            if (done >= 3 * quarter) __builtin_amdgcn_s_setprio(0);
            else if (done >= 2 * quarter) __builtin_amdgcn_s_setprio(1);
            else if (done >= quarter) __builtin_amdgcn_s_setprio(2);
            else __builtin_amdgcn_s_setprio(3);
            float x[8];
            st.first_product(x);
            if (i % kBatch == 0 && i + kBatch < w.count) held_after = load_ids(w, i + kBatch);
            Step then = now;
            int kvh = w.kvh;
            if (i + 1 < w.count) {
                if ((i + 1) % kBatch == 0) {
                    asm volatile("" : "+v"(held_after));
                    held = held_after;
                }
                then = step_at(w, held, i + 1);
            } else if (follows && next.count > 0) {
                then = step_at(next, next_held, 0);
                kvh = next.kvh;
            }
            load_keys(kvh, then);
            bool masked = now.t < w.r.first || now.t + kUnit > w.r.len;
#pragma unroll
            for (int k = 0; k < kIds; ++k) masked = masked || !valid(now.id[k]);
            unsigned seen = 0xFF;
            if (masked) {
                seen = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int id = now.id[e >> 2];
#pragma unroll
                    for (int r = 1; r < R; ++r) id = A::copy() == r ? now.id[2 * r + (e >> 2)] : id;
                    const int u = now.t + A::copy() * 32 + 4 * kb + (e >> 2) * 16 + (e & 3);
                    if (valid(id) && u >= w.r.first && u < w.r.len) seen |= 1u << e;
                }
            }
            u32x4 weights[A::kPieces];
            st.softmax(x, seen, masked, weights);
            load_pairs(kvh, then);
            st.second_product(weights);
            load_values();
            now = then;
        }
        if (w.count > 0 && follows) st.load_q(a, next.b, next.kvh, next.gt);
        ready = w.count > 0 && follows && next.count > 0;
        // join the waves and the copies of the columns
        // the weights' scale 2^kShift goes out of the sums
        const float l_all = column_sum(st.l) * A::kUnscale, z_all = column_sum(st.zsum) * A::kUnscale;
        __syncthreads();                            // the last row's s_m and s_o have been read
        if (kb == 0) {
            s_m[wave][column] = st.m;
            s_l[wave][column] = l_all;
            s_z[wave][column] = z_all;
        }
        __syncthreads();
        const int rows = min(kCols, a.group - w.gt * 16);
        const int g_own = column % kCols;
        auto top_of = [&](int g) {
            float M = -__builtin_inff();
            for (int v = 0; v < kWaves; ++v)
#pragma unroll
                for (int c = 0; c < R; ++c) M = fmaxf(M, s_m[v][c * kCols + g]);
            return M;
        };
        if (g_own < rows) {
            const float M = top_of(g_own), f = rescale(st.m, M) * A::kOUnit;
            float *so = s_o + (wave * 16 + column) * kPad;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<f32x4 *>(so + A::channel(4 * kb + i, e)) =
                        f32x4{st.o[e][i] * f, st.o[e + 1][i] * f, st.o[e + 2][i] * f, st.o[e + 3][i] * f};
        }
        __syncthreads();
        const bool opens = w.row0 + kRowCost >= begin, whole = opens && w.row0 + w.n <= end;
        const int slot = cut.slot(blockIdx.x, w.row0), hq0 = w.kvh * a.group + w.gt * 16;
        for (int i = tid * 4; i < rows * A::VD; i += 1024) {
            const int g = i / A::VD, d = i - g * A::VD;
            if (d >= a.dim) continue;
            const float M = top_of(g);
            float L = 0.f, Z = 0.f;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            for (int u = 0; u < kWaves; ++u)
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    const int col = c * kCols + g;
                    const float fw = rescale(s_m[u][col], M);
                    L += s_l[u][col] * fw;
                    Z += s_z[u][col] * fw;
                    v += *reinterpret_cast<const f32x4 *>(s_o + (u * 16 + col) * kPad + d);
                }
            v += Z;
            if (whole) {
                write_out<QT>(a, w.b, hq0 + g, d, M, L, v);
            } else {
                const int64_t at = static_cast<int64_t>(slot) * a.group_rows + g;
                *reinterpret_cast<f32x4 *>(a.part_o + at * a.dim + d) = v;
                if (d == 0) a.part_ml[at] = f32x2{M, L};
            }
        }
        if (a.shares && opens && tid == 0)          // for the join: whose partials make up the row
            a.spans[(w.b * a.heads + w.kvh) * a.gtiles + w.gt] =
                make_int2(slot, cut.share_of(w.row0 + w.n - 1));
        if (!follows) break;
        w = next;
        held = next_held;
    }
}

// Joins the shares of the rows that span several, in order, and writes the
// rows without a token.  One block per query head: its thread groups take
// every so many shares each, and their sums meet in LDS.
template <typename QT>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a)
{
    __shared__ float s_w[kMaxShares], s_red[2 * kWaves];
    __shared__ __align__(16) float s_v[1024];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.x / a.q_heads, hq = blockIdx.x - b * a.q_heads;
    const int kvh = hq / a.group, gi = hq - kvh * a.group, gt = gi / 16, g = gi - gt * 16;
    const int row = (b * a.heads + kvh) * a.gtiles + gt;
    const Range r = range_of(a, a.lens[b]);
    const int2 span = a.spans[row];                 // unset for a row without steps
    const int quads = a.dim / 4, groups = 256 / quads, q = tid % quads, part = tid / quads;
    if (r.len <= r.first) {
        if (part == 0) write_out<QT>(a, b, hq, 4 * q, 0.f, 0.f, f32x4{0.f, 0.f, 0.f, 0.f});
        return;
    }
    const int first = span.x >> 1, n = span.y - first + 1;
    if (n == 1) return;                             // written by its share
    auto slot_of = [&](int s) { return static_cast<int64_t>(s == 0 ? span.x : 2 * (first + s)) * a.group_rows + g; };
    const bool on = part < groups;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < n; s0 += 8 * groups) {
        f32x4 p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + part + k * groups;
            p[k] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (on && s < n) p[k] = *reinterpret_cast<const f32x4 *>(a.part_o + slot_of(s) * a.dim + 4 * q);
        }
        if (s0 == 0) {                              // meanwhile the weights: (m, l) of up to two shares a thread
            f32x2 ml[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) ml[k] = tid + 256 * k < n ? a.part_ml[slot_of(tid + 256 * k)] : f32x2{-__builtin_inff(), 0.f};
            float M = fmaxf(ml[0][0], ml[1][0]);
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
            if (lane == 0) s_red[wave] = M;
            __syncthreads();
            M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
            float L = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float f = rescale(ml[k][0], M);
                if (tid + 256 * k < n) s_w[tid + 256 * k] = f;
                L = __builtin_fmaf(ml[k][1], f, L);
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) L += __shfl_xor(L, o);
            if (lane == 0) s_red[kWaves + wave] = L;
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + part + k * groups;
            const float f = on && s < n ? s_w[s] : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(p[k][e], f, v[e]);
        }
    }
    *reinterpret_cast<f32x4 *>(s_v + 4 * tid) = v;
    __syncthreads();
    if (part > 0) return;
    for (int k = 1; k < groups; ++k) v += *reinterpret_cast<const f32x4 *>(s_v + 4 * (k * quads + q));
    write_out<QT>(a, b, hq, 4 * q, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])),
                  s_red[kWaves] + s_red[kWaves + 1] + s_red[kWaves + 2] + s_red[kWaves + 3], v);
}

// Rows of at most kWholeRow tokens are not split: one block takes such a row
// in a few rounds, and a second launch would cost more (one bf16 sequence of
// 1000 tokens 9.8 us against 11.7, of 2000 16.1 against 11.6; 64 of up to
// 1000 in 8 bits, 512 rows, 20 against 28).  Where the rows alone fill the
// chip that holds up to kWholeRowMany (512 rows of evenly spread lengths up to
// 2000 tokens 40 us against 41; 128 rows 26 against 22).
constexpr int kWholeRow = 1024, kWholeRowMany = 2048;
constexpr int kManyRows = 256;      // one per CU

// A call whose cache is larger than the memory-side cache (256 MB) finds
// nothing of it there: its loads are non-temporal then (32 contexts of 16 Ki
// bf16 tokens, 1.9 GB: 294 us against 315), but only where a row is whole
// 128-byte lines, else lines that two loads share are fetched twice (bf16 rows
// of 80 channels: 108 us against 85).  A smaller cache may still lie there
// from the call before (16 chats, 67 MB: 21 us against 17.2).
constexpr int64_t kStreamBytes = int64_t(256) << 20;

template <typename QT, int FMT, int DP, int R, bool NT>
void launch_one(AttnArgs a, int64_t longest, hipStream_t s)
{
    const int unit = 32 * R;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * a.gtiles;
    if (longest <= (rows >= kManyRows ? kWholeRowMany : kWholeRow)) {
        a.shares = 0;
        hipLaunchKernelGGL((k_attn_decode<QT, FMT, DP, R, NT>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, a);
        return;
    }
    const int64_t want = (rows * ((longest + unit - 1) / unit) + kWaves - 1) / kWaves;    // a step per wave at least
    a.shares = static_cast<int>(want > kMaxShares ? kMaxShares : want);
    hipLaunchKernelGGL((k_attn_decode<QT, FMT, DP, R, NT>), dim3(static_cast<unsigned>(a.shares)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_attn_join<QT>, dim3(static_cast<unsigned>(a.batch * a.q_heads)), dim3(256), 0, s, a);
}

template <typename QT, int FMT, int DP, int R>
void launch_stream(const AttnArgs &a, int64_t longest, hipStream_t s)
{
    constexpr int kRow = FMT == PQ_KV_16 ? 2 * DP : DP;     // bytes of a full row
    constexpr int kHeld = 2 * (kRow + (FMT == PQ_KV_16 ? 0 : 4));
    if constexpr (FMT != PQ_KV_4 && kRow % 128 == 0) {
        if (a.dim == DP && longest * a.batch * a.heads * kHeld > kStreamBytes && a.token_stride % 128 == 0)
            return launch_one<QT, FMT, DP, R, true>(a, longest, s);
    }
    launch_one<QT, FMT, DP, R, false>(a, longest, s);
}

template <typename QT, int FMT, int DP>
void launch_copies(const AttnArgs &a, int64_t longest, hipStream_t s)
{
    // Two copies of the heads in the columns where the group leaves room, for
    // 4 bits (64 ragged contexts of 64 channels 32 us against 38, of 128
    // channels 43.9 against 45.8) of up to 128 channels (of 256: 66 against 53).
    // More bytes a token outlast the softmax (8 bits, 128 channels: 71.5 us
    // with two copies, 68.6 with one).
    if constexpr (FMT == PQ_KV_4 && DP <= 128) {
        if (a.group <= 8) return launch_stream<QT, FMT, DP, 2>(a, longest, s);
    }
    launch_stream<QT, FMT, DP, 1>(a, longest, s);
}

template <typename QT, int FMT>
void launch_dim(const AttnArgs &a, int64_t longest, hipStream_t s)
{
    if (a.dim <= 64) return launch_copies<QT, FMT, 64>(a, longest, s);
    // Vector instructions bound 4 bits: the first product leaves out the last
    // 32 channels where it can (64 contexts of 80 channels 37.6 us against
    // 38.5).  Other formats wait for their bytes.
    if constexpr (FMT == PQ_KV_4) {
        if (a.dim <= 96) return launch_copies<QT, FMT, 96>(a, longest, s);
    }
    if (a.dim <= 128) launch_copies<QT, FMT, 128>(a, longest, s);
    else launch_copies<QT, FMT, 256>(a, longest, s);
}

template <typename QT>
pq_status launch_attn(int format, const AttnArgs &a, int64_t longest, hipStream_t s)
{
    if (format == PQ_KV_16) launch_dim<QT, PQ_KV_16>(a, longest, s);
    else if (format == PQ_KV_8) launch_dim<QT, PQ_KV_8>(a, longest, s);
    else launch_dim<QT, PQ_KV_4>(a, longest, s);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

// Workspace: o, then (m, l), then the spans.
int64_t part_rows(int group) { return static_cast<int64_t>(2) * kMaxShares * (group < 16 ? group : 16); }
int64_t attn_workspace(const pq_kv_cache &c, int64_t batch, int group)
{
    const int64_t n = batch < kMaxBatch ? batch : kMaxBatch;
    return part_rows(group) * (c.dim + 2) * 4 + n * c.heads * ((group + 15) / 16) * 8;
}

}  // namespace
}  // namespace pq

extern "C" {

int64_t pq_attn_decode_workspace_bytes(const pq_kv_cache *cache, int64_t batch, int64_t q_heads)
{
    using namespace pq;
    if (kv_cache_status(cache) != PQ_OK || batch < 0 || q_heads < 1 || q_heads > 65535 || q_heads % cache->heads) return -1;
    if (batch == 0) return 0;
    return (attn_workspace(*cache, batch, static_cast<int>(q_heads / cache->heads)) + 15) / 16 * 16;
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
    if (max_pages < 0 || max_pages > (int64_t(1) << 30) / c.page_size || table_stride < 0) return PQ_ERR_SHAPE;
    if (((q_batch_stride | q_head_stride | out_batch_stride | out_head_stride) & 7) != 0) return PQ_ERR_SHAPE;
    if (!std::isfinite(scale) || window < 0 || max_len < 0) return PQ_ERR_ARG;
    if (batch == 0) return PQ_OK;
    if (!q || !out || !lens || (!block_table && max_pages > 0) || !workspace) return PQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return PQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(lse)) % 4)
        return PQ_ERR_ALIGN;
    const int group = static_cast<int>(q_heads / c.heads);
    if (workspace_bytes < attn_workspace(c, batch, group)) return PQ_ERR_ARG;
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
    a.max_tokens = static_cast<int>(max_pages * c.page_size);
    a.lens = lens;
    a.group = group;
    a.gtiles = (group + 15) / 16;
    a.group_rows = group < 16 ? group : 16;
    a.window = window < INT32_MAX ? static_cast<int>(window) : 0;   // longer than any sequence: everything
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634074);
    a.out = static_cast<uint16_t *>(out);
    a.out_bs = out_batch_stride;
    a.out_hs = out_head_stride;
    a.lse = lse;
    a.q_heads = static_cast<int>(q_heads);
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<f32x2 *>(a.part_o + part_rows(group) * c.dim);
    a.spans = reinterpret_cast<int2 *>(a.part_ml + part_rows(group));
    // lens past max_len count as max_len: rows are then known to be short
    if (max_len > 0 && max_len < a.max_tokens) a.max_tokens = static_cast<int>(max_len);
    int64_t longest = a.max_tokens;
    // its first tile may start 15 tokens early
    if (a.window > 0 && longest > int64_t(a.window) + 15) longest = int64_t(a.window) + 15;
    // the kernel counts steps of at least 32 tokens and row costs in 32 bits
    const int64_t row_steps = (static_cast<int64_t>(a.max_tokens) + 31) / 32 + 1 + kRowCost;
    int64_t most = INT32_MAX / (row_steps * c.heads * a.gtiles);
    if (most < 1) return PQ_ERR_SHAPE;
    if (most > kMaxBlocks / q_heads) most = kMaxBlocks / q_heads;     // a block per query head joins the shares
    if (most > kMaxBatch) most = kMaxBatch;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    for (int64_t b0 = 0; b0 < batch; b0 += most) {
        AttnArgs x = a;
        x.batch = static_cast<int>(batch - b0 < most ? batch - b0 : most);
        x.q += b0 * q_batch_stride;
        x.out += b0 * out_batch_stride;
        if (x.lse) x.lse += b0 * q_heads;
        if (x.table) x.table += b0 * table_stride;
        x.lens += b0;
        const pq_status r = q_dtype == PQ_BF16 ? launch_attn<bf16_t>(c.format, x, longest, s)
                                               : launch_attn<f16_t>(c.format, x, longest, s);
        if (r != PQ_OK) return r;
    }
    return PQ_OK;
}

}  // extern "C"
