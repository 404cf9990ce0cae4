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

// More columns than this: two column tiles a block of the stream kernel, four from
// twice as many on.
constexpr int64_t kStreamPair = 16 * 2 * 192;

// Few rows (16 MT): the weights' stream bounds it, and memory gives its rate only
// with tens of KB in flight a CU.  A block takes TN 16-column tiles; its NW waves
// share K by 64-byte groups of codes, wave w taking groups w, w + NW, ..., each
// through a ring of D stages in LDS of its own that direct loads fill (codes with
// the streaming hint: they are read once), so that a wave waits for its own loads
// only and the block meets once, to add the sums.  In the export byte order the
// blocks of a launch then read one window of consecutive addresses.
// A load of activations brings RPL rows' chunks of a group, interleaved by 16
// bytes, and lies 16 RPL bytes further from the next than it is long, so that
// sixteen rows' reads fall on different banks; rows past M read the last one.
// 16384 x 16384 at 2 bits, out of HBM: 14.9 us with one row, 16.5 with sixteen
// (4.5 and 4.1 TB/s; codes and activations loaded to registers 20 and 28, the
// activations' 16-byte pieces of many rows being what that waits for).
template <int BITS, int TN, int XI, int MT>
struct StreamShape {
    static constexpr int GK = 512 / BITS, STEPS = GK / 64;      // k and products of a group
    static constexpr int RPL = 1024 / GK, XS = 1024 + 16 * RPL; // rows a load, bytes between loads
    // eight waves' rings of 8 KB of activations a stage do not fit
    static constexpr int NW = XI == 8 || MT == 2 ? 4 : 8, D = 2, SLOT = TN * 1024 + XI * XS;
    static constexpr int RED = NW * TN * MT * 16 * 80;               // the waves' sums: rows of 16 tiles' columns, 16 bytes apart
    static constexpr int LDS = NW * D * SLOT > RED ? NW * D * SLOT : RED;
};

template <int BITS, int TN, int XI, int MT>
__global__ __launch_bounds__((64 * StreamShape<BITS, TN, XI, MT>::NW)) void k_a8_stream(A8Args a)
{
    using C = StreamShape<BITS, TN, XI, MT>;
    constexpr int GK = C::GK, RPL = C::RPL, NW = C::NW, D = C::D;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int i16 = lane & 15, g = lane >> 4;
    const int groups = (a.K + GK - 1) / GK, turns = groups > w ? (groups - w + NW - 1) / NW : 0;
    const int last_tile = (a.N - 1) >> 4;
    uint32_t co[TN], xo[XI];
#pragma unroll
    for (int t = 0; t < TN; ++t)
        co[t] = static_cast<uint32_t>(min(static_cast<int>(blockIdx.x) * TN + t, last_tile) * 1024 + i16 * 64 + g * 16);
#pragma unroll
    for (int q = 0; q < XI; ++q) xo[q] = static_cast<uint32_t>(min(RPL * q + lane % RPL, a.M - 1) * a.x_st);
    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds)) +
                          w * (D * C::SLOT);
    auto issue = [&](int t, int slot) __attribute__((always_inline)) {
        const int group = w + NW * t;
        const uint8_t *cb = a.packed + group * a.gstride;
#pragma unroll
        for (int i = 0; i < TN; ++i) dma16<true>(cb, co[i], ring + slot * C::SLOT + i * 1024);
        // chunks past K: the row's last one (no product is made of them)
        const uint32_t k = static_cast<uint32_t>(min(group * GK + lane / RPL * 16, a.K - 16));
#pragma unroll
        for (int q = 0; q < XI; ++q) dma16(a.X, xo[q] + k, ring + slot * C::SLOT + TN * 1024 + q * C::XS);
    };
    intx4 acc[MT][TN];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < TN; ++t) acc[m][t] = intx4{0, 0, 0, 0};
    const uint8_t *own = lds + w * (D * C::SLOT);
    const uint8_t *xr[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = min(16 * m + i16, a.M - 1);
        xr[m] = own + TN * 1024 + row / RPL * C::XS + row % RPL * 16 + g * (C::STEPS * 16 * RPL);
    }
    auto compute = [&](int t, int slot) __attribute__((always_inline)) {
        u32x4 c[TN];
        intx4 x[MT][C::STEPS];
#pragma unroll
        for (int i = 0; i < TN; ++i) c[i] = *reinterpret_cast<const u32x4 *>(own + slot * C::SLOT + i * 1024 + lane * 16);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < C::STEPS; ++j) x[m][j] = *reinterpret_cast<const intx4 *>(xr[m] + slot * C::SLOT + j * (16 * RPL));
        const int k = (w + NW * t) * GK + g * (GK / 4);
        if ((w + NW * t + 1) * GK > a.K) {
#pragma unroll
            for (int j = 0; j < C::STEPS; ++j)
                if (k + 16 * j >= a.K) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) x[m][j] = intx4{0, 0, 0, 0};
                }
        }
#pragma unroll
        for (int j = 0; j < C::STEPS; ++j)
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                Words<BITS> wd;
                if constexpr (BITS == 1) wd.w = c[i][j >> 1] >> (16 * (j & 1));
                if constexpr (BITS == 2) wd.w = c[i][j];
                if constexpr (BITS == 4) wd = {c[i][2 * j], c[i][2 * j + 1]};
                const intx4 b = decode(a, wd);
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, x[m][j], acc[m][i], 0, 0, 0);
            }
    };
    // The counted waits hold because the loop has no other vector memory operation
    // (a spilled register would be one: every variant keeps all of its own).
    for (int t = 0; t < min(D, turns); ++t) issue(t, t);
    int t = 0, slot = 0;
    for (; t + D < turns; ++t) {
        wait_vmcnt<(D - 1) * (TN + XI)>();
        compute(t, slot);
        wait_lgkmcnt0();                // the slot's reads have returned
        issue(t + D, slot);
        slot = slot + 1 == D ? 0 : slot + 1;
    }
    static_for<0, D>([&](auto left) {
        constexpr int after = D - 1 - decltype(left)::value;    // turns issued after this one
        const int at = turns - 1 - after;
        if (at >= t) {
            wait_vmcnt<after * (TN + XI)>();
            compute(at, at % D);
        }
    });
    __syncthreads();
    intx4 *red = reinterpret_cast<intx4 *>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < TN; ++i) red[((w * MT + m) * TN + i) * 80 + i16 * 5 + g] = acc[m][i];
    __syncthreads();
    // a lane takes eight columns of a row
    for (int at = threadIdx.x; at < 32 * TN * MT; at += 64 * NW) {
        const int h = at % (2 * TN), r = at / (2 * TN), c = blockIdx.x * (2 * TN) + h;
        if (r >= a.M || 8 * c >= a.N) continue;
        intx4 lo = {0, 0, 0, 0}, hi = lo;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const intx4 *p = red + ((i * MT + (r >> 4)) * TN + (h >> 1)) * 80 + (r & 15) * 5 + 2 * (h & 1);
            lo += p[0];
            hi += p[1];
        }
        int sum[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sum[e] = lo[e];
            sum[4 + e] = hi[e];
        }
        float cs[8], cb[8];
        columns8(a, c, cs, cb);
        with_type(a.y_dtype, [&](auto type) __attribute__((always_inline)) { finish8<decltype(type)>(a, r, c, a.x_scale[r], sum, cs, cb); });
    }
}

// Output tiles of many rows: WN waves side by side, each 16 MT rows by 16 NT
// columns, over K in stages of 128.  A stage's activations (128 bytes a row,
// 16-byte chunks swizzled as in the bf16 kernels) and code bytes go from memory
// to LDS directly, into a ring of P slots.  KG groups of such waves take every
// KG-th stage and add their sums at the end: a small tile's stage is so short
// that the turn to the next one costs more than its products.
template <int BITS, int WN, int KG, int MT, int NT, int P>
struct TileCfg {
    static constexpr int BM = 16 * MT, BN = 16 * NT * WN, THREADS = 64 * WN * KG;
    static constexpr int PIECES = BITS == 4 ? 4 : 2;            // 16-byte pieces of a column a stage (1 bit: two stages' worth)
    static constexpr int XB = BM * 128, CB = BN * PIECES * 16, SLOT = XB + CB;
    static constexpr int XI = XB / 1024 / WN, CI = CB / 1024 / WN;   // loads a wave and stage
    static constexpr int EPI = 8 * MT * (BN * 4 + 16);              // the epilogue's half tile
    static constexpr int LDS = P * KG * SLOT > EPI ? P * KG * SLOT : EPI;
    static_assert(XI * WN * 1024 == XB && CI * WN * 1024 == CB, "whole loads");
};

template <int BITS, int WN, int KG, int MT, int NT, int P>
__global__ __launch_bounds__(64 * WN * KG, 2) void k_a8_tile(A8Args a, int mtiles, int ntiles)
{
    using C = TileCfg<BITS, WN, KG, MT, NT, P>;
    static_assert(MT < 8 || KG == 1, "the large tile has one group");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int w = KG == 1 ? wave : wave % WN, kg = KG == 1 ? 0 : wave / WN;
    const int i16 = lane & 15, g = lane >> 4;

    // Tiles go eight row tiles by all columns at a time.  Where the number of
    // blocks is a multiple of eight, one XCD's blocks take consecutive ones, so
    // that its L2 serves both operands; other launches deal them round the XCDs.
    int t = blockIdx.x;
    const int nb = gridDim.x;
    if ((nb & 7) == 0) t = (t & 7) * (nb >> 3) + (t >> 3);
    const int band = t / (8 * ntiles), rows = min(8, mtiles - 8 * band), in = t - band * 8 * ntiles;
    const int m0 = (8 * band + in % rows) * C::BM, n0 = in / rows * C::BN;

    const uint8_t *xb = reinterpret_cast<const uint8_t *>(a.X) + m0 * a.x_st;
    uint32_t xo[C::XI];
#pragma unroll
    for (int q = 0; q < C::XI; ++q) {
        const int r = 8 * (C::XI * w + q) + (lane >> 3);
        xo[q] = static_cast<uint32_t>((min(m0 + r, a.M - 1) - m0) * a.x_st) + ((lane & 7) ^ xswz(r)) * 16;
    }
    // 64 in the lanes that load a stage's second half: the same for every q,
    // since the rows' swizzles differ in the chunk's lowest bit only
    const uint32_t far = (((lane & 7) ^ (lane >> 3)) & 4) * 16;
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
    // the block's share of K: stages [first, last); only the smallest tile's is a part
    const int stages = (a.K / 64 + 1) / 2, share = static_cast<int>(blockIdx.y);
    const int first = MT > 2 ? 0 : share * stages / a.splits, last = MT > 2 ? stages : (share + 1) * stages / a.splits;
    const int steps = min(a.K / 64, 2 * last) - 2 * first;
    const int turns = (last - first + KG - 1) / KG;

    // The group's stage of turn t to its slot; past the last one the last
    // again, so that the number of loads in flight is the same at every wait.
    // The second half of an odd last stage is not there: its chunks read the
    // first half.
    auto stage_of = [&](int t) __attribute__((always_inline)) { return first + KG * t + kg; };
    auto issue = [&](int t, int slot) __attribute__((always_inline)) {
        const int s = min(stage_of(t), last - 1);
        const uint32_t at = lds_base + (slot * KG + kg) * C::SLOT;
        const uint32_t back = far & (2 * s + 1 < a.K / 64 ? 0 : 64);
#pragma unroll
        for (int q = 0; q < C::XI; ++q) dma16(xb + s * 128, xo[q] - back, at + (C::XI * w + q) * 1024);
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
    for (int h = 0; h < 2; ++h) xr[h] = lds + kg * C::SLOT + i16 * 128 + (((4 * h + g) ^ xswz(i16)) << 4);
    const uint8_t *cr = lds + kg * C::SLOT + C::XB + w * NT * (C::PIECES * 256) + i16 * 16 +
                        (BITS == 4 ? (g >> 1) * 256 + (g & 1) * 8 : BITS == 2 ? g * 4 : (g >> 1) * 4);

    // Operands of a step of 64: activations and the code words.
    struct Operands {
        intx4 x[MT];
        Words<BITS> w[NT];
    };
    auto read_codes = [&](auto h_c, int s, int slot, Operands &o) __attribute__((always_inline)) {
        constexpr int H = decltype(h_c)::value;
        const uint8_t *cp = cr + slot * (KG * C::SLOT) + (BITS == 4 ? H * 512 : BITS == 2 ? H * 256 : H * 8 + (s & 1) * 256);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if constexpr (BITS == 4) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(cp + j * (C::PIECES * 256));
                o.w[j] = {v[0], v[1]};
            } else {
                o.w[j].w = *reinterpret_cast<const uint32_t *>(cp + j * (C::PIECES * 256));
                if constexpr (BITS == 1) o.w[j].w >>= 16 * (g & 1);
            }
        }
    };
    auto read_rows = [&](auto h_c, int slot, int i, Operands &o) __attribute__((always_inline)) {
        o.x[i] = *reinterpret_cast<const intx4 *>(xr[decltype(h_c)::value] + slot * (KG * C::SLOT) + i * 2048);
    };
    // The products of a step, a column tile at a time.  While one's run, the
    // next one's codes are decoded (at the end those of `then`, the first of
    // the step after) and the operands `to` of a later step are read, half H of
    // stage s: the matrix unit takes 16 cycles a product, time for two of the
    // decoding's operations and a read.  The scheduler is held to that order.
    intx4 b;
    auto multiply = [&](const Operands &o, const Words<BITS> &then, auto h_c, int s, int slot, Operands &to)
                        __attribute__((always_inline)) {
        read_codes(h_c, s, slot, to);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const intx4 bn = decode(a, j + 1 < NT ? o.w[j + 1] : then);
#pragma unroll
            for (int i = j * MT / NT; i < (j + 1) * MT / NT; ++i) read_rows(h_c, slot, i, to);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, o.x[i], acc[i][j], 0, 0, 0);
            b = bn;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // a product
                __builtin_amdgcn_sched_group_barrier(0x100, MT < 8 ? 2 : 1, 0);      // reads
                __builtin_amdgcn_sched_group_barrier(0x002, MT < 8 ? 4 : 2, 0);      // vector operations
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<int, 0> half0{};
    constexpr std::integral_constant<int, 1> half1{};
    auto read_all = [&](auto h_c, int s, int slot, Operands &o) __attribute__((always_inline)) {
        read_codes(h_c, s, slot, o);
#pragma unroll
        for (int i = 0; i < MT; ++i) read_rows(h_c, slot, i, o);
    };

    // Counted waits, as in the stream kernel: nothing but `issue` touches vector memory.
#pragma unroll
    for (int t = 0; t < P; ++t) issue(t, t);
    wait_vmcnt<(P - 1) * (C::XI + C::CI)>();
    block_barrier();
    int slot = 0;
    // Every read of the slot's stages is done in all waves and the next turn's
    // stages have landed: the slot takes those of turn t + P.
    auto turn = [&](int t) __attribute__((always_inline)) {
        wait_lgkmcnt0();
        wait_vmcnt<(P - 2) * (C::XI + C::CI)>();
        block_barrier();
        issue(t + P, slot);
        __builtin_amdgcn_sched_barrier(0);
        slot = slot == P - 1 ? 0 : slot + 1;
    };
    if constexpr (MT == 8) {
        // Operands a step ahead: a stage's first half is multiplied while its
        // second half's are read, and that one while the next stage's first
        // are.
        Operands even, odd;
        read_all(half0, first, 0, even);
        b = decode(a, even.w[0]);
        for (int t = 0; t < steps / 2; ++t) {
            multiply(even, odd.w[0], half1, first + t, slot, odd);
            turn(t);
            multiply(odd, even.w[0], half0, first + t + 1, slot, even);
        }
        if (steps & 1) multiply(even, odd.w[0], half0, 0, slot, odd);
    } else {
        // A step's products are shorter than a read's way: operands a whole
        // stage ahead.
        Operands x0, x1, y0, y1;
        read_all(half0, stage_of(0), 0, x0);
        read_all(half1, stage_of(0), 0, x1);
        b = decode(a, x0.w[0]);
        auto stage = [&](int t, Operands &c0, Operands &c1, Operands &n0, Operands &n1) __attribute__((always_inline)) {
            turn(t);
            multiply(c0, c1.w[0], half0, stage_of(t + 1), slot, n0);
            multiply(c1, n0.w[0], half1, stage_of(t + 1), slot, n1);
        };
        // the last turn, in which a group may have no stage, or half of one
        auto end = [&](Operands &c0, Operands &c1, Operands &n0) __attribute__((always_inline)) {
            const int s = stage_of(turns - 1);
            if (s < last) multiply(c0, c1.w[0], half0, s, slot, n0);
            if (s < last && 2 * s + 1 < a.K / 64) multiply(c1, c1.w[0], half0, s, slot, n0);
        };
        int t = 0;
        for (; t + 2 < turns; t += 2) {
            stage(t, x0, x1, y0, y1);
            stage(t + 1, y0, y1, x0, x1);
        }
        if (t + 1 < turns) {
            stage(t, x0, x1, y0, y1);
            end(y0, y1, x0);
        } else {
            end(x0, x1, y0);
        }
    }
    wait_vmcnt<0>();        // no load is in flight into LDS when the block ends

    // The sums through LDS, so that every output line is written whole: MT / 2
    // row tiles at a time, rows 16 bytes further apart than they are long (the
    // sixteen rows of a write then lie in different banks).  A thread takes the
    // same eight columns of every TR-th row.
    constexpr int RS = C::BN * 4 + 16, TC = C::BN / 8, HR = 8 * MT;        // HR: rows of a half
    constexpr int TR = C::THREADS / TC < HR ? C::THREADS / TC : HR, RT = HR / TR;
    const int tc = threadIdx.x % TC, tr = threadIdx.x / TC, c = (n0 >> 3) + tc;
    auto to_lds = [&](int half) __attribute__((always_inline)) {
#pragma unroll
        for (int k = KG - 1; k >= 0; --k) {
            __syncthreads();
            if (KG > 1 && kg != k) continue;
#pragma unroll
            for (int i = 0; i < MT / 2; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    intx4 *p = reinterpret_cast<intx4 *>(lds + (16 * i + i16) * RS + ((w * NT + j) * 16 + 4 * g) * 4);
                    *p = k == KG - 1 ? acc[half * (MT / 2) + i][j] : acc[half * (MT / 2) + i][j] + *p;
                }
        }
        __syncthreads();
    };
    auto sums = [&](int r, int (&sum)[8]) __attribute__((always_inline)) {
        const intx4 *p = reinterpret_cast<const intx4 *>(lds + r * RS + tc * 32);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sum[e] = p[0][e];
            sum[4 + e] = p[1][e];
        }
    };
    if (MT == 2 && a.splits > 1) {  // the sums as they are, joined by k_a8_join
        int32_t *out = a.partial + static_cast<int64_t>(blockIdx.y) * a.M * a.p_st;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row0 = m0 + half * (MT / 2) * 16;
            to_lds(half);
            for (int r = tr; r < min(HR, a.M - row0); r += C::THREADS / TC) {
                const intx4 *p = reinterpret_cast<const intx4 *>(lds + r * RS + tc * 32);
                intx4 *to = reinterpret_cast<intx4 *>(out + (row0 + r) * a.p_st + 8 * c);
                if (8 * c < a.p_st) {
                    to[0] = p[0];
                    to[1] = p[1];
                }
            }
        }
        return;
    }
    float cs[8], cb[8];
    columns8(a, c, cs, cb);
    with_type(a.y_dtype, [&](auto type) __attribute__((always_inline)) {
        using T = decltype(type);
        const T *other = static_cast<const T *>(a.other);
        T *y = static_cast<T *>(a.Y);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row0 = m0 + half * (MT / 2) * 16, rows = min(HR, a.M - row0);
            if (n0 + C::BN <= a.N && rows == HR) {
                // a whole half: everything that it loads is on its way while
                // the sums go through LDS
                Raw8<T> o[RT];
                float rs[RT];
#pragma unroll
                for (int k = 0; k < RT; ++k) {
                    const int64_t m = row0 + min(tr, TR - 1) + k * TR;
                    if (other) o[k] = load_whole8(other + m * a.o_st + 8 * c);
                    rs[k] = a.x_scale[m];
                }
                to_lds(half);
#pragma unroll
                for (int k = 0; k < RT; ++k) {
                    if (tr >= TR) break;        // a half of fewer rows than threads
                    int sum[8];
                    float v[8];
                    sums(tr + k * TR, sum);
                    outputs8<T>(a, rs[k], sum, cs, cb, o[k], v);
                    T *to = y + (row0 + tr + k * TR) * a.y_st + 8 * c;
                    if (MT == 8 && a.nt) store_whole8<true>(to, v);
                    else store_whole8(to, v);
                }
            } else {
                to_lds(half);
                if (8 * c < a.N)
                    for (int r = tr; r < rows; r += C::THREADS / TC) {
                        int sum[8];
                        sums(r, sum);
                        finish8<T>(a, row0 + r, c, a.x_scale[row0 + r], sum, cs, cb);
                    }
            }
        }
    });
}

// Split K: the shares' sums added up, and the epilogue.
__global__ __launch_bounds__(256) void k_a8_join(A8Args a)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int chunks = static_cast<int>(a.p_st / 8);
    const int64_t m = at / chunks;
    const int c = static_cast<int>(at - m * chunks);
    if (m >= a.M) return;
    const intx4 *p = reinterpret_cast<const intx4 *>(a.partial + m * a.p_st + 8 * c);
    const int64_t step = a.M * a.p_st / 4;
    intx4 lo = p[0], hi = p[1];
    for (int i = 1; i < a.splits; ++i) {
        lo += p[i * step];
        hi += p[i * step + 1];
    }
    int sum[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sum[e] = lo[e];
        sum[4 + e] = hi[e];
    }
    float cs[8], cb[8];
    columns8(a, c, cs, cb);
    with_type(a.y_dtype, [&](auto type) __attribute__((always_inline)) { finish8<decltype(type)>(a, m, c, a.x_scale[m], sum, cs, cb); });
}

// How a shape is cut.  Up to 16 rows the stream kernel; up to 32 too (at 2 and 4
// bits: 32 rows of 14336 x 4096 9.0 us, of 1600 x 4352 7.3, in tiles 11.8 and 9.8),
// but for long K under few columns, where every one-tile block reads all
// activations (32 rows of a 4-bit 4096 x 14336 16.8 us, in tiles 15.0).  At 1 bit
// a group of 32 rows' activations is 16 loads, for which the ring has room with two
// waves only (32 rows of 14336 x 4096 9.9 us, of 1600 x 4352 6.0; in tiles 9.0 and
// 9.2): there is no such form.
// 128 x 256 tiles from 176 of them on (512 rows of 14336 x
// 4096, 224 tiles: 33 us against 40; 333 rows, 168 tiles: 34 both ways; 256 rows,
// 112 tiles: 31 against 21).  Else 64 x 128, of one group of waves
// where there are two a CU and of two groups down to 192 tiles (1024 rows of N =
// K = 4096, 512 tiles: 23 us against 26; 512 rows, 256 tiles: 16 against 14; 1024
// rows of 1600 x 1600, 208 tiles: 9.5 against 8.7).  Below
// that 32 x 64, two waves and two groups, two blocks a CU (64 rows of N = K = 4096
// 8.4 us, 128 rows with 4 bits 8.6, 200 rows of 1600 x 4352 8.9, 40 of 576 x 576
// 4.7; as 32 x 128, one a CU, 10.5, 10.9, 11.2 and 5.5), with K split while that
// pays: a second launch and the way of the partial sums take 3 us and their 8
// bytes at 4 TB/s; a stage takes 0.15 us, and one less in each of the shares, which
// run side by side, is counted with 0.125 (64 rows of 4096 x 14336 20.9 us in one
// share, 14.8 in four, where this expects 15.5; of 4096 x 28672 37.9, 20.3 and 22).
struct A8Plan {
    int mt, groups;          // 16-row tiles a block (0: the stream kernel), groups of waves
    int splits;              // shares of K
    int64_t p_st;            // columns of a row of partial sums
};

inline A8Plan a8_plan(int bits, int64_t M, int64_t N, int64_t K)
{
    if (M <= 16 || (M <= 32 && bits > 1 && (N > kStreamPair || K <= 8192))) return {0, 1, 1, 0};
    if (((M + 127) / 128) * ((N + 255) / 256) >= 176) return {8, 1, 1, 0};
    const int64_t tiles = ((M + 63) / 64) * ((N + 127) / 128);
    if (M > 32 && tiles >= 192) return {4, tiles >= 512 ? 1 : 2, 1, 0};
    const int64_t blocks = ((M + 31) / 32) * ((N + 63) / 64), stages = (K / 64 + 1) / 2;
    int64_t splits = 1;
    double least = 125.0 * stages;                      // ns
    for (int64_t n = 2; n * blocks <= 512 && 4 * n <= stages; ++n) {
        const double cost = 125.0 * ((stages + n - 1) / n) + 3000.0 + 0.002 * M * N * n;
        if (cost < least) {
            least = cost;
            splits = n;
        }
    }
    if (splits < 2) return {2, 2, 1, 0};
    return {2, 2, static_cast<int>(splits), (N + 7) / 8 * 8};
}

template <int BITS, int WN, int KG, int MT, int NT, int P>
pq_status launch_tile(const A8Args &a, hipStream_t s)
{
    using C = TileCfg<BITS, WN, KG, MT, NT, P>;
    const int mtiles = (a.M + C::BM - 1) / C::BM, ntiles = (a.N + C::BN - 1) / C::BN;
    const int64_t blocks = static_cast<int64_t>(mtiles) * ntiles;
    if (blocks > kMaxBlocks) return PQ_ERR_SHAPE;
    hipLaunchKernelGGL((k_a8_tile<BITS, WN, KG, MT, NT, P>), dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.splits)),
                       dim3(C::THREADS), 0, s, a, mtiles, ntiles);
    if (hipGetLastError() != hipSuccess) return PQ_ERR_HIP;
    if (a.splits == 1) return PQ_OK;
    const int64_t threads = a.M * (a.p_st / 8);
    hipLaunchKernelGGL(k_a8_join, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

template <int BITS, int XI, int MT, int TN>
pq_status launch_stream_tn(const A8Args &a, hipStream_t s)
{
    constexpr int threads = 64 * StreamShape<BITS, TN, XI, MT>::NW;
    hipLaunchKernelGGL((k_a8_stream<BITS, TN, XI, MT>), dim3(static_cast<unsigned>((a.N + 16 * TN - 1) / (16 * TN))), dim3(threads), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

// Column tiles a block: four or two while that leaves over 192 blocks (16 rows
// of 14336 columns, K = 4096: 224 blocks of four 6.8 us, 448 of two 10.0: the
// activations are read once a block).
template <int BITS, int XI, int MT = 1>
pq_status launch_stream(const A8Args &a, hipStream_t s)
{
    if (a.N > 2 * kStreamPair) return launch_stream_tn<BITS, XI, MT, 4>(a, s);
    if (a.N > kStreamPair) return launch_stream_tn<BITS, XI, MT, 2>(a, s);
    return launch_stream_tn<BITS, XI, MT, 1>(a, s);
}

template <int BITS>
pq_status launch_a8(const A8Args &a, const A8Plan &plan, hipStream_t s)
{
    if (plan.mt == 0) {
        constexpr int RPL = 1024 / (512 / BITS);
        const int xi = (a.M + RPL - 1) / RPL;           // loads of activations a group
        if (xi == 1) return launch_stream<BITS, 1>(a, s);
        if (xi == 2) return launch_stream<BITS, 2>(a, s);
        if constexpr (RPL <= 4) {
            if (xi <= 4) return launch_stream<BITS, 4>(a, s);
        }
        if constexpr (RPL <= 2) return launch_stream<BITS, 8>(a, s);
        if constexpr (RPL > 2) return launch_stream<BITS, 32 / RPL, 2>(a, s);
    }
    // The large tile's ring has the slots that let two blocks share a CU's LDS, at 4
    // bits two: with three the 8192 x 14336 x 4096 of 3 and 4 bits take 502 and 494
    // us, with two 404 and 417 (2 bits 407 with either).
    if (plan.mt == 2) return launch_tile<BITS, 2, 2, 2, 2, 4>(a, s);
    if (plan.mt == 4 && plan.groups == 2) return launch_tile<BITS, 4, 2, 4, 2, 3>(a, s);
    if (plan.mt == 4) return launch_tile<BITS, 4, 1, 4, 2, 4>(a, s);
    return launch_tile<BITS, 4, 1, 8, 4, BITS == 4 ? 2 : 3>(a, s);
}

inline bool a8_shape_ok(int mode, int64_t M, int64_t N, int64_t K)
{
    return valid_mode(mode) && M >= 0 && M <= kMaxA8 && N >= 0 && N <= kMaxA8 && K > 0 && K % 64 == 0 && K <= kMaxA8K;
}

// The mode's levels as whole numbers of a unit, and how the kernels decode them.
inline void set_levels(A8Args &a, int mode)
{
    auto lut = [&](int l0, int l1, int l2, int l3, float unit) {
        a.lut = (l0 & 255u) | (l1 & 255u) << 8 | (l2 & 255u) << 16 | (l3 & 255u) << 24;
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
    if (!pq::a8_shape_ok(mode, M, N, K)) return -1;
    if (M == 0 || N == 0) return 0;
    const pq::A8Plan p = pq::a8_plan(pq::code_bits(mode), M, N, K);
    return p.splits > 1 ? p.splits * M * p.p_st * 4 : 0;
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
    if (rows_overlap(M, N, y_stride)) return PQ_ERR_SHAPE;
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
    const A8Plan plan = a8_plan(code_bits(mode), M, N, K);
    a.splits = plan.splits;
    a.p_st = plan.p_st;
    // An output of half the memory-side cache's size and more is not written
    // into the caches (16384 x 14336 x 576 in bf16 190 us against 198, in fp32 272
    // against 281; 8192 x 14336 x 4096 with a second operand 410 against 416).
    a.nt = M * N * size >= (int64_t(1) << 27);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int bits = code_bits(mode);
    return bits == 1 ? launch_a8<1>(a, plan, s) : bits == 2 ? launch_a8<2>(a, plan, s) : launch_a8<4>(a, plan, s);
}

}  // extern "C"
