// pq_rope.hip -- gfx950 kernels and C entry points for rotary positions: the
// (cos, sin) table of a model and the rotation of queries and keys by it.
//
// The rotation of a pair (x1, x2) by angle a is (x1 cos a - x2 sin a,
// x2 cos a + x1 sin a); its transpose, which is its inverse and the gradient's
// map, is the rotation by -a.  Three multiply-adds a channel on 4 bytes of
// traffic (16-bit types): the memory system bounds it.  The angles come from a
// table, not from sin and cos in place: p f_c in binary32 is off by p 2^-24
// turns of a radian, 0.004 at position 65536, while the table's rows are
// rounded from binary64 and cost one row per token, shared by all its heads.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pq_kv_common.hpp"

namespace pq {
namespace {

struct TableArgs {
    float *table;
    int64_t rows;
    int pairs, kind;
    double log_base;        // natural logarithm of the (NTK: scaled) base
    double inv_factor, magnitude;
    double a, b;            // YARN: lo, 1 / (hi - lo); BANDS: beta_slow, 1 / (beta_fast - beta_slow)
    double trained;
};

// Frequency of pair c in radians per position, binary64.
__device__ __forceinline__ double table_freq(const TableArgs &t, int c)
{
    const double f = exp(-t.log_base * (static_cast<double>(c) / t.pairs));
    double g = 1.0;         // share of the unscaled frequency
    if (t.kind == PQ_ROPE_LINEAR) g = 0.0;
    if (t.kind == PQ_ROPE_YARN) g = 1.0 - fmin(fmax((c - t.a) * t.b, 0.0), 1.0);
    if (t.kind == PQ_ROPE_BANDS) {
        const double turns = t.trained * f * 0.15915494309189533577;   // trained / wavelength
        g = fmin(fmax((turns - t.a) * t.b, 0.0), 1.0);
    }
    return f * ((1.0 - g) * t.inv_factor + g);
}

__global__ __launch_bounds__(256) void k_rope_table(TableArgs t)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= t.rows * t.pairs) return;
    const int64_t p = i / t.pairs;
    double s, c;
    sincos(static_cast<double>(p) * table_freq(t, static_cast<int>(i - p * t.pairs)), &s, &c);
    t.table[2 * i] = static_cast<float>(c * t.magnitude);
    t.table[2 * i + 1] = static_cast<float>(s * t.magnitude);
}

struct RopeArgs {
    const void *x;
    void *y;
    int64_t x_ts, x_hs, y_ts, y_hs;   // elements
    const int32_t *positions;
    const float *table;
    int64_t tokens;
    int heads, dim, rot, max_pos, half;
    int rot_units, units;             // units of VP pairs (or 2 VP copied channels) per head
    int head_lanes, slices;           // heads side by side in a wave; waves per token
    float sign;                       // -1: inverse
};

// One wave per token and slice of its heads.  A lane keeps one unit -- VP
// pairs, with their 2 VP table values in registers -- and walks the heads, so
// that the table is read once per token and wave and not once per head.
template <typename T, int VP, bool NT>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a)
{
    const int64_t token = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    if (token >= a.tokens) return;
    const int lane = threadIdx.x & 63;
    const int hl = lane / a.units;                  // 0 when the units take several lane rounds
    if (hl >= a.head_lanes) return;
    const int h0 = hl + a.head_lanes * static_cast<int>(blockIdx.y), step = a.head_lanes * a.slices;
    const int pos = a.positions[token];
    const T *x = static_cast<const T *>(a.x) + token * a.x_ts;
    T *y = static_cast<T *>(a.y) + token * a.y_ts;
    for (int u = lane - hl * a.units; u < a.units; u += 64) {
        const bool turn = u < a.rot_units && pos >= 0;
        float c[VP] = {}, s[VP] = {};
        int o1, o2;                                 // channels of the unit's two vectors
        if (u < a.rot_units) {
            o1 = a.half ? u * VP : 2 * u * VP;
            o2 = a.half ? o1 + a.rot / 2 : o1 + VP;
        } else {
            o1 = a.rot + 2 * (u - a.rot_units) * VP;
            o2 = VP == 1 ? min(o1 + 1, a.dim - 1) : o1 + VP;   // an odd rest: its last channel twice
        }
        if (turn) {
            float cs[2 * VP];
            if (pos < a.max_pos) {
                const float *row = a.table + (static_cast<int64_t>(pos) * (a.rot / 2) + u * VP) * 2;
                if constexpr (VP == 1) {
                    cs[0] = row[0];
                    cs[1] = row[1];
                } else {
                    load_f32<float, 2 * VP>(row, cs);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2 * VP; ++e) cs[e] = __builtin_nanf("");
            }
#pragma unroll
            for (int e = 0; e < VP; ++e) {
                c[e] = cs[2 * e];
                s[e] = cs[2 * e + 1] * a.sign;
            }
        }
        constexpr int B = 4;                        // heads in flight per lane
        for (int h = h0; h < a.heads; h += B * step) {
            float p[B][VP], q[B][VP];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int64_t hh = min(h + b * step, a.heads - 1);
                load_f32<T, VP>(x + hh * a.x_hs + o1, p[b]);
                load_f32<T, VP>(x + hh * a.x_hs + o2, q[b]);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (h + b * step >= a.heads) break;
                float r1[VP], r2[VP];
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    // half: p, q are x1, x2; interleaved: p holds the first VP
                    // channels of the unit, pairs inside
                    if (a.half || VP == 1) {
                        r1[e] = p[b][e] * c[e] - q[b][e] * s[e];
                        r2[e] = q[b][e] * c[e] + p[b][e] * s[e];
                    } else {
                        const int i = e >> 1;       // pair inside p; q's pairs follow
                        r1[e] = e & 1 ? p[b][e] * c[i] + p[b][e ^ 1] * s[i] : p[b][e] * c[i] - p[b][e ^ 1] * s[i];
                        const int j = VP / 2 + i;
                        r2[e] = e & 1 ? q[b][e] * c[j] + q[b][e ^ 1] * s[j] : q[b][e] * c[j] - q[b][e ^ 1] * s[j];
                    }
                }
                T *out = y + static_cast<int64_t>(h + b * step) * a.y_hs;
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    r1[e] = turn ? r1[e] : p[b][e];
                    r2[e] = turn ? r2[e] : q[b][e];
                }
                store_f32<T, VP, NT>(out + o1, r1);
                store_f32<T, VP, NT>(out + o2, r2);
            }
        }
    }
}

template <typename T, int VP>
pq_status launch_rope(RopeArgs a, bool in_place, hipStream_t s)
{
    a.rot_units = a.rot / (2 * VP);
    // in place the channels past `rot` stay as they are
    a.units = a.rot_units + (in_place ? 0 : (a.dim - a.rot + 2 * VP - 1) / (2 * VP));
    if (a.units == 0) return PQ_OK;
    a.head_lanes = a.units >= 64 ? 1 : 64 / a.units;
    const int rounds = (a.heads + a.head_lanes - 1) / a.head_lanes;   // head steps of one wave per token
    // Few tokens: a token's heads go to several waves, until the chip has
    // about eight waves per CU or every wave has one step left (4 tokens of 40
    // heads 3.2 us, unsliced 4.1).
    int64_t slices = (2048 + a.tokens - 1) / a.tokens;
    if (slices > rounds) slices = rounds;
    a.slices = static_cast<int>(slices);
    const int64_t blocks = (a.tokens + 3) / 4;
    if (blocks > kMaxBlocks) return PQ_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(slices));
    // Past the memory-side cache (256 MB) the rotated heads are not written
    // into the caches: the 8 x 2048 batch (340 MB) 60 us against 63.  A smaller
    // result may be found there by its reader: 66 MB in fp32 13.5 us against 17.6.
    if (static_cast<double>(a.tokens) * a.heads * a.dim * 2 * sizeof(T) > 0x1p28)
        hipLaunchKernelGGL((k_rope<T, VP, true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_rope<T, VP, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

}  // namespace
}  // namespace pq

extern "C" {

pq_status pq_rope_table(int64_t max_pos, int64_t rot, double base, const pq_rope_scaling *scaling, float *table,
                        void *stream)
{
    using namespace pq;
    if (max_pos < 0 || max_pos > INT32_MAX || rot < 2 || rot > 1024 || rot % 2) return PQ_ERR_SHAPE;
    if (!(base > 1.0) || !std::isfinite(base)) return PQ_ERR_ARG;
    TableArgs t = {};
    t.kind = scaling ? scaling->kind : PQ_ROPE_PLAIN;
    if (t.kind < PQ_ROPE_PLAIN || t.kind > PQ_ROPE_BANDS) return PQ_ERR_MODE;
    if (scaling && scaling->reserved != 0) return PQ_ERR_ARG;
    t.table = table;
    t.rows = max_pos;
    t.pairs = static_cast<int>(rot / 2);
    t.log_base = std::log(base);
    t.inv_factor = 1.0;
    t.magnitude = 1.0;
    if (t.kind != PQ_ROPE_PLAIN) {
        const double s = scaling->factor;
        if (!(s >= 1.0) || !std::isfinite(s)) return PQ_ERR_ARG;
        t.inv_factor = 1.0 / s;
        if (t.kind == PQ_ROPE_NTK) {
            if (rot <= 2) return PQ_ERR_SHAPE;
            t.log_base += std::log(s) * static_cast<double>(rot) / static_cast<double>(rot - 2);
        }
        if (t.kind == PQ_ROPE_YARN || t.kind == PQ_ROPE_BANDS) {
            const double L = scaling->trained, fast = scaling->beta_fast, slow = scaling->beta_slow;
            if (!(L > 0.0) || !std::isfinite(L) || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast))
                return PQ_ERR_ARG;
            t.trained = L;
            if (t.kind == PQ_ROPE_YARN) {
                // pair index whose wavelength fits `turns` times into L
                auto index = [&](double turns) {
                    return static_cast<double>(rot) * std::log(L / (turns * 2.0 * M_PI)) / (2.0 * t.log_base);
                };
                const double top = static_cast<double>(rot - 1);
                const double lo = std::fmin(std::fmax(std::floor(index(fast)), 0.0), top);
                double hi = std::fmin(std::fmax(std::ceil(index(slow)), 0.0), top);
                if (hi <= lo) hi = lo + 0.001;      // a step
                t.a = lo;
                t.b = 1.0 / (hi - lo);
                t.magnitude = 0.1 * std::log(s) + 1.0;
            } else {
                t.a = slow;
                t.b = 1.0 / (fast - slow);
            }
        }
    }
    if (max_pos == 0) return PQ_OK;
    if (!table) return PQ_ERR_NULL;
    if (!aligned16(table)) return PQ_ERR_ALIGN;
    const int64_t blocks = (max_pos * t.pairs + 255) / 256;
    if (blocks > kMaxBlocks) return PQ_ERR_SHAPE;
    hipLaunchKernelGGL(k_rope_table, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), t);
    return hipGetLastError() == hipSuccess ? PQ_OK : PQ_ERR_HIP;
}

pq_status pq_rope(int dtype, int64_t tokens, int64_t heads, int64_t dim, int64_t rot, int layout, int inverse,
                  const void *x, int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions,
                  const float *table, int64_t max_pos, void *y, int64_t y_token_stride, int64_t y_head_stride,
                  void *stream)
{
    using namespace pq;
    const int size = dtype_bytes(dtype);
    if (!size || (layout != PQ_ROPE_HALF && layout != PQ_ROPE_INTERLEAVED)) return PQ_ERR_MODE;
    // the kernel steps through the heads in 32 bits, up to 2^19 at a time
    if (tokens < 0 || heads < 0 || heads > (1 << 30) || dim < 1 || dim > 1024 || rot < 0 || rot > dim || rot % 2)
        return PQ_ERR_SHAPE;
    if (max_pos < 0 || max_pos > INT32_MAX) return PQ_ERR_SHAPE;
    if (tokens == 0 || heads == 0) return PQ_OK;
    if (!x || !y || !positions || (!table && rot > 0 && max_pos > 0)) return PQ_ERR_NULL;
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
    if ((xa | ya) % size || reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(table) % 16)
        return PQ_ERR_ALIGN;
    const bool in_place = x == y;
    if (in_place && (x_token_stride != y_token_stride || x_head_stride != y_head_stride)) return PQ_ERR_ARG;
    RopeArgs a = {};
    a.x = x;
    a.y = y;
    a.x_ts = x_token_stride;
    a.x_hs = x_head_stride;
    a.y_ts = y_token_stride;
    a.y_hs = y_head_stride;
    a.positions = positions;
    a.table = table;
    a.tokens = tokens;
    a.heads = static_cast<int>(heads);
    a.dim = static_cast<int>(dim);
    a.rot = static_cast<int>(rot);
    a.max_pos = static_cast<int>(max_pos);
    a.half = layout == PQ_ROPE_HALF;
    a.sign = inverse ? -1.f : 1.f;
    // Widest vectors that keep every unit whole and aligned: VP pairs a lane
    // (16384 tokens of 40 heads of 128 in bf16 with 8, 4, 1: 61, 63, 69 us;
    // 4099 of 25 heads of 80 in fp32 with 4 and 1: 13 and 16).
    auto fits = [&](int64_t vp) {
        const int64_t bytes = vp * size < 16 ? vp * size : 16;
        const int64_t strides = x_token_stride | x_head_stride | y_token_stride | y_head_stride;
        return rot % (2 * vp) == 0 && (dim - rot) % (2 * vp) == 0 && (xa | ya) % bytes == 0 &&
               (strides * size) % bytes == 0;
    };
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == PQ_F32) return fits(4) ? launch_rope<float, 4>(a, in_place, s) : launch_rope<float, 1>(a, in_place, s);
    if (dtype == PQ_BF16)
        return fits(8)   ? launch_rope<bf16_t, 8>(a, in_place, s)
               : fits(4) ? launch_rope<bf16_t, 4>(a, in_place, s)
                         : launch_rope<bf16_t, 1>(a, in_place, s);
    return fits(8)   ? launch_rope<f16_t, 8>(a, in_place, s)
           : fits(4) ? launch_rope<f16_t, 4>(a, in_place, s)
                     : launch_rope<f16_t, 1>(a, in_place, s);
}

}  // extern "C"
