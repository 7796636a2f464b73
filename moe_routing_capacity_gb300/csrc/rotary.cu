// rotary.cu -- rotary positions: the table of angles, and the rotation of the
// query and key heads.
//
// The rotation reads and writes every head once and is bound by those bytes.
// A thread owns 16 channels of a token (8 pairs): it loads their 8 cosines
// and sines once and walks over the heads with them, two 16-byte loads and
// stores a head.  Neighbouring threads own neighbouring channels, so a warp
// covers whole 128-byte lines.  The heads of a token are split over several
// threads when there are too few tokens to fill the machine.
//   65536 tokens of 56 heads of 128 (1.9 GB moved): 282 us, 6.67 TB/s, what a copy
// reaches.  8192 tokens of 20 heads (84 MB): 18.5 us where heads are strided (15.7
// where they are not), of which 12.4 are the bytes at that rate.  The rest is three
// loads one behind the other (the position, its angles, then the heads), which each of
// 2.8 rounds of CTAs waits for again.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

__global__ void __launch_bounds__(256)
    rotary_table_kernel(const moe_rotary_table_t c, double base, float2* table) {
    const int half = c.rot_dim / 2;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= c.rows * half) return;
    const int64_t pos = i / half;
    const int pair = static_cast<int>(i - pos * half);
    double f = pow(base, -2.0 * pair / c.rot_dim);
    if (c.scaling == 1) f /= c.factor;
    if (c.scaling == 3) {
        const double turns = c.orig_len * f / 6.283185307179586476925;
        double keep = (turns - c.beta_slow) / (c.beta_fast - c.beta_slow);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        f = f * keep + f / c.factor * (1 - keep);
    }
    double s, co;
    sincos(static_cast<double>(pos) * f, &s, &co);
    table[i] = make_float2(static_cast<float>(co * c.magnitude),
                           static_cast<float>(s * c.magnitude));
}

struct RotaryParams {
    int64_t T, table_rows;
    int hq, heads, units, rot_units, half, D;   // units: 16-channel pieces of a head
    int splits, inverse;
    int64_t q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h;
    const uint16_t *q, *k;
    uint16_t *qo, *ko;
    const float* table;
    const int32_t* pos;
    int32_t* status;
};

// Turns pairs (x[i], y[i]); c[i] = {cos, sin}.
__device__ __forceinline__ void turn(uint32_t& xw, uint32_t& yw, const float2& c0,
                                     const float2& c1) {
    const float x0 = bf16_lo(xw), x1 = bf16_hi(xw), y0 = bf16_lo(yw), y1 = bf16_hi(yw);
    xw = pack_bf16x2(x0 * c0.x - y0 * c0.y, x1 * c1.x - y1 * c1.y);
    yw = pack_bf16x2(y0 * c0.x + x0 * c0.y, y1 * c1.x + x1 * c1.y);
}

// Turns the pairs that lie side by side in a word.
__device__ __forceinline__ uint32_t turn_pair(uint32_t w, const float2& c) {
    const float x = bf16_lo(w), y = bf16_hi(w);
    return pack_bf16x2(x * c.x - y * c.y, y * c.x + x * c.y);
}

constexpr int kRotThreads = 256;
constexpr int kRotHeads = 4;     // heads a thread has under way at once
template <bool PAIRS>
__global__ void __launch_bounds__(kRotThreads, 3) rotary_kernel(const RotaryParams p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
    int64_t t;
    int u, split;
    if (p.T * p.units * p.splits < (1ll << 31)) {   // 32-bit divisions where they do
        const uint32_t ts = static_cast<uint32_t>(i) / p.units;
        u = static_cast<int>(static_cast<uint32_t>(i) - ts * p.units);
        const uint32_t t32 = ts / p.splits;
        split = static_cast<int>(ts - t32 * p.splits);
        t = t32;
    } else {
        const int64_t ts = i / p.units;
        u = static_cast<int>(i - ts * p.units);
        t = ts / p.splits;
        split = static_cast<int>(ts - t * p.splits);
    }
    if (t >= p.T) return;
    const int64_t pos = p.pos ? p.pos[t] : t;
    if (pos < 0 || pos >= p.table_rows) {
        report_error(p.status, MOE_EINVAL);
        return;
    }
    // the two 8-channel chunks of this unit, and whether the second exists
    const bool rot = u < p.rot_units;
    const int rest = 16 * p.rot_units + 16 * (u - p.rot_units);
    const int c0 = rot ? (PAIRS ? 16 * u : 8 * u) : rest;
    const int c1 = rot ? (PAIRS ? c0 + 8 : c0 + p.half) : rest + 8;
    const bool two = c1 < p.D;
    if (!moe_check(c0 + 8 <= p.D && (!two || c1 + 8 <= p.D) && split < p.splits, 1221)) return;
    float2 cs[8];
    if (rot) {
        const float4* tab = reinterpret_cast<const float4*>(p.table + (pos * p.half + 8 * u) * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = __ldg(tab + e);
            cs[2 * e] = make_float2(v.x, p.inverse ? -v.y : v.y);
            cs[2 * e + 1] = make_float2(v.z, p.inverse ? -v.w : v.w);
        }
    }
    for (int h0 = split; h0 < p.heads; h0 += kRotHeads * p.splits) {
        uint4 a[kRotHeads], b[kRotHeads];
#pragma unroll
        for (int j = 0; j < kRotHeads; ++j) {
            const int h = h0 + j * p.splits;
            if (h < p.heads) {
                const uint16_t* s = h < p.hq ? p.q + t * p.q_t + h * p.q_h
                                             : p.k + t * p.k_t + (h - p.hq) * p.k_h;
                a[j] = *reinterpret_cast<const uint4*>(s + c0);
                if (two) b[j] = *reinterpret_cast<const uint4*>(s + c1);
            }
        }
#pragma unroll
        for (int j = 0; j < kRotHeads; ++j) {
            const int h = h0 + j * p.splits;
            if (h >= p.heads) continue;
            uint16_t* o = h < p.hq ? p.qo + t * p.qo_t + h * p.qo_h
                                   : p.ko + t * p.ko_t + (h - p.hq) * p.ko_h;
            if (rot) {
                if (PAIRS) {
                    a[j] = make_uint4(turn_pair(a[j].x, cs[0]), turn_pair(a[j].y, cs[1]),
                                      turn_pair(a[j].z, cs[2]), turn_pair(a[j].w, cs[3]));
                    b[j] = make_uint4(turn_pair(b[j].x, cs[4]), turn_pair(b[j].y, cs[5]),
                                      turn_pair(b[j].z, cs[6]), turn_pair(b[j].w, cs[7]));
                } else {
                    turn(a[j].x, b[j].x, cs[0], cs[1]);
                    turn(a[j].y, b[j].y, cs[2], cs[3]);
                    turn(a[j].z, b[j].z, cs[4], cs[5]);
                    turn(a[j].w, b[j].w, cs[6], cs[7]);
                }
            }
            *reinterpret_cast<uint4*>(o + c0) = a[j];
            if (two) *reinterpret_cast<uint4*>(o + c1) = b[j];
        }
    }
}

}  // namespace

int check_status_rotary() { return moe_check_read_reset(); }

int launch_rotary_table(const moe_rotary_table_t& c, float* table, cudaStream_t st) {
    const double base = c.scaling == 2
                            ? c.base * std::pow(c.factor, c.rot_dim / (c.rot_dim - 2.0))
                            : c.base;
    const int64_t n = c.rows * (c.rot_dim / 2);
    if ((n + 255) / 256 >= (1ll << 31)) return MOE_EINVAL;
    rotary_table_kernel<<<static_cast<int>((n + 255) / 256), 256, 0, st>>>(
        c, base, reinterpret_cast<float2*>(table));
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "rotary_table");
    return MOE_OK;
}

int launch_rotary(const moe_rotary_t& c, const uint16_t* q, const uint16_t* k, const float* table,
                  const int32_t* pos, uint16_t* q_out, uint16_t* k_out, int32_t* status,
                  cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    RotaryParams p;
    p.T = c.T;
    p.table_rows = c.table_rows;
    p.hq = c.hq;
    p.heads = c.hq + c.hk;
    p.rot_units = c.rot_dim / 16;
    // channels past rot_dim are copied, or already in their place
    const bool in_place = q == q_out && (c.hk == 0 || k == k_out);
    p.units = p.rot_units + (in_place ? 0 : (c.D - c.rot_dim + 15) / 16);
    p.half = c.rot_dim / 2;
    p.D = c.D;
    p.inverse = c.inverse;
    p.q_t = c.q_t;
    p.q_h = c.q_h;
    p.k_t = c.k_t;
    p.k_h = c.k_h;
    p.qo_t = c.qo_t;
    p.qo_h = c.qo_h;
    p.ko_t = c.ko_t;
    p.ko_h = c.ko_h;
    p.q = q;
    p.k = k;
    p.qo = q_out;
    p.ko = k_out;
    p.table = table;
    p.pos = pos;
    p.status = status;
    // up to eight rounds of resident CTAs, as long as a thread keeps four heads: a
    // short last round costs little (65536 tokens x 56 heads 291 -> 282 us against
    // one round; 8192 x 20, where the four heads allow five splits and 2.8 rounds,
    // 20.5 -> 18.5 us)
    const int64_t want = static_cast<int64_t>(sms) * 3 * kRotThreads * 8;
    const int64_t have = c.T * p.units;
    int64_t splits = (want + have - 1) / have;
    const int most = (p.heads + kRotHeads - 1) / kRotHeads;
    if (splits > most) splits = most;
    p.splits = splits < 1 ? 1 : static_cast<int>(splits);
    const int64_t grid = (c.T * p.splits * p.units + kRotThreads - 1) / kRotThreads;
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    if (c.interleaved)
        rotary_kernel<true><<<static_cast<int>(grid), kRotThreads, 0, st>>>(p);
    else
        rotary_kernel<false><<<static_cast<int>(grid), kRotThreads, 0, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "rotary");
    return MOE_OK;
}

}  // namespace moe
