// head_norm_rotary.cu -- norm of every query and key head and its rotation to the
// token's position in one pass, and the gradient of both.
//
// Forward, a head row x of D channels:  r = (mean(x^2) + eps)^-1/2, y = R(pos) (w x r).
// Backward, with dn = R^T dy and u = w dn:
//     dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of dn x r
// so one look at x and dy gives both means, and nothing of the forward is kept.
//
// A head row is a group of G lanes, each with 16 channels: both chunks of 8 that a
// rotation pairs, or 16 channels behind the rotated ones.  The lanes of a group walk over
// the heads of their token with its angles and the weights in registers.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

struct HeadParams {
    int64_t T, table_rows;
    int hq, hk, D, units, rot_units, half, splits;   // units: 16-channel pieces of a head
    int64_t q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h, dq_t, dq_h, dk_t, dk_h;
    const uint16_t *q, *k, *dq, *dk, *w_q, *w_k;
    uint16_t *qo, *ko;
    const float* table;
    const int32_t* pos;
    float* part;
    int32_t* status;
    float eps, inv_d;
};

constexpr int kThreads = 256;

// Where this lane's two chunks of 8 channels stand in a head.
template <bool PAIRS>
struct Place {
    int c0, c1;
    bool rot, one, two;   // rotated; the first chunk exists; the second does
    __device__ Place(const HeadParams& p, int u) {
        rot = u < p.rot_units;
        const int rest = 16 * u;
        c0 = rot ? (PAIRS ? 16 * u : 8 * u) : rest;
        c1 = rot ? (PAIRS ? c0 + 8 : c0 + p.half) : rest + 8;
        one = u < p.units;
        two = one && c1 < p.D;
    }
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Turns the 8 pairs of a lane's 16 channels; cs[i] = {cos, sin}.
template <bool PAIRS>
__device__ __forceinline__ void turn(float (&f)[16], const float2 (&cs)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = PAIRS ? 2 * i : i, ib = PAIRS ? 2 * i + 1 : i + 8;
        const float x = f[ia], y = f[ib];
        f[ia] = x * cs[i].x - y * cs[i].y;
        f[ib] = y * cs[i].x + x * cs[i].y;
    }
}

__device__ __forceinline__ void load_angles(const HeadParams& p, int64_t pos, int u, float sign,
                                            float2 (&cs)[8]) {
    const float4* tab = reinterpret_cast<const float4*>(p.table + (pos * p.half + 8 * u) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 v = __ldg(tab + e);
        cs[2 * e] = make_float2(v.x, sign * v.y);
        cs[2 * e + 1] = make_float2(v.z, sign * v.w);
    }
}

__device__ __forceinline__ void load16(const uint16_t* s, int c0, int c1, bool one, bool two,
                                       uint4& a, uint4& b) {
    a = one ? *reinterpret_cast<const uint4*>(s + c0) : make_uint4(0, 0, 0, 0);
    b = two ? *reinterpret_cast<const uint4*>(s + c1) : make_uint4(0, 0, 0, 0);
}

constexpr int kHeads = 4;   // heads that a lane of the forward has under way at once

template <bool PAIRS, int G>
__global__ void __launch_bounds__(kThreads, 3) head_norm_kernel(const HeadParams p) {
    const int lane = threadIdx.x & 31, u = lane & (G - 1);
    const unsigned mask = (G == 32 ? 0xffffffffu : ((1u << G) - 1u)) << (lane & ~(G - 1));
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / G;
    const int64_t t = item / p.splits;
    const int split = static_cast<int>(item - t * p.splits);
    if (t >= p.T) return;
    const Place<PAIRS> at(p, u);
    if (!moe_check((!at.one || at.c0 + 8 <= p.D) && (!at.two || at.c1 + 8 <= p.D), 1601)) return;
    const int heads = p.hq + p.hk;
    float2 cs[8];
    uint4 wq[2], wk[2];
    bool ready = false;
    for (int h0 = split; h0 < heads; h0 += kHeads * p.splits) {
        uint4 a[kHeads], b[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = h0 + j * p.splits;
            const uint16_t* s = h < p.hq ? p.q + t * p.q_t + h * p.q_h
                                         : p.k + t * p.k_t + (h - p.hq) * p.k_h;
            load16(s, at.c0, at.c1, at.one && h < heads, at.two && h < heads, a[j], b[j]);
        }
        if (!ready) {   // behind the first heads' loads, so that the waits overlap
            if (p.table) {
                const int64_t pos = p.pos ? p.pos[t] : t;
                if (pos < 0 || pos >= p.table_rows) {
                    report_error(p.status, MOE_EINVAL);
                    return;
                }
                if (at.rot) load_angles(p, pos, u, 1.0f, cs);
            }
            load16(p.w_q, at.c0, at.c1, at.one, at.two, wq[0], wq[1]);
            if (p.hk) load16(p.w_k, at.c0, at.c1, at.one, at.two, wk[0], wk[1]);
            ready = true;
        }
        float ss[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            float f[16];
            unpack8(a[j], f);
            unpack8(b[j], f + 8);
            ss[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss[j] = fmaf(f[i], f[i], ss[j]);
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
            for (int j = 0; j < kHeads; ++j) ss[j] += __shfl_xor_sync(mask, ss[j], o);
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = h0 + j * p.splits;
            if (h >= heads) continue;
            const float r = rsqrtf(fmaf(ss[j], p.inv_d, p.eps));
            float f[16], w[16];
            unpack8(a[j], f);
            unpack8(b[j], f + 8);
            unpack8(h < p.hq ? wq[0] : wk[0], w);
            unpack8(h < p.hq ? wq[1] : wk[1], w + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
            if (at.rot) turn<PAIRS>(f, cs);
            uint16_t* o = h < p.hq ? p.qo + t * p.qo_t + h * p.qo_h
                                   : p.ko + t * p.ko_t + (h - p.hq) * p.ko_h;
            if (at.one) *reinterpret_cast<uint4*>(o + at.c0) = pack8(f);
            if (at.two) *reinterpret_cast<uint4*>(o + at.c1) = pack8(f + 8);
        }
    }
}

constexpr int kBwdHeads = 2;

// The heads h0, h0 + step, ... < n of one token: their gradients, and their part of dw.
template <bool PAIRS, int G>
__device__ __forceinline__ void backward_heads(const HeadParams& p, const Place<PAIRS>& at,
                                               unsigned mask, const uint16_t* x, int64_t x_h,
                                               const uint16_t* dy, int64_t dy_h, uint16_t* dx,
                                               int64_t dx_h, int h0, int n, const uint4 (&wv)[2],
                                               const float2 (&cs)[8], float (&dw)[16]) {
    for (; h0 < n; h0 += kBwdHeads * p.splits) {
        uint4 xa[kBwdHeads], xb[kBwdHeads], ya[kBwdHeads], yb[kBwdHeads];
#pragma unroll
        for (int j = 0; j < kBwdHeads; ++j) {
            const int h = h0 + j * p.splits;
            load16(x + h * x_h, at.c0, at.c1, at.one && h < n, at.two && h < n, xa[j], xb[j]);
            load16(dy + h * dy_h, at.c0, at.c1, at.one && h < n, at.two && h < n, ya[j], yb[j]);
        }
#pragma unroll
        for (int j = 0; j < kBwdHeads; ++j) {
            const int h = h0 + j * p.splits;
            float f[16], d[16], w[16];
            unpack8(xa[j], f);
            unpack8(xb[j], f + 8);
            unpack8(ya[j], d);
            unpack8(yb[j], d + 8);
            unpack8(wv[0], w);
            unpack8(wv[1], w + 8);
            if (at.rot) turn<PAIRS>(d, cs);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                ss = fmaf(f[i], f[i], ss);
                dot = fmaf(d[i] * w[i], f[i], dot);
            }
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(mask, ss, o);
                dot += __shfl_xor_sync(mask, dot, o);
            }
            if (h >= n) continue;
            const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
            const float c = dot * p.inv_d * r * r;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                dw[i] = fmaf(d[i], f[i] * r, dw[i]);
                f[i] = r * fmaf(-c, f[i], d[i] * w[i]);
            }
            if (at.one) *reinterpret_cast<uint4*>(dx + h * dx_h + at.c0) = pack8(f);
            if (at.two) *reinterpret_cast<uint4*>(dx + h * dx_h + at.c1) = pack8(f + 8);
        }
    }
}

template <bool PAIRS, int G>
__global__ void __launch_bounds__(kThreads, 2) head_norm_bwd_kernel(const HeadParams p) {
    __shared__ float red[kThreads / G][G * 16];
    const int lane = threadIdx.x & 31, u = lane & (G - 1), group = threadIdx.x / G;
    const unsigned mask = (G == 32 ? 0xffffffffu : ((1u << G) - 1u)) << (lane & ~(G - 1));
    const Place<PAIRS> at(p, u);
    if (!moe_check((!at.one || at.c0 + 8 <= p.D) && (!at.two || at.c1 + 8 <= p.D), 1602)) return;
    uint4 wq[2], wk[2];
    load16(p.w_q, at.c0, at.c1, at.one, at.two, wq[0], wq[1]);
    load16(p.w_k, at.c0, at.c1, at.one && p.hk, at.two && p.hk, wk[0], wk[1]);
    float dwq[16], dwk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) dwq[i] = dwk[i] = 0.0f;
    const int64_t items = p.T * p.splits;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / G) + group; item < items;
         item += static_cast<int64_t>(gridDim.x) * (kThreads / G)) {
        const int64_t t = item / p.splits;
        const int split = static_cast<int>(item - t * p.splits);
        float2 cs[8];
        if (p.table) {
            const int64_t pos = p.pos ? p.pos[t] : t;
            if (pos < 0 || pos >= p.table_rows) {
                report_error(p.status, MOE_EINVAL);
                continue;
            }
            if (at.rot) load_angles(p, pos, u, -1.0f, cs);
        }
        backward_heads<PAIRS, G>(p, at, mask, p.q + t * p.q_t, p.q_h, p.dq + t * p.dq_t, p.dq_h,
                                 p.qo + t * p.qo_t, p.qo_h, split, p.hq, wq, cs, dwq);
        if (p.hk)
            backward_heads<PAIRS, G>(p, at, mask, p.k + t * p.k_t, p.k_h, p.dk + t * p.dk_t,
                                     p.dk_h, p.ko + t * p.ko_t, p.ko_h, split, p.hk, wk, cs, dwk);
    }
    // the block's sums, its groups in their order
    for (int kind = 0; kind < 2; ++kind) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) red[group][u * 16 + i] = kind ? dwk[i] : dwq[i];
        __syncthreads();
        for (int e = threadIdx.x; e < p.units * 16; e += kThreads) {
            const Place<PAIRS> pl(p, e >> 4);
            const int i = e & 15, c = i < 8 ? pl.c0 + i : pl.c1 + i - 8;
            if (i >= 8 && !pl.two) continue;
            float s = 0.0f;
            for (int g = 0; g < kThreads / G; ++g) s += red[g][e];
            p.part[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * p.D + c] = s;
        }
    }
}

// dw_q, dw_k: the blocks' sums, 32 runs of blocks side by side and then their 32 sums.
__global__ void __launch_bounds__(1024) head_norm_sums_kernel(const float* part, int blocks, int D,
                                                              float* dw_q, float* dw_k) {
    __shared__ float red[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are complete
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * D)
        for (int b = run; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * 2 * D + c];
    red[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < 2 * D) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        if (c < D)
            dw_q[c] = s;
        else if (dw_k)
            dw_k[c - D] = s;
    }
}

HeadParams head_params(const moe_head_norm_t& c) {
    HeadParams p = {};
    p.T = c.T;
    p.table_rows = c.table_rows;
    p.hq = c.hq;
    p.hk = c.hk;
    p.D = c.D;
    p.rot_units = c.rot_dim / 16;
    p.units = (c.D + 15) / 16;
    p.half = c.rot_dim / 2;
    p.q_t = c.q_t;
    p.q_h = c.q_h;
    p.k_t = c.k_t;
    p.k_h = c.k_h;
    p.qo_t = c.qo_t;
    p.qo_h = c.qo_h;
    p.ko_t = c.ko_t;
    p.ko_h = c.ko_h;
    p.dq_t = c.dq_t;
    p.dq_h = c.dq_h;
    p.dk_t = c.dk_t;
    p.dk_h = c.dk_h;
    p.eps = c.eps;
    p.inv_d = 1.0f / static_cast<float>(c.D);
    return p;
}

int lanes_of(int units) { return units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32; }

// The heads of a token are split over several groups of lanes while there are too few
// tokens to fill the machine.
int head_splits(int64_t T, int lanes, int most, int64_t threads) {
    const int64_t have = T * lanes;
    int64_t s = (threads + have - 1) / have;
    if (s > most) s = most;
    return s < 1 ? 1 : static_cast<int>(s);
}

constexpr int kMaxParts = 2 * 160;   // blocks of a backward launch, on a device of 160 SMs at most

template <bool PAIRS>
void start_forward(const HeadParams& p, int lanes, int grid, cudaStream_t st) {
    switch (lanes) {
        case 4: head_norm_kernel<PAIRS, 4><<<grid, kThreads, 0, st>>>(p); break;
        case 8: head_norm_kernel<PAIRS, 8><<<grid, kThreads, 0, st>>>(p); break;
        case 16: head_norm_kernel<PAIRS, 16><<<grid, kThreads, 0, st>>>(p); break;
        default: head_norm_kernel<PAIRS, 32><<<grid, kThreads, 0, st>>>(p); break;
    }
}

template <bool PAIRS>
void start_backward(const HeadParams& p, int lanes, int grid, cudaStream_t st) {
    switch (lanes) {
        case 4: head_norm_bwd_kernel<PAIRS, 4><<<grid, kThreads, 0, st>>>(p); break;
        case 8: head_norm_bwd_kernel<PAIRS, 8><<<grid, kThreads, 0, st>>>(p); break;
        case 16: head_norm_bwd_kernel<PAIRS, 16><<<grid, kThreads, 0, st>>>(p); break;
        default: head_norm_bwd_kernel<PAIRS, 32><<<grid, kThreads, 0, st>>>(p); break;
    }
}

}  // namespace

int check_status_head_norm() { return moe_check_read_reset(); }

int64_t head_norm_backward_ws(int D) { return static_cast<int64_t>(kMaxParts) * 2 * D * 4; }

int launch_head_norm(const moe_head_norm_t& c, const uint16_t* q, const uint16_t* k,
                     const uint16_t* w_q, const uint16_t* w_k, const float* table,
                     const int32_t* pos, uint16_t* q_out, uint16_t* k_out, int32_t* status,
                     cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    HeadParams p = head_params(c);
    p.q = q;
    p.k = k;
    p.w_q = w_q;
    p.w_k = w_k;
    p.table = c.rot_dim ? table : nullptr;
    p.pos = pos;
    p.qo = q_out;
    p.ko = k_out;
    p.status = status;
    const int lanes = lanes_of(p.units);
    p.splits = head_splits(c.T, lanes, (c.hq + c.hk + kHeads - 1) / kHeads,
                           static_cast<int64_t>(sms) * 3 * kThreads * 8);
    const int64_t grid = (c.T * p.splits * lanes + kThreads - 1) / kThreads;
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    if (c.interleaved)
        start_forward<true>(p, lanes, static_cast<int>(grid), st);
    else
        start_forward<false>(p, lanes, static_cast<int>(grid), st);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "head_norm_rotary");
    return MOE_OK;
}

int launch_head_norm_backward(const moe_head_norm_t& c, const uint16_t* dq, const uint16_t* dk,
                              const uint16_t* q, const uint16_t* k, const uint16_t* w_q,
                              const uint16_t* w_k, const float* table, const int32_t* pos,
                              uint16_t* dq_out, uint16_t* dk_out, float* dw_q, float* dw_k,
                              void* ws, int32_t* status, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    HeadParams p = head_params(c);
    p.q = q;
    p.k = k;
    p.dq = dq;
    p.dk = dk;
    p.w_q = w_q;
    p.w_k = w_k;
    p.table = c.rot_dim ? table : nullptr;
    p.pos = pos;
    p.qo = dq_out;
    p.ko = dk_out;
    p.part = static_cast<float*>(ws);
    p.status = status;
    const int lanes = lanes_of(p.units);
    p.splits = head_splits(c.T, lanes, c.hq, static_cast<int64_t>(sms) * 2 * kThreads);
    const int64_t need = (c.T * p.splits * lanes + kThreads - 1) / kThreads;
    const int64_t most = sms * 2 < kMaxParts ? sms * 2 : kMaxParts;
    const int grid = static_cast<int>(need < most ? need : most);
    if (c.interleaved)
        start_backward<true>(p, lanes, grid, st);
    else
        start_backward<false>(p, lanes, grid, st);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "head_norm_rotary_bwd");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((2 * c.D + 31) / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, head_norm_sums_kernel, static_cast<const float*>(p.part), grid,
                           c.D, dw_q, dw_k) != cudaSuccess)
        return MOE_ECUDA;
    trace_after(st, "head_norm_rotary_sums");
    return MOE_OK;
}

}  // namespace moe
