// norm_residual.cu -- norm after a branch, gate, residual sum and norm before
// the next branch in one pass over the rows, and its gradient.
//
//   p = b rb,  y = alpha r + beta g p w_post,  n = y ry w_pre
// (rb, ry = 1 / root mean square).  Bytes bound both directions: forward b,
// r -> y, n; backward b, r, dn, dy -> db, dr.  Each value is read once: a
// thread holds its 8 channels of a row in registers across the two sums of
// the row, the weights for all its rows.  Rows arrive through a ring of
// cp.async stages, each thread copying what it will read itself, so that the
// loads of the next rows run under the sums of this one and no barrier
// guards the ring.
//   d <= 1024: a warp a row (1, 2 or 4 times 8 channels a lane), 8 rows a CTA.
//   d >  1024: a CTA a row, d / 8 threads.
// The backward's sums over tokens (dw_post, dw_pre, dgate) stay in registers
// over all of a CTA's rows; each CTA writes one partial row and a second
// kernel adds the partials in their order: no atomics.
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

struct NormParams {
    int64_t T;
    int d, chunks;            // chunks = d / 8
    int stages, slots;        // ring depth; 16-byte slots of a thread and chunk
    float alpha, beta, eps, inv_d;
    const uint16_t *b, *gate, *w_post, *w_pre, *dn;
    const void *r, *dy;
    int gate_mode;            // 0 none, 1 [d], 2 [T, d]
    void *y, *dr, *dgate;
    uint16_t *n, *db;
    float *rstd_post, *rstd_pre;          // forward: out
    const float *in_post, *in_pre;        // backward: in
    float* part;                           // [CTAs, 3, d]
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void as_floats(const uint4& a, const uint4& b, float (&f)[8]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the row's threads, the same value in all of them.  `red` is a slot
// of 32 words that no thread still reads (the caller alternates them).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = sum32(v);
    if (WARP) return v;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return sum32(lane < nw ? red[lane] : 0.f);
}

__device__ __forceinline__ void wait_stage(int stages) {
    if (stages == 2)
        cp_async_wait<1>();
    else if (stages == 3)
        cp_async_wait<2>();
    else
        cp_async_wait<3>();
}

// A residual-stream chunk: one slot of bf16 or two of fp32.
template <bool F32>
__device__ __forceinline__ void load_res(const uint4* slot, int pitch, float (&f)[8]) {
    if (F32)
        as_floats(slot[0], slot[pitch], f);
    else
        unpack8(slot[0], f);
}

template <bool F32>
__device__ __forceinline__ void store_res(void* base, int64_t at, const float (&f)[8]) {
    if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(f);
    }
}

template <bool F32>
__device__ __forceinline__ void copy_res(uint32_t dst, uint32_t pitch, const void* base,
                                         int64_t at) {
    if (F32) {
        const float* s = static_cast<const float*>(base) + at;
        cp_async_16(dst, s, 16);
        cp_async_16(dst + pitch, s + 4, 16);
    } else {
        cp_async_16(dst, static_cast<const uint16_t*>(base) + at, 16);
    }
}

// ------------------------------------------------------------------ forward

// Slots of a thread and chunk: b, gate (if per token), r (1 or 2).
template <bool F32, bool WARP, int CH, int NT, int OCC>
__global__ void __launch_bounds__(NT, OCC) norm_fwd_kernel(const NormParams p) {
    extern __shared__ uint4 ring[];
    __shared__ float red[4][32];
    const int nt = blockDim.x;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int gs = WARP ? 32 : nt;
    const int rows = WARP ? nt / 32 : 1;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const bool has_b = p.b != nullptr, has_n = p.n != nullptr;
    const int s_gate = 1, s_r = p.gate_mode == 2 ? 2 : 1;
    const auto slot = [&](int stage, int i, int k) {
        return ((stage * CH + i) * p.slots + k) * nt + static_cast<int>(threadIdx.x);
    };
    const auto fetch = [&](int64_t row, int stage) {
        if (row < p.T) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = lane + gs * i;
                if (c < p.chunks) {
                    const int64_t at = row * p.d + c * 8;
                    if (has_b) cp_async_16(smem_u32(ring + slot(stage, i, 0)), p.b + at, 16);
                    if (p.gate_mode == 2)
                        cp_async_16(smem_u32(ring + slot(stage, i, s_gate)), p.gate + at, 16);
                    copy_res<F32>(smem_u32(ring + slot(stage, i, s_r)), nt * 16, p.r, at);
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);

    uint4 wq[CH], wp[CH], wg[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = lane + gs * i;
        wq[i] = wp[i] = wg[i] = make_uint4(0, 0, 0, 0);
        if (c < p.chunks) {
            if (has_b) wq[i] = *reinterpret_cast<const uint4*>(p.w_post + c * 8);
            if (has_n) wp[i] = *reinterpret_cast<const uint4*>(p.w_pre + c * 8);
            if (p.gate_mode == 1) wg[i] = *reinterpret_cast<const uint4*>(p.gate + c * 8);
        }
    }
    int stage = 0, par = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        wait_stage(p.stages);
        float b[CH][8], y[CH][8];
        uint4 gt[CH];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[i][e] = y[i][e] = 0.f;
            gt[i] = wg[i];
            if (lane + gs * i < p.chunks) {
                if (has_b) unpack8(ring[slot(stage, i, 0)], b[i]);
                if (p.gate_mode == 2) gt[i] = ring[slot(stage, i, s_gate)];
                load_res<F32>(ring + slot(stage, i, s_r), nt, y[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += b[i][e] * b[i][e];
                y[i][e] *= p.alpha;
            }
        }
        fetch(row + p.stages * step, stage);   // this thread has read the slots
        if (++stage == p.stages) stage = 0;
        if (has_b) {
            const float rb = rsqrtf(row_sum<WARP>(ss, red[par]) * p.inv_d + p.eps);
            if (lane == 0 && p.rstd_post) p.rstd_post[row] = rb;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float w[8], g[8];
                unpack8(wq[i], w);
                unpack8(gt[i], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = p.beta * (b[i][e] * rb * w[e]);
                    y[i][e] += p.gate_mode ? u * g[e] : u;
                }
            }
        }
        if (p.y)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (lane + gs * i < p.chunks)
                    store_res<F32>(p.y, row * p.d + (lane + gs * i) * 8, y[i]);
        if (has_n) {
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += y[i][e] * y[i][e];
            const float ry = rsqrtf(row_sum<WARP>(ss, red[2 + par]) * p.inv_d + p.eps);
            if (lane == 0 && p.rstd_pre) p.rstd_pre[row] = ry;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float w[8];
                unpack8(wp[i], w);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] *= y[i][e] * ry;
                if (lane + gs * i < p.chunks)
                    *reinterpret_cast<uint4*>(p.n + row * p.d + (lane + gs * i) * 8) = pack8(w);
            }
        }
        par ^= 1;
    }
}

// ------------------------------------------------------------------ backward

// Slots of a thread and chunk: b, dn, gate (if per token), r, dy (1 or 2 each).
template <bool F32, bool WARP, int CH, int NT, int OCC>
__global__ void __launch_bounds__(NT, OCC) norm_bwd_kernel(const NormParams p) {
    extern __shared__ uint4 ring[];
    __shared__ float red[4][32];
    const int nt = blockDim.x;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int gs = WARP ? 32 : nt;
    const int rows = WARP ? nt / 32 : 1;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const bool has_b = p.b != nullptr, has_n = p.dn != nullptr, has_y = p.dy != nullptr;
    const int s_dn = 1, s_gate = 2, s_r = p.gate_mode == 2 ? 3 : 2, s_dy = s_r + (F32 ? 2 : 1);
    const auto slot = [&](int stage, int i, int k) {
        return ((stage * CH + i) * p.slots + k) * nt + static_cast<int>(threadIdx.x);
    };
    const auto fetch = [&](int64_t row, int stage) {
        if (row < p.T) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = lane + gs * i;
                if (c < p.chunks) {
                    const int64_t at = row * p.d + c * 8;
                    if (has_b) cp_async_16(smem_u32(ring + slot(stage, i, 0)), p.b + at, 16);
                    if (has_n) {
                        cp_async_16(smem_u32(ring + slot(stage, i, s_dn)), p.dn + at, 16);
                        copy_res<F32>(smem_u32(ring + slot(stage, i, s_r)), nt * 16, p.r, at);
                    }
                    if (p.gate_mode == 2)
                        cp_async_16(smem_u32(ring + slot(stage, i, s_gate)), p.gate + at, 16);
                    if (has_y)
                        copy_res<F32>(smem_u32(ring + slot(stage, i, s_dy)), nt * 16, p.dy, at);
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);

    uint4 wq[CH], wp[CH], wg[CH];
    float a_post[CH][8], a_pre[CH][8], a_gate[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = lane + gs * i;
        wq[i] = wp[i] = wg[i] = make_uint4(0, 0, 0, 0);
        if (c < p.chunks) {
            if (has_b) wq[i] = *reinterpret_cast<const uint4*>(p.w_post + c * 8);
            if (has_n) wp[i] = *reinterpret_cast<const uint4*>(p.w_pre + c * 8);
            if (p.gate_mode == 1) wg[i] = *reinterpret_cast<const uint4*>(p.gate + c * 8);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) a_post[i][e] = a_pre[i][e] = a_gate[i][e] = 0.f;
    }
    const auto stat = [&](const float* s, int64_t row) { return s && row < p.T ? s[row] : 0.f; };
    float rb = stat(p.in_post, row0), ry = stat(p.in_pre, row0);
    int stage = 0, par = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        const float rb_next = stat(p.in_post, row + step), ry_next = stat(p.in_pre, row + step);
        wait_stage(p.stages);
        // pv: p; du: first dy, then dL/dy
        float pv[CH][8], q[CH][8], t[CH][8], du[CH][8];
        uint4 gt[CH];
        float s1 = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float dn[8], w[8], g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) pv[i][e] = q[i][e] = du[i][e] = dn[e] = 0.f;
            gt[i] = wg[i];
            if (lane + gs * i < p.chunks) {
                if (has_b) unpack8(ring[slot(stage, i, 0)], pv[i]);
                if (p.gate_mode == 2) gt[i] = ring[slot(stage, i, s_gate)];
                if (has_n) {
                    unpack8(ring[slot(stage, i, s_dn)], dn);
                    load_res<F32>(ring + slot(stage, i, s_r), nt, q[i]);
                }
                if (has_y) load_res<F32>(ring + slot(stage, i, s_dy), nt, du[i]);
            }
            unpack8(wq[i], w);
            unpack8(gt[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                pv[i][e] *= rb;
                const float u = p.beta * (pv[i][e] * w[e]);
                q[i][e] = (p.alpha * q[i][e] + (p.gate_mode ? u * g[e] : u)) * ry;
            }
            unpack8(wp[i], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a_pre[i][e] += dn[e] * q[i][e];
                t[i][e] = dn[e] * w[e];
                s1 += t[i][e] * q[i][e];
            }
        }
        fetch(row + p.stages * step, stage);   // this thread has read the slots
        if (++stage == p.stages) stage = 0;
        const float k1 = has_n ? row_sum<WARP>(s1, red[par]) * p.inv_d : 0.f;
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float w[8], g[8], o[8];
            unpack8(wq[i], w);
            unpack8(gt[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                du[i][e] += ry * (t[i][e] - q[i][e] * k1);
                o[e] = p.alpha * du[i][e];
            }
            const bool in = lane + gs * i < p.chunks;
            const int64_t at = row * p.d + (lane + gs * i) * 8;
            if (in) store_res<F32>(p.dr, at, o);
            if (has_b) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = p.beta * du[i][e];
                    o[e] = v * (pv[i][e] * w[e]);                // the gate's gradient
                    const float dm = p.gate_mode ? v * g[e] : v;
                    a_gate[i][e] += o[e];
                    a_post[i][e] += dm * pv[i][e];
                    du[i][e] = dm * w[e];                        // dL/dp
                    s2 += du[i][e] * pv[i][e];
                }
                if (p.gate_mode == 2 && in)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dgate) + at) = pack8(o);
            }
        }
        if (has_b) {
            const float k2 = row_sum<WARP>(s2, red[2 + par]) * p.inv_d;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = rb * (du[i][e] - pv[i][e] * k2);
                if (lane + gs * i < p.chunks)
                    *reinterpret_cast<uint4*>(p.db + row * p.d + (lane + gs * i) * 8) = pack8(o);
            }
        }
        par ^= 1;
        rb = rb_next;
        ry = ry_next;
    }
    // this CTA's partial sums over its tokens: post, pre, gate
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 3 * p.d;
    float* acc = reinterpret_cast<float*>(ring);
    const int turns = WARP ? rows : 1;
    if (WARP) {
        cp_async_wait<0>();
        __syncthreads();   // every warp is done with the ring, which adds the warps' sums
    }
    for (int w = 0; w < turns; ++w) {
        if (!WARP || static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = lane + gs * i;
                if (c >= p.chunks) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v[3] = {a_post[i][e], a_pre[i][e], a_gate[i][e]};
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const int at = k * p.d + c * 8 + e;
                        const float sum = w ? acc[at] + v[k] : v[k];
                        if (w + 1 < turns)
                            acc[at] = sum;
                        else
                            part[at] = sum;
                    }
                }
            }
        }
        if (WARP) __syncthreads();
    }
}

// out_k[c] = sum over the partial rows, in a fixed order: 32 columns a CTA,
// eight threads a column over an eighth of the rows each.
__global__ void __launch_bounds__(256) norm_sums_kernel(const float* part, int n, int d, float* o0,
                                                        float* o1, float* o2) {
    __shared__ float s[8][32];
    const int x = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float v = 0.f;
    if (col < 3ll * d)
#pragma unroll 8
        for (int i = g; i < n; i += 8) v += part[static_cast<int64_t>(i) * 3 * d + col];
    s[g][x] = v;
    __syncthreads();
    if (g == 0 && col < 3ll * d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][x];
        const int k = static_cast<int>(col / d);
        float* o = k == 0 ? o0 : k == 1 ? o1 : o2;
        if (o) o[col - static_cast<int64_t>(k) * d] = v;
    }
}

// One launch shape for a width: threads, chunks a thread, CTAs an SM.
struct Shape {
    int threads, rows, occ, grid, stages, smem;
};

// ring budget of an SM; a CTA's share keeps room for its 512 bytes of sums
constexpr int kRingBytes = 220 * 1024;

Shape norm_shape(int64_t T, int d, int slots, int sms, bool bwd) {
    Shape s;
    const int chunks = d / 8;
    int per_thread = 1;
    if (chunks <= 128) {
        s.threads = 256;
        s.rows = 8;
        per_thread = chunks <= 32 ? 1 : chunks <= 64 ? 2 : 4;
        s.occ = per_thread == 4 ? (bwd ? 1 : 2) : (bwd ? 2 : 4);
    } else {
        s.threads = (chunks + 31) / 32 * 32;
        s.rows = 1;
        s.occ = s.threads <= 256 ? (bwd ? 2 : 4) : s.threads <= 512 ? (bwd ? 1 : 2) : 1;
    }
    const int stage_bytes = s.threads * per_thread * slots * 16;
    s.stages = kRingBytes / s.occ / stage_bytes;
    s.stages = s.stages > 4 ? 4 : s.stages < 2 ? 2 : s.stages;
    s.smem = s.stages * stage_bytes;
    if (bwd && s.rows > 1 && s.smem < 3 * d * 4) s.smem = 3 * d * 4;   // the warps' sums
    const int64_t want = (T + s.rows - 1) / s.rows;
    s.grid = static_cast<int>(want < static_cast<int64_t>(s.occ) * sms ? want : s.occ * sms);
    return s;
}

template <bool F32, bool WARP, int CH, int NT, int OF, int OB>
int launch_norm(const NormParams& p, const Shape& s, bool bwd, cudaStream_t st) {
    const auto f = norm_fwd_kernel<F32, WARP, CH, NT, OF>;
    const auto b = norm_bwd_kernel<F32, WARP, CH, NT, OB>;
    if (ensure_smem_attr(bwd ? reinterpret_cast<const void*>(b) : reinterpret_cast<const void*>(f),
                         s.smem))
        return MOE_ECUDA;
    if (bwd)
        b<<<s.grid, s.threads, s.smem, st>>>(p);
    else
        f<<<s.grid, s.threads, s.smem, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, bwd ? "norm_residual_bwd" : "norm_residual");
    return MOE_OK;
}

template <bool F32>
int launch_width(const NormParams& p, const Shape& s, bool bwd, cudaStream_t st) {
    if (p.chunks <= 32) return launch_norm<F32, true, 1, 256, 4, 2>(p, s, bwd, st);
    if (p.chunks <= 64) return launch_norm<F32, true, 2, 256, 4, 2>(p, s, bwd, st);
    if (p.chunks <= 128) return launch_norm<F32, true, 4, 256, 2, 1>(p, s, bwd, st);
    if (p.chunks <= 256) return launch_norm<F32, false, 1, 256, 4, 2>(p, s, bwd, st);
    if (p.chunks <= 512) return launch_norm<F32, false, 1, 512, 2, 1>(p, s, bwd, st);
    if (p.chunks <= 768) return launch_norm<F32, false, 1, 768, 1, 1>(p, s, bwd, st);
    return launch_norm<F32, false, 1, 1024, 1, 1>(p, s, bwd, st);
}

NormParams norm_params(const moe_norm_t& c, const uint16_t* b, const void* r, const uint16_t* gate,
                       const uint16_t* w_post, const uint16_t* w_pre) {
    NormParams p;
    memset(&p, 0, sizeof(p));
    p.T = c.T;
    p.d = c.d;
    p.chunks = c.d / 8;
    p.alpha = c.alpha;
    p.beta = c.beta;
    p.eps = c.eps;
    p.inv_d = 1.0f / static_cast<float>(c.d);
    p.b = b;
    p.r = r;
    p.gate = gate;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.gate_mode = gate ? (c.gate_per_token ? 2 : 1) : 0;
    return p;
}

}  // namespace

int launch_norm_residual(const moe_norm_t& c, const uint16_t* b, const void* r,
                         const uint16_t* gate, const uint16_t* w_post, const uint16_t* w_pre,
                         void* y, uint16_t* n, float* rstd_post, float* rstd_pre,
                         cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    NormParams p = norm_params(c, b, r, gate, w_post, w_pre);
    p.y = y;
    p.n = n;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.slots = 1 + (p.gate_mode == 2) + (c.res_f32 ? 2 : 1);
    const Shape s = norm_shape(c.T, c.d, p.slots, sms, false);
    p.stages = s.stages;
    return c.res_f32 ? launch_width<true>(p, s, false, st) : launch_width<false>(p, s, false, st);
}

// Partial rows for the most CTAs of any device this runs on, two an SM.
constexpr int64_t kMaxPartRows = 2 * 160;

int64_t norm_backward_ws(int64_t T, int d) {
    return (T < kMaxPartRows ? T : kMaxPartRows) * 3 * d * 4;
}

int launch_norm_residual_backward(const moe_norm_t& c, const uint16_t* dn, const void* dy,
                                  const uint16_t* b, const void* r, const uint16_t* gate,
                                  const uint16_t* w_post, const uint16_t* w_pre,
                                  const float* rstd_post, const float* rstd_pre, uint16_t* db,
                                  void* dr, void* dgate, float* dw_post, float* dw_pre, void* ws,
                                  cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    NormParams p = norm_params(c, b, r, gate, w_post, w_pre);
    p.dn = dn;
    p.dy = dy;
    p.db = db;
    p.dr = dr;
    p.dgate = dgate;
    p.in_post = rstd_post;
    p.in_pre = rstd_pre;
    p.part = static_cast<float*>(ws);
    p.slots = 2 + (p.gate_mode == 2) + (c.res_f32 ? 4 : 2);
    const Shape s = norm_shape(c.T, c.d, p.slots, sms < 160 ? sms : 160, true);
    p.stages = s.stages;
    const int rc = c.res_f32 ? launch_width<true>(p, s, true, st)
                             : launch_width<false>(p, s, true, st);
    if (rc != MOE_OK) return rc;
    norm_sums_kernel<<<(3 * c.d + 31) / 32, 256, 0, st>>>(
        p.part, s.grid, c.d, dw_post, dw_pre,
        p.gate_mode == 1 ? static_cast<float*>(dgate) : nullptr);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "norm_sums");
    return MOE_OK;
}

}  // namespace moe
