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
//   d <= 256: a warp a row, 8 rows a CTA.  d > 256: a CTA a row, d / 8
//   threads, several CTAs an SM while their registers allow.
// The backward's sums over tokens (dw_post, dw_pre, dgate) stay in registers
// over all of a CTA's rows; each CTA writes one partial row and a second
// kernel adds the partials in their order: no atomics.
//   16384 rows of 6144 in bf16: forward 121 us (6.65 TB/s; a copy reaches 6.78),
// backward 182 us (6.64 TB/s).  8191 rows of 2048, fp32 stream and a gate a
// token, backward: 67 us (5.5 TB/s; 5 us of them are the sums over tokens).
// One row of 2048: 2.4 us on the device.  Forward of 16384 rows, bf16 with a gate a
// channel, and fp32 rows with a gate a token: 256 channels 9.4 and 9.8 us, 1024 28
// and 44, 2048 48 and 87, 4096 89 and 165, 6144 120 and 245, 8192 182 and 282.
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

struct NormParams {
    int64_t T;
    int d, chunks;            // chunks = d / 8
    int stages;               // ring depth
    bool wide;                // fp32 output on a 32-byte boundary
    float alpha, beta, eps, inv_d;
    const uint16_t *b, *gate, *w_post, *w_pre, *dn;
    const void *r, *dy;
    int gate_mode;            // 0 none, 1 [d], 2 [T, d]
    void *y, *dr, *dgate;
    uint16_t *n, *db;
    float *rstd_post, *rstd_pre;          // forward: out
    const float *in_post, *in_pre;        // backward: in
    float* part;                           // [CTAs, 2, d]
    int64_t part_rows;                     // that the scratch has
};

// Eight channels as four pairs.
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
    f[0] = bf16x2_f32(v.x);
    f[1] = bf16x2_f32(v.y);
    f[2] = bf16x2_f32(v.z);
    f[3] = bf16x2_f32(v.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                      pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}

__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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

// A residual-stream chunk: one slot of bf16, or two of fp32.  Of fp32 a thread
// copies 16 bytes 512 apart of its warp's 1 KB instead of its own 32, so that
// a warp's copy is whole lines; it reads its own 8 values behind a __syncwarp.
// `slot` is this thread's place in the first slot, `pitch` the slots' distance.
template <bool F32>
__device__ __forceinline__ void load_res(const uint4* slot, int pitch, float2 (&f)[4]) {
    if (F32) {
        const int wl = threadIdx.x & 31;
        const uint4* q = slot - wl + (wl >> 4) * pitch + ((2 * wl) & 31);
        const uint4 a = q[0], b = q[1];
        f[0] = as_float2(a.x, a.y);
        f[1] = as_float2(a.z, a.w);
        f[2] = as_float2(b.x, b.y);
        f[3] = as_float2(b.z, b.w);
    } else {
        unpack8(slot[0], f);
    }
}

// An fp32 chunk is a whole 32-byte sector: written by one instruction where
// the tensor starts on such a boundary (wide), or L2 sees two halves.
template <bool F32>
__device__ __forceinline__ void store_res(void* base, int64_t at, const float2 (&f)[4], bool wide) {
    if (F32) {
        float* o = static_cast<float*>(base) + at;
        if (wide) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o),
                         "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x),
                         "f"(f[2].y), "f"(f[3].x), "f"(f[3].y)
                         : "memory");
        } else {
            reinterpret_cast<float4*>(o)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            reinterpret_cast<float4*>(o)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        }
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(f);
    }
}

// at: the row's start; col: this thread's first channel.
template <bool F32>
__device__ __forceinline__ void copy_res(uint32_t dst, uint32_t pitch, const void* base, int64_t at,
                                         int col, int d) {
    if (F32) {
        const int wl = threadIdx.x & 31, e = col - 4 * wl;   // of the warp's first channel: + 4 wl
        const float* s = static_cast<const float*>(base) + at + e;
        if (e < d) cp_async_16(dst, s, 16);
        if (e + 128 < d) cp_async_16(dst + pitch, s + 128, 16);
    } else if (col < d) {
        cp_async_16(dst, static_cast<const uint16_t*>(base) + at + col, 16);
    }
}

// beta w_post (with a gate that all tokens share: times the gate) of 8 channels.
__device__ __forceinline__ void load_factor(const NormParams& p, bool with_gate, int c,
                                            float2 (&G)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) G[e] = both(0.f);
    if (!p.w_post || c >= p.chunks) return;
    float2 g[4];
    unpack8(*reinterpret_cast<const uint4*>(p.w_post + c * 8), G);
#pragma unroll
    for (int e = 0; e < 4; ++e) G[e] = mul2(G[e], both(p.beta));
    if (!with_gate || p.gate_mode != 1) return;
    unpack8(*reinterpret_cast<const uint4*>(p.gate + c * 8), g);
#pragma unroll
    for (int e = 0; e < 4; ++e) G[e] = mul2(G[e], g[e]);
}

// ------------------------------------------------------------------ forward

// Slots of a thread and chunk: b, gate (TOKEN), r (1 or 2).  TOKEN: a gate
// value for each token and channel; otherwise beta, the gate and w_post are
// one factor a channel, held in fp32 over all rows.
template <bool F32, bool TOKEN, bool WARP, int NT, int OCC>
__global__ void __launch_bounds__(NT, OCC) norm_fwd_kernel(const NormParams p) {
    extern __shared__ uint4 ring[];
    __shared__ float red[4][32];
    constexpr int SLOTS = 1 + TOKEN + (F32 ? 2 : 1);
    const int nt = blockDim.x;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int rows = WARP ? nt / 32 : 1;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const int col = lane * 8;               // this thread's channels
    const bool in = lane < p.chunks;
    const bool has_b = p.b != nullptr, has_n = p.n != nullptr;
    const auto slot = [&](int stage, int k) {
        return (stage * SLOTS + k) * nt + static_cast<int>(threadIdx.x);
    };
    const auto fetch = [&](int64_t row, int stage) {
        if (row < p.T) {
            const int64_t at = row * p.d;
            if (in && has_b) cp_async_16(smem_u32(ring + slot(stage, 0)), p.b + at + col, 16);
            if (in && TOKEN) cp_async_16(smem_u32(ring + slot(stage, 1)), p.gate + at + col, 16);
            copy_res<F32>(smem_u32(ring + slot(stage, 1 + TOKEN)), nt * 16, p.r, at, col, p.d);
        }
        cp_async_commit();
    };
    for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);

    float2 G[4];
    load_factor(p, !TOKEN, lane, G);
    uint4 wp = make_uint4(0, 0, 0, 0);
    if (in && has_n) wp = *reinterpret_cast<const uint4*>(p.w_pre + col);
    int stage = 0, par = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        wait_stage(p.stages);
        if (F32) __syncwarp();   // the other lanes' copies too
        float2 b[4], y[4], ss = both(0.f);
        float2 g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = y[e] = g[e] = both(0.f);
        if (in) {
            if (has_b) unpack8(ring[slot(stage, 0)], b);
            if (TOKEN) unpack8(ring[slot(stage, 1)], g);
            load_res<F32>(ring + slot(stage, 1 + TOKEN), nt, y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ss = fma2(b[e], b[e], ss);
            y[e] = mul2(y[e], both(p.alpha));
            if (TOKEN) b[e] = mul2(b[e], g[e]);
        }
        if (F32) __syncwarp();
        fetch(row + p.stages * step, stage);   // this thread (fp32: its warp) has read the slots
        if (++stage == p.stages) stage = 0;
        if (has_b) {
            const float rb = rsqrtf(row_sum<WARP>(ss.x + ss.y, red[par]) * p.inv_d + p.eps);
            if (lane == 0 && p.rstd_post) p.rstd_post[row] = rb;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = fma2(G[e], mul2(b[e], both(rb)), y[e]);
        }
        if (p.y && in)
            store_res<F32>(p.y, row * p.d + col, y, p.wide);
        if (has_n) {
            ss = both(0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fma2(y[e], y[e], ss);
            const float ry = rsqrtf(row_sum<WARP>(ss.x + ss.y, red[2 + par]) * p.inv_d + p.eps);
            if (lane == 0 && p.rstd_pre) p.rstd_pre[row] = ry;
            float2 w[4];
            unpack8(wp, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = mul2(w[e], mul2(y[e], both(ry)));
            if (in)
                *reinterpret_cast<uint4*>(p.n + row * p.d + col) = pack8(w);
        }
        par ^= 1;
    }
}

// ------------------------------------------------------------------ backward

// Slots of a thread and chunk: b, dn, gate (TOKEN), r, dy (1 or 2 each).
// Two sums over the tokens: dw_pre = sum dn q, and S = sum p du (TOKEN: sum
// g p du), from which dw_post = beta g S and dgate = beta w_post S follow a
// channel at the end, for a gate that all tokens share.
template <bool F32, bool TOKEN, bool WARP, int CH, int NT, int OCC>
__global__ void __launch_bounds__(NT, OCC) norm_bwd_kernel(const NormParams p) {
    extern __shared__ uint4 ring[];
    __shared__ float red[4][32];
    constexpr int R = F32 ? 2 : 1, SLOTS = 2 + TOKEN + 2 * R;
    constexpr int s_dn = 1, s_gate = 2, s_r = 2 + TOKEN, s_dy = s_r + R;
    const int nt = blockDim.x;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int rows = WARP ? nt / 32 : 1;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const bool has_b = p.b != nullptr, has_n = p.dn != nullptr, has_y = p.dy != nullptr;
    // this thread's chunks are lane + nt i
    const auto in = [&](int i) { return lane + nt * i < p.chunks; };
    const auto slot = [&](int stage, int i, int k) {
        return ((stage * CH + i) * SLOTS + k) * nt + static_cast<int>(threadIdx.x);
    };
    const auto fetch = [&](int64_t row, int stage) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (row < p.T) {
                const int col = (lane + nt * i) * 8;
                const int64_t at = row * p.d;
                if (in(i)) {
                    if (has_b) cp_async_16(smem_u32(ring + slot(stage, i, 0)), p.b + at + col, 16);
                    if (has_n)
                        cp_async_16(smem_u32(ring + slot(stage, i, s_dn)), p.dn + at + col, 16);
                    if (TOKEN)
                        cp_async_16(smem_u32(ring + slot(stage, i, s_gate)), p.gate + at + col, 16);
                }
                if (has_n)
                    copy_res<F32>(smem_u32(ring + slot(stage, i, s_r)), nt * 16, p.r, at, col, p.d);
                if (has_y)
                    copy_res<F32>(smem_u32(ring + slot(stage, i, s_dy)), nt * 16, p.dy, at, col, p.d);
            }
        cp_async_commit();
    };
    // slots that no copy fills (absent tensors, channels past d) read as zero
    for (int s = 0; s < p.stages * CH * SLOTS; ++s) ring[slot(0, 0, s)] = make_uint4(0, 0, 0, 0);
    for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);

    float2 G[CH][4], S[CH][4], a_pre[CH][4];
    uint4 wp[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        load_factor(p, !TOKEN, lane + nt * i, G[i]);
        wp[i] = make_uint4(0, 0, 0, 0);
        if (in(i) && has_n)
            wp[i] = *reinterpret_cast<const uint4*>(p.w_pre + (lane + nt * i) * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][e] = a_pre[i][e] = both(0.f);
    }
    // a row ahead of its use; volatile, or the load sinks to the use and every
    // row waits for it
    const auto stat = [&](const float* s, int64_t row) {
        float v = 0.f;
        if (s && row < p.T) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(s + row));
        return v;
    };
    float rb = stat(p.in_post, row0), ry = stat(p.in_pre, row0);
    int stage = 0, par = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        const float rb_next = stat(p.in_post, row + step), ry_next = stat(p.in_pre, row + step);
        wait_stage(p.stages);
        if (F32) __syncwarp();   // the other lanes' copies too
        // pv: p; du: first dy, then dL/dy, then dL/dp; gt: the token's gate
        float2 pv[CH][4], q[CH][4], t[CH][4], du[CH][4], s1 = both(0.f);
        uint4 gt[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float2 g[4], w[4];
            unpack8(ring[slot(stage, i, 0)], pv[i]);
            unpack8(ring[slot(stage, i, s_dn)], t[i]);
            load_res<F32>(ring + slot(stage, i, s_r), nt, q[i]);
            load_res<F32>(ring + slot(stage, i, s_dy), nt, du[i]);
            if (TOKEN) {
                gt[i] = ring[slot(stage, i, s_gate)];
                unpack8(gt[i], g);
            }
            unpack8(wp[i], w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pv[i][e] = mul2(pv[i][e], both(rb));
                float2 m = mul2(pv[i][e], G[i][e]);
                if (TOKEN) m = mul2(m, g[e]);
                q[i][e] = mul2(fma2(q[i][e], both(p.alpha), m), both(ry));
                a_pre[i][e] = fma2(t[i][e], q[i][e], a_pre[i][e]);
                t[i][e] = mul2(t[i][e], w[e]);
                s1 = fma2(t[i][e], q[i][e], s1);
            }
        }
        if (F32) __syncwarp();
        fetch(row + p.stages * step, stage);   // this thread (fp32: its warp) has read the slots
        if (++stage == p.stages) stage = 0;
        const float k1 = has_n ? row_sum<WARP>(s1.x + s1.y, red[par]) * p.inv_d : 0.f;
        float2 s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float2 o[4], g[4];
            const int64_t at = row * p.d + (lane + nt * i) * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                du[i][e] = fma2(both(ry), fma2(q[i][e], both(-k1), t[i][e]), du[i][e]);
                o[e] = mul2(du[i][e], both(p.alpha));
            }
            if (in(i)) store_res<F32>(p.dr, at, o, p.wide);
            if (TOKEN) unpack8(gt[i], g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 pd = mul2(pv[i][e], du[i][e]);
                du[i][e] = mul2(du[i][e], G[i][e]);
                if (TOKEN) {
                    o[e] = mul2(pd, G[i][e]);
                    S[i][e] = fma2(pd, g[e], S[i][e]);
                    du[i][e] = mul2(du[i][e], g[e]);
                } else {
                    S[i][e] = add2(S[i][e], pd);
                }
                s2 = fma2(du[i][e], pv[i][e], s2);
            }
            if (TOKEN && in(i))
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dgate) + at) = pack8(o);
        }
        if (has_b) {
            const float k2 = row_sum<WARP>(s2.x + s2.y, red[2 + par]) * p.inv_d;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float2 o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = mul2(both(rb), fma2(pv[i][e], both(-k2), du[i][e]));
                if (in(i))
                    *reinterpret_cast<uint4*>(p.db + row * p.d + (lane + nt * i) * 8) = pack8(o);
            }
        }
        par ^= 1;
        rb = rb_next;
        ry = ry_next;
    }
    // this CTA's partial sums over its tokens: S, then dw_pre
    if (!moe_check(blockIdx.x < p.part_rows, 1211)) return;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
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
                if (!in(i)) continue;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2(&v)[4] = k ? a_pre[i] : S[i];
                    const int at = k * p.d + (lane + nt * i) * 8;
                    float4* to = reinterpret_cast<float4*>((w + 1 < turns ? acc : part) + at);
                    const float4* was = reinterpret_cast<const float4*>(acc + at);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float4 x = make_float4(v[2 * e].x, v[2 * e].y, v[2 * e + 1].x,
                                               v[2 * e + 1].y);
                        if (w) {
                            const float4 y = was[e];
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        to[e] = x;
                    }
                }
            }
        }
        if (WARP) __syncthreads();
    }
}

// The sums over the partial rows in a fixed order (32 columns a CTA, 32
// threads a column over a part of the rows each, so that all loads of a thread
// are under way at once), and what follows from S.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const NormParams p, int n, float* dw_post,
                                                         float* dw_pre, float* dgate) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + x;
    const bool in = col < 2ll * p.d;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are complete
    float v = 0.f;
    if (in)
#pragma unroll 8
        for (int i = g; i < n; i += 32) v += p.part[static_cast<int64_t>(i) * 2 * p.d + col];
    s[g][x] = v;
    __syncthreads();
    v = sum32(s[x][g]);   // column g of the CTA, its 32 parts in the warp's lanes
    __syncthreads();
    if (x == 0) s[0][g] = v;
    __syncthreads();
    if (g == 0 && in) {
        v = s[0][x];
        if (col >= p.d) {
            if (dw_pre) dw_pre[col - p.d] = v;
            return;
        }
        v *= p.beta;
        const auto bf = [](const uint16_t* t, int64_t i) {
            return __uint_as_float(static_cast<uint32_t>(t[i]) << 16);
        };
        if (dw_post) dw_post[col] = p.gate_mode == 1 ? v * bf(p.gate, col) : v;
        if (dgate) dgate[col] = v * bf(p.w_post, col);
    }
}

// The launch shape for a width: threads and rows of a CTA, chunks of a
// thread, CTAs an SM (as many as the kernels' registers allow).  A warp a row
// up to 256 channels: 16384 rows of 256 take 11.3 us forward and 14.7 backward,
// a CTA of one warp a row 12.8 and 16.4.
struct Shape {
    int threads, rows, per_thread, occ, grid, stages, smem;
};

constexpr int fwd_occ(int threads) {
    return threads <= 64 ? 16 : threads <= 128 ? 8 : threads <= 256 ? 4 : threads <= 512 ? 2 : 1;
}
// Backward: 8 channels a thread up to 1024 channels, 16 past them, up to 168
// registers.  16384 rows of 1024: 41.7 us (8) and 47.4 (16), with fp32 rows and
// a gate a token 61 and 80; 8191 rows of 2048 64.6 either way.  CTAs of 256 and 512
// threads (2056 to 4096 and 6152 to 8192 channels) have 128 registers a thread and
// spill 20 to 140 bytes: 16384 rows of 4096 and 8192 take 155 and 314 us (1.3 times
// their bytes), with fp32 rows and a gate a token 399 and 604 (1.8 and 1.4), where
// 6144, without spills, takes 182 (1.02) and 383 (1.17).
constexpr int bwd_occ(int threads) {
    return threads <= 64 ? 8 : threads <= 128 ? 3 : threads <= 256 ? 2 : 1;
}

// ring budget of an SM; a CTA's share keeps room for its 512 bytes of sums
constexpr int kRingBytes = 212 * 1024;

Shape norm_shape(int64_t T, int d, int slots, int sms, bool bwd) {
    Shape s;
    const int chunks = d / 8;
    s.rows = chunks <= 32 ? 8 : 1;
    s.per_thread = bwd && chunks > 128 ? 2 : 1;
    s.threads = chunks <= 32 ? 256 : ((chunks + s.per_thread - 1) / s.per_thread + 31) / 32 * 32;
    s.occ = bwd ? bwd_occ(s.threads) : fwd_occ(s.threads);
    const int stage_bytes = s.threads * s.per_thread * slots * 16;
    while (s.occ > 1 && kRingBytes / s.occ / stage_bytes < 2) --s.occ;
    s.stages = kRingBytes / s.occ / stage_bytes;
    s.stages = s.stages > 4 ? 4 : s.stages < 2 ? 2 : s.stages;
    s.smem = s.stages * stage_bytes;
    const int64_t want = (T + s.rows - 1) / s.rows;
    s.grid = static_cast<int>(want < static_cast<int64_t>(s.occ) * sms ? want : s.occ * sms);
    return s;
}

template <class K>
int launch_kernel(K kern, const NormParams& p, const Shape& s, const char* name, cudaStream_t st) {
    if (ensure_smem_attr(reinterpret_cast<const void*>(kern), s.smem)) return MOE_ECUDA;
    kern<<<s.grid, s.threads, s.smem, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, name);
    return MOE_OK;
}

template <bool F32, bool TOKEN, bool WARP, int NT>
int launch_fwd(const NormParams& p, const Shape& s, cudaStream_t st) {
    return launch_kernel(norm_fwd_kernel<F32, TOKEN, WARP, NT, fwd_occ(NT)>, p, s,
                         "norm_residual", st);
}

template <bool F32, bool TOKEN, bool WARP, int CH, int NT>
int launch_bwd(const NormParams& p, const Shape& s, cudaStream_t st) {
    return launch_kernel(norm_bwd_kernel<F32, TOKEN, WARP, CH, NT, bwd_occ(NT)>, p, s,
                         "norm_residual_bwd", st);
}

template <bool F32, bool TOKEN>
int launch_width(const NormParams& p, const Shape& s, bool bwd, cudaStream_t st) {
    if (bwd) {
        if (s.rows > 1) return launch_bwd<F32, TOKEN, true, 1, 256>(p, s, st);
        if (s.per_thread == 1)
            return s.threads <= 64 ? launch_bwd<F32, TOKEN, false, 1, 64>(p, s, st)
                                   : launch_bwd<F32, TOKEN, false, 1, 128>(p, s, st);
        if (s.threads <= 128) return launch_bwd<F32, TOKEN, false, 2, 128>(p, s, st);
        if (s.threads <= 256) return launch_bwd<F32, TOKEN, false, 2, 256>(p, s, st);
        if (s.threads <= 384) return launch_bwd<F32, TOKEN, false, 2, 384>(p, s, st);
        return launch_bwd<F32, TOKEN, false, 2, 512>(p, s, st);
    }
    if (s.rows > 1) return launch_fwd<F32, TOKEN, true, 256>(p, s, st);
    if (s.threads <= 64) return launch_fwd<F32, TOKEN, false, 64>(p, s, st);
    if (s.threads <= 128) return launch_fwd<F32, TOKEN, false, 128>(p, s, st);
    if (s.threads <= 256) return launch_fwd<F32, TOKEN, false, 256>(p, s, st);
    if (s.threads <= 512) return launch_fwd<F32, TOKEN, false, 512>(p, s, st);
    if (s.threads <= 768) return launch_fwd<F32, TOKEN, false, 768>(p, s, st);
    return launch_fwd<F32, TOKEN, false, 1024>(p, s, st);
}

int launch_any(const NormParams& p, const Shape& s, bool f32, bool bwd, cudaStream_t st) {
    const bool token = p.gate_mode == 2;
    if (f32) return token ? launch_width<true, true>(p, s, bwd, st) : launch_width<true, false>(p, s, bwd, st);
    return token ? launch_width<false, true>(p, s, bwd, st) : launch_width<false, false>(p, s, bwd, st);
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

int check_status_norm() { return moe_check_read_reset(); }

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
    const int slots = 1 + (p.gate_mode == 2) + (c.res_f32 ? 2 : 1);
    const Shape s = norm_shape(c.T, c.d, slots, sms, false);
    p.stages = s.stages;
    p.wide = (reinterpret_cast<uintptr_t>(y) & 31) == 0;
    return launch_any(p, s, c.res_f32, false, st);
}

// Partial rows: the most CTAs of a launch, on a device of 160 SMs at most.
constexpr int64_t kMaxPartRows = bwd_occ(64) * 160;

int64_t norm_backward_ws(int64_t T, int d) {
    return (T < kMaxPartRows ? T : kMaxPartRows) * 2 * d * 4;
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
    p.part_rows = norm_backward_ws(c.T, c.d) / (8 * c.d);
    const int slots = 2 + (p.gate_mode == 2) + (c.res_f32 ? 4 : 2);
    const Shape s = norm_shape(c.T, c.d, slots, sms < 160 ? sms : 160, true);
    p.stages = s.stages;
    p.wide = (reinterpret_cast<uintptr_t>(dr) & 31) == 0;
    if (const int rc = launch_any(p, s, c.res_f32, true, st)) return rc;
    // launched while the rows are still being worked on; it waits for them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((2 * c.d + 31) / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, norm_sums_kernel, p, s.grid, dw_post, dw_pre,
                           p.gate_mode == 1 ? static_cast<float*>(dgate) : nullptr) != cudaSuccess)
        return MOE_ECUDA;
    trace_after(st, "norm_sums");
    return MOE_OK;
}

}  // namespace moe
