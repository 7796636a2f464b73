// attention_bwd.cu -- gradients of the causal packed attention.
//
//   P_ij = 2^(c s_ij - lse_i log2 e)      D_i = dO_i . O_i
//   dV_j = sum_i P_ij dO_i                dS_ij = P_ij (dO_i . V_j - D_i)
//   dK_j = scale sum_i dS_ij Q_i          dQ_i = scale sum_j dS_ij K_j
//
// Three kernels.  The first forms D (from O in two bf16 parts) and the scaled
// lse.  The second gives one CTA 128 query rows and walks their key blocks
// for dQ.  The third gives one CTA 128 keys of one key/value head and walks
// the query blocks of all the group's heads, so dK and dV are summed in TMEM
// and written once: no atomics, the same bits every time.  Both compute P and
// dP again (seven products of 128 x 128 x D a block pair where five are
// needed): the price of a fixed order without a pass over memory for dQ.
// Warps 0-7 form P and dS (a thread holds 64 of the 128 columns of its TMEM
// lane), warp 8 issues the MMAs, warp 9 the TMA loads.  P and dS return to
// the columns of S and dP as bf16 A operands.
#include <cstring>

#include "attention.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    CUtensorMap mapQ, mapK, mapV, mapO;   // mapO: dout; box {64, 128, 1}
    const int4* tiles;
    const int32_t* header;
    int list;
    int units;             // CTAs of one block: heads
    int group, D;
    int64_t T;
    int64_t q_t, q_h, k_t, k_h, v_t, v_h, do_t, do_h;
    const uint16_t *q, *k, *v, *dout;
    int64_t dq_t, dq_h, dk_t, dk_h, dv_t, dv_h;
    uint16_t *dq, *dk, *dv;
    const float* lse2;     // [heads, T]
    float* delta;          // [heads, T]
    float scale, scale_log2;
    int32_t* status;
};

// ------------------------------------------------------------------ D and lse

struct DeltaParams {
    int64_t T;
    int heads, D;
    int64_t o_t, o_h, do_t, do_h;
    const uint16_t *out, *rest, *dout;
    const float* lse;
    float *lse2, *delta;
};

// Eight lanes a row (16 bytes a load), four rows a warp.
__global__ void __launch_bounds__(256) attn_delta_kernel(const DeltaParams p) {
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 8;
    const int part = threadIdx.x & 7;
    const int64_t rows = p.T * p.heads;
    const int64_t t = r / p.heads;
    const int h = static_cast<int>(r - t * p.heads);
    float sum = 0.f;
    if (r < rows) {
        const int64_t o = t * p.o_t + h * p.o_h, g = t * p.do_t + h * p.do_h;
        for (int c = part * 8; c < p.D; c += 64) {
            const uint4 a = *reinterpret_cast<const uint4*>(p.out + o + c);
            const uint4 b = *reinterpret_cast<const uint4*>(p.rest + o + c);
            const uint4 d = *reinterpret_cast<const uint4*>(p.dout + g + c);
            const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w},
                           dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum += bf16_lo(dv[i]) * (bf16_lo(av[i]) + bf16_lo(bv[i]));
                sum += bf16_hi(dv[i]) * (bf16_hi(av[i]) + bf16_hi(bv[i]));
            }
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (r < rows && part == 0) {
        p.delta[h * p.T + t] = sum;
        p.lse2[h * p.T + t] = p.lse[h * p.T + t] * kLog2e;
    }
}

// ------------------------------------------------------------------ rows by the definition

// Rows whose products met a non-finite value, on the CUDA cores: pairs that
// the mask hides are skipped instead of multiplied by 0.  One warp a row.
struct RowPair {
    float p, ds;
};

__device__ __forceinline__ RowPair row_pair(const BwdParams& p, const float (&a)[4],
                                            const float (&b)[4], const uint16_t* x,
                                            const uint16_t* y, float lse2, float delta, int lane) {
    float s = 0.f, dp = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.D) {
            s += a[i] * bf16_f32(x[lane + 32 * i]);
            dp += b[i] * bf16_f32(y[lane + 32 * i]);
        }
    s = warp_sum(s);
    dp = warp_sum(dp);
    RowPair r;
    r.p = exp2f(s * p.scale_log2 - lse2);
    r.ds = r.p * (dp - delta);
    return r;
}

__device__ __noinline__ void dq_row(const BwdParams& p, int64_t start, int row, int h, int kvh) {
    const int lane = threadIdx.x & 31;
    const int64_t t = start + row;
    float q[4], g[4], acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = lane + 32 * i < p.D;
        q[i] = in ? bf16_f32(p.q[t * p.q_t + h * p.q_h + lane + 32 * i]) : 0.f;
        g[i] = in ? bf16_f32(p.dout[t * p.do_t + h * p.do_h + lane + 32 * i]) : 0.f;
    }
    const float lse2 = p.lse2[h * p.T + t], delta = p.delta[h * p.T + t];
    for (int j = 0; j <= row; ++j) {
        const uint16_t* k = p.k + (start + j) * p.k_t + kvh * p.k_h;
        const uint16_t* v = p.v + (start + j) * p.v_t + kvh * p.v_h;
        const RowPair r = row_pair(p, q, g, k, v, lse2, delta, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < p.D) acc[i] += r.ds * bf16_f32(k[lane + 32 * i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.D)
            p.dq[t * p.dq_t + h * p.dq_h + lane + 32 * i] = f32_bf16(acc[i] * p.scale);
}

// which: 0 the row of dV, 1 of dK.
__device__ __noinline__ void dkv_row(const BwdParams& p, int64_t start, int len, int row, int kvh,
                                     int which) {
    const int lane = threadIdx.x & 31;
    const int64_t t = start + row;
    float k[4], v[4], acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = lane + 32 * i < p.D;
        k[i] = in ? bf16_f32(p.k[t * p.k_t + kvh * p.k_h + lane + 32 * i]) : 0.f;
        v[i] = in ? bf16_f32(p.v[t * p.v_t + kvh * p.v_h + lane + 32 * i]) : 0.f;
    }
    for (int h = kvh * p.group; h < (kvh + 1) * p.group; ++h)
        for (int i = row; i < len; ++i) {
            const uint16_t* q = p.q + (start + i) * p.q_t + h * p.q_h;
            const uint16_t* g = p.dout + (start + i) * p.do_t + h * p.do_h;
            const RowPair r = row_pair(p, k, v, q, g, p.lse2[h * p.T + start + i],
                                       p.delta[h * p.T + start + i], lane);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (lane + 32 * e < p.D)
                    acc[e] += which ? r.ds * bf16_f32(q[lane + 32 * e])
                                    : r.p * bf16_f32(g[lane + 32 * e]);
        }
    uint16_t* o = which ? p.dk + t * p.dk_t + kvh * p.dk_h : p.dv + t * p.dv_t + kvh * p.dv_h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.D) o[lane + 32 * i] = f32_bf16(which ? acc[i] * p.scale : acc[i]);
}

__device__ __forceinline__ void zero_rows(uint16_t* base, int64_t st_t, int D, int rows) {
    for (int i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
        *reinterpret_cast<uint4*>(base + (i / (D / 8)) * st_t + i % (D / 8) * 8) =
            make_uint4(0, 0, 0, 0);
}

// Columns [c0, c0 + N) of the warp's 32 accumulator rows, times `f`, as bf16
// to global memory (base: its first row; rows: how many exist); returns
// whether a value of this thread's row was not finite.
template <int N>
__device__ __forceinline__ bool store_rows(uint32_t taddr, int c0, int D, float f, uint16_t* base,
                                           int64_t stride, int rows) {
    float2 sick = make_float2(0.f, 0.f);   // NaN once a value is not finite
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
        uint32_t a[32];
        tmem_ld32(taddr + c0 + 32 * i, a);
        uint4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = mul2(make_float2(__uint_as_float(a[8 * g + 2 * e]),
                                                  __uint_as_float(a[8 * g + 2 * e + 1])),
                                      make_float2(f, f));
                sick = fma2(x, make_float2(0.f, 0.f), sick);
                w[e] = pack_bf16x2(x.x, x.y);
            }
            v[g] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        store_quad(v, base, stride, rows, c0 + 32 * i, D);
    }
    return !(sick.x + sick.y == 0.f);
}

template <int D>
struct BwdCfg {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int SMEM = 2 * TILE + STAGES * TILE + 1024 + 256 + 2048;
};

// Shared-memory layout and barriers of both kernels: two resident tiles, a
// ring of streamed ones.
template <int D>
struct BwdSmem {
    uint8_t *res, *ring;
    float* rows;                    // dK/dV: lse2 and delta of a query block, two buffers
    uint64_t *full, *empty, *res_full, *s_full, *dp_full, *p_full, *ds_full, *acc_full, *done;
    uint32_t* tmem_slot;
    volatile int* abort_flag;
    __device__ explicit BwdSmem(uint8_t* raw_ptr) {
        using C = BwdCfg<D>;
        const uint32_t raw = smem_u32(raw_ptr);
        res = raw_ptr + (((raw + 1023u) & ~1023u) - raw);
        ring = res + 2 * C::TILE;
        rows = reinterpret_cast<float*>(ring + C::STAGES * C::TILE);
        full = reinterpret_cast<uint64_t*>(rows + 512);
        empty = full + C::STAGES;
        res_full = empty + C::STAGES;
        s_full = res_full + 1;
        dp_full = s_full + 1;
        p_full = dp_full + 1;
        ds_full = p_full + 1;
        acc_full = ds_full + 1;
        done = acc_full + 1;
        tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
        abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    }
    __device__ void init() {
        for (int s = 0; s < BwdCfg<D>::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(res_full, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, 256);
        mbar_init(ds_full, 256);
        mbar_init(acc_full, 1);
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
};

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                          int token, int head) {
    for (int b = 0; b < D / 64; ++b)
        tma_load_3d(dst + b * kBoxBytes, map, bar, b * 64, token, head);
}

// ------------------------------------------------------------------ dK, dV

template <int D>
__global__ void __launch_bounds__(384, 1) attn_dkv_kernel(const __grid_constant__ BwdParams p) {
    using C = BwdCfg<D>;
    const int tile = blockIdx.x / p.units;
    if (tile >= p.header[p.list]) return;
    const int kvh = blockIdx.x - tile * p.units;
    const int4 te = p.tiles[tile];
    const int64_t start = te.x;
    const int len = te.y;
    if (te.z < 0) {   // tokens of no sequence
        zero_rows(p.dk + start * p.dk_t + kvh * p.dk_h, p.dk_t, p.D, len);
        zero_rows(p.dv + start * p.dv_t + kvh * p.dv_h, p.dv_t, p.D, len);
        return;
    }
    const int nb = te.z, nblk = (len + 127) / 128;
    const int per_head = nblk - nb;          // query blocks of one head
    const int n = p.group * per_head;

    extern __shared__ uint8_t smem_raw[];
    BwdSmem<D> sm(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sm.init();
    if (warp == 8) {
        tmem_alloc(sm.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *sm.tmem_slot;
    const uint32_t tmS = tm, tmP = tm + 128, tmV = tm + 256, tmK = tm + 384;

    if (warp >= 8) {
        setmaxnreg_dec<88>();
        if (warp == 9 && lane == 0) {
            // -------------------------------------------------------- loads
            const uint32_t ar = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const int tok = static_cast<int>(start);
            mbar_arrive_expect_tx(sm.res_full, 2 * C::TILE);
            load_tile<D>(ar, &p.mapK, sm.res_full, tok + nb * 128, kvh);
            load_tile<D>(ar + C::TILE, &p.mapV, sm.res_full, tok + nb * 128, kvh);
            uint32_t st = 0, ph = 0, armed = 0, par = 0;
            bool ok = true;
            int h = kvh * p.group, i = nb;
            for (int it = 0; it < 2 * n; ++it) {
                if (!mbar_wait(&sm.empty[st], ph ^ 1u, sm.abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&sm.full[st], C::TILE);
                armed |= 1u << st;
                par = (par & ~(1u << st)) | (ph << st);
                load_tile<D>(ag + st * C::TILE, (it & 1) ? &p.mapO : &p.mapQ, &sm.full[st],
                             tok + i * 128, h);
                if ((it & 1) && ++i == nblk) {
                    i = nb;
                    ++h;
                }
                if (++st == C::STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok || *sm.abort_flag) {   // let the armed copies land before leaving
                volatile int no_abort = 0;
                mbar_wait(sm.res_full, 0, &no_abort, nullptr, 20000000ull);
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait(&sm.full[s], (par >> s) & 1u, &no_abort, nullptr, 20000000ull);
            }
        } else if (warp == 8) {
            // -------------------------------------------------------- MMAs
            const uint32_t one = elect_lane();
            const uint32_t aK = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const uint64_t dK = desc_k(aK), dV = desc_k(aK + C::TILE);
            const auto stage = [](int it) { return static_cast<uint32_t>(it % C::STAGES); };
            const auto phase = [](int it) { return static_cast<uint32_t>(it / C::STAGES) & 1u; };
            const auto at = [&](int it) { return ag + stage(it) * C::TILE; };
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = warp_wait(bar, parity, sm.abort_flag, p.status);
                tc_fence_after();
                return got;
            };
            bool ok = wait(sm.res_full, 0) && wait(&sm.full[0], 0);
            if (ok) {
                mma_scores<D>(one, tmS, dK, desc_k(at(0)));
                commit(one, sm.s_full);
                ok = wait(&sm.full[1], 0);
            }
            if (ok) {
                mma_scores<D>(one, tmP, dV, desc_k(at(1)));
                commit(one, sm.dp_full);
            }
            for (int it = 0; ok && it < n; ++it) {
                const int iq = 2 * it, io = iq + 1;
                if (!(ok = wait(sm.p_full, it & 1u))) break;
                mma_tokens<D>(one, tmV, tmS, desc_mn(at(io)), 0, it > 0);
                mma_tokens<D>(one, tmV, tmS + 64, desc_mn(at(io)), 1, true);
                commit(one, &sm.empty[stage(io)]);
                if (it + 1 < n) {
                    if (!(ok = wait(&sm.full[stage(iq + 2)], phase(iq + 2)))) break;
                    // runs after the product above has read P from these columns
                    mma_scores<D>(one, tmS, dK, desc_k(at(iq + 2)));
                    commit(one, sm.s_full);
                }
                if (!(ok = wait(sm.ds_full, it & 1u))) break;
                mma_tokens<D>(one, tmK, tmP, desc_mn(at(iq)), 0, it > 0);
                mma_tokens<D>(one, tmK, tmP + 64, desc_mn(at(iq)), 1, true);
                commit(one, &sm.empty[stage(iq)]);
                if (it + 1 < n) {
                    if (!(ok = wait(&sm.full[stage(io + 2)], phase(io + 2)))) break;
                    mma_scores<D>(one, tmP, dV, desc_k(at(io + 2)));
                    commit(one, sm.dp_full);
                }
            }
            if (ok) commit(one, sm.acc_full);
            commit(one, sm.done);
            volatile int no_abort = 0;
            mbar_wait(sm.done, 0, &no_abort, p.status);
        }
    } else {
        setmaxnreg_inc<208>();
        // ------------------------------------------------------------ P and dS
        // a thread: key row r, query columns [64 half, 64 half + 64)
        const int half = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmS + lane_off + 64 * half, tp = tmP + lane_off + 64 * half;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        // this thread's share of the query rows' scalars: lse2 or delta of row r
        const float* src = half ? static_cast<const float*>(p.delta) : p.lse2;
        const auto fetch = [&](int it) {
            const int g = it / per_head, i = (nb + it - g * per_head) * 128 + r;
            return i < len ? src[(kvh * p.group + g) * p.T + start + i] : 0.f;
        };
        float next = fetch(0);
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            float* rows = sm.rows + (it & 1) * 256;
            rows[half * 128 + r] = next;
            named_bar_sync(1, 256);
            if (!ok) continue;   // given up: only meets the others at the barrier
            if (it + 1 < n) next = fetch(it + 1);
            const int qb = nb + it % per_head;
            const int limit = min(128, len - qb * 128);   // query rows in this block
            const bool masked = qb == nb || limit < 128;
            const int lo = qb == nb ? r : 0;               // columns lo .. limit-1 count

            if (!warp_wait(sm.s_full, it & 1u, sm.abort_flag, p.status)) {
                ok = false;
                continue;
            }
            tc_fence_after();
            float x[64];
            tmem_ld32_async(ts, reinterpret_cast<uint32_t*>(x));
            tmem_ld32_async(ts + 32, reinterpret_cast<uint32_t*>(x) + 32);
            tmem_wait_ld();
            uint32_t pk[32];
            const float4* l4 = reinterpret_cast<const float4*>(rows + 64 * half);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 l = l4[i];
                const float2 a = fma2(make_float2(x[4 * i], x[4 * i + 1]), c2,
                                      make_float2(-l.x, -l.y));
                const float2 b = fma2(make_float2(x[4 * i + 2], x[4 * i + 3]), c2,
                                      make_float2(-l.z, -l.w));
                x[4 * i] = exp2_fast(a.x);
                x[4 * i + 1] = exp2_fast(a.y);
                x[4 * i + 2] = exp2_fast(b.x);
                x[4 * i + 3] = exp2_fast(b.y);
            }
            if (masked) {
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const int col = 64 * half + i;
                    if (col < lo || col >= limit) x[i] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st32(ts, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(sm.p_full);

            if (!warp_wait(sm.dp_full, it & 1u, sm.abort_flag, p.status)) {
                ok = false;
                continue;
            }
            tc_fence_after();
            float d[64];
            tmem_ld32_async(tp, reinterpret_cast<uint32_t*>(d));
            tmem_ld32_async(tp + 32, reinterpret_cast<uint32_t*>(d) + 32);
            tmem_wait_ld();
            const float4* e4 = reinterpret_cast<const float4*>(rows + 128 + 64 * half);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 e = e4[i];
                const float2 a = mul2(make_float2(x[4 * i], x[4 * i + 1]),
                                      add2(make_float2(d[4 * i], d[4 * i + 1]),
                                           make_float2(-e.x, -e.y)));
                const float2 b = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]),
                                      add2(make_float2(d[4 * i + 2], d[4 * i + 3]),
                                           make_float2(-e.z, -e.w)));
                d[4 * i] = a.x;
                d[4 * i + 1] = a.y;
                d[4 * i + 2] = b.x;
                d[4 * i + 3] = b.y;
            }
            if (masked) {   // a hidden pair's dP may be anything
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const int col = 64 * half + i;
                    if (col < lo || col >= limit) d[i] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
            tmem_st32(tp, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(sm.ds_full);
        }
        if (ok) ok = warp_wait(sm.acc_full, 0, sm.abort_flag, p.status);
        tc_fence_after();
        if (ok) {   // warps 0-3 write dV, warps 4-7 dK
            const int row = nb * 128 + r;
            const bool valid = row < len;
            const int64_t st_t = half ? p.dk_t : p.dv_t;
            uint16_t* o = (half ? p.dk + kvh * p.dk_h : p.dv + kvh * p.dv_h) +
                          (start + row - lane) * st_t;
            const bool bad = store_rows<D>((half ? tmK : tmV) + lane_off, 0, p.D,
                                           half ? p.scale : 1.0f, o, st_t, len - (row - lane));
            __syncwarp();   // a row's pieces come from four lanes
            uint32_t again = __ballot_sync(0xFFFFFFFFu, bad && valid);
            while (again) {
                const int s = __ffs(again) - 1;
                again &= again - 1;
                dkv_row(p, start, len, __shfl_sync(0xFFFFFFFFu, row, s), kvh, half);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ dQ

template <int D>
__global__ void __launch_bounds__(384, 1) attn_dq_kernel(const __grid_constant__ BwdParams p) {
    using C = BwdCfg<D>;
    const int tile = blockIdx.x / p.units;
    if (tile >= p.header[p.list]) return;
    const int h = blockIdx.x - tile * p.units;
    const int kvh = h / p.group;
    const int4 te = p.tiles[tile];
    const int64_t start = te.x;
    const int len = te.y;
    if (te.z < 0) {   // tokens of no sequence
        zero_rows(p.dq + start * p.dq_t + h * p.dq_h, p.dq_t, p.D, len);
        return;
    }
    const int n = te.z + 1;   // key blocks

    extern __shared__ uint8_t smem_raw[];
    BwdSmem<D> sm(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sm.init();
    if (warp == 8) {
        tmem_alloc(sm.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *sm.tmem_slot;
    const uint32_t tmP = tm + 256, tmQ = tm + 384;   // S alternates between tm and tm + 128

    if (warp >= 8) {
        setmaxnreg_dec<88>();
        if (warp == 9 && lane == 0) {
            // -------------------------------------------------------- loads
            const uint32_t ar = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const int tok = static_cast<int>(start);
            mbar_arrive_expect_tx(sm.res_full, 2 * C::TILE);
            load_tile<D>(ar, &p.mapQ, sm.res_full, tok + te.z * 128, h);
            load_tile<D>(ar + C::TILE, &p.mapO, sm.res_full, tok + te.z * 128, h);
            uint32_t st = 0, ph = 0, armed = 0, par = 0;
            bool ok = true;
            for (int it = 0; it < 2 * n; ++it) {
                if (!mbar_wait(&sm.empty[st], ph ^ 1u, sm.abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&sm.full[st], C::TILE);
                armed |= 1u << st;
                par = (par & ~(1u << st)) | (ph << st);
                load_tile<D>(ag + st * C::TILE, (it & 1) ? &p.mapV : &p.mapK, &sm.full[st],
                             tok + (it >> 1) * 128, kvh);
                if (++st == C::STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok || *sm.abort_flag) {   // let the armed copies land before leaving
                volatile int no_abort = 0;
                mbar_wait(sm.res_full, 0, &no_abort, nullptr, 20000000ull);
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait(&sm.full[s], (par >> s) & 1u, &no_abort, nullptr, 20000000ull);
            }
        } else if (warp == 8) {
            // -------------------------------------------------------- MMAs
            const uint32_t one = elect_lane();
            const uint32_t aQ = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const uint64_t dQ = desc_k(aQ), dO = desc_k(aQ + C::TILE);
            const auto stage = [](int it) { return static_cast<uint32_t>(it % C::STAGES); };
            const auto phase = [](int it) { return static_cast<uint32_t>(it / C::STAGES) & 1u; };
            const auto at = [&](int it) { return ag + stage(it) * C::TILE; };
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = warp_wait(bar, parity, sm.abort_flag, p.status);
                tc_fence_after();
                return got;
            };
            bool ok = wait(sm.res_full, 0) && wait(&sm.full[0], 0);
            if (ok) {
                mma_scores<D>(one, tm, dQ, desc_k(at(0)));
                commit(one, sm.s_full);
                ok = wait(&sm.full[1], 0);
            }
            if (ok) {
                mma_scores<D>(one, tmP, dO, desc_k(at(1)));
                commit(one, sm.dp_full);
                commit(one, &sm.empty[1]);
            }
            for (int j = 0; ok && j < n; ++j) {
                const int ik = 2 * j;
                if (j + 1 < n) {
                    // into the other S: its last scores were read before dS of
                    // block j - 1 was written
                    if (!(ok = wait(&sm.full[stage(ik + 2)], phase(ik + 2)))) break;
                    mma_scores<D>(one, tm + 128 * ((j + 1) & 1), dQ, desc_k(at(ik + 2)));
                    commit(one, sm.s_full);
                }
                if (!(ok = wait(sm.ds_full, j & 1u))) break;
                mma_tokens<D>(one, tmQ, tmP, desc_mn(at(ik)), 0, j > 0);
                mma_tokens<D>(one, tmQ, tmP + 64, desc_mn(at(ik)), 1, true);
                commit(one, &sm.empty[stage(ik)]);
                if (j + 1 < n) {
                    if (!(ok = wait(&sm.full[stage(ik + 3)], phase(ik + 3)))) break;
                    mma_scores<D>(one, tmP, dO, desc_k(at(ik + 3)));
                    commit(one, sm.dp_full);
                    commit(one, &sm.empty[stage(ik + 3)]);
                }
            }
            if (ok) commit(one, sm.acc_full);
            commit(one, sm.done);
            volatile int no_abort = 0;
            mbar_wait(sm.done, 0, &no_abort, p.status);
        }
    } else {
        setmaxnreg_inc<208>();
        // ------------------------------------------------------------ P and dS
        // a thread: query row r, key columns [64 half, 64 half + 64)
        const int half = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tp = tmP + lane_off + 64 * half;
        const int row = te.z * 128 + r;
        const bool valid = row < len;
        const float lse2 = valid ? p.lse2[h * p.T + start + row] : 0.f;
        float delta = valid ? p.delta[h * p.T + start + row] : 0.f;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nl = make_float2(-lse2, -lse2);
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const uint32_t ts = tm + 128 * (j & 1) + lane_off + 64 * half;
            if (!warp_wait(sm.s_full, j & 1u, sm.abort_flag, p.status)) {
                ok = false;
                if (n == 1) named_bar_sync(1, 256);   // given up: meets the others
                break;
            }
            tc_fence_after();
            float x[64];
            tmem_ld32_async(ts, reinterpret_cast<uint32_t*>(x));
            tmem_ld32_async(ts + 32, reinterpret_cast<uint32_t*>(x) + 32);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 a = fma2(make_float2(x[2 * i], x[2 * i + 1]), c2, nl);
                x[2 * i] = exp2_fast(a.x);
                x[2 * i + 1] = exp2_fast(a.y);
            }
            if (!warp_wait(sm.dp_full, j & 1u, sm.abort_flag, p.status)) {
                ok = false;
                if (n == 1) named_bar_sync(1, 256);
                break;
            }
            tc_fence_after();
            float d[64];
            tmem_ld32_async(tp, reinterpret_cast<uint32_t*>(d));
            tmem_ld32_async(tp + 32, reinterpret_cast<uint32_t*>(d) + 32);
            tmem_wait_ld();
            if (n == 1) {
                // the first 128 tokens of a sequence: the whole row is here,
                // so D_i = sum_j P_ij dP_ij without the rounding of P that
                // O's product carries, which weighs most in short rows (it
                // falls as 1 / sqrt(row)); the next kernel reads it too
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    part += 64 * half + i <= r ? x[i] * d[i] : 0.f;
                sm.rows[half * 128 + r] = part;
                named_bar_sync(1, 256);
                delta = sm.rows[r] + sm.rows[128 + r];
                if (valid && half == 0) p.delta[h * p.T + start + row] = delta;
            }
            const float2 nd = make_float2(-delta, -delta);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 a = mul2(make_float2(x[2 * i], x[2 * i + 1]),
                                      add2(make_float2(d[2 * i], d[2 * i + 1]), nd));
                d[2 * i] = a.x;
                d[2 * i + 1] = a.y;
            }
            if (j == n - 1) {   // the diagonal block; a hidden pair may hold anything
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (64 * half + i > r) d[i] = 0.f;
            }
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
            tmem_st32(tp, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(sm.ds_full);
        }
        if (ok) ok = warp_wait(sm.acc_full, 0, sm.abort_flag, p.status);
        tc_fence_after();
        uint32_t again = 0;
        if (ok) {
            uint16_t* o = p.dq + (start + row - lane) * p.dq_t + h * p.dq_h;
            const bool bad = store_rows<D / 2>(tmQ + lane_off, half * (D / 2), p.D, p.scale, o,
                                               p.dq_t, len - (row - lane));
            again = __ballot_sync(0xFFFFFFFFu, bad && valid);
        }
        // either half of a row may have met the value: the warps of the other
        // half have stored theirs before a row is written whole
        named_bar_sync(1, 256);
        while (again) {
            const int s = __ffs(again) - 1;
            again &= again - 1;
            dq_row(p, start, __shfl_sync(0xFFFFFFFFu, row, s), h, kvh);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 512);
}

template <int D>
int launch_pair(BwdParams& p, const AttnPlanLayout& l, const uint8_t* plan, int n_heads,
                int n_kv_heads, cudaStream_t st) {
    const int smem = BwdCfg<D>::SMEM;
    if (ensure_smem_attr(reinterpret_cast<const void*>(attn_dkv_kernel<D>), smem) ||
        ensure_smem_attr(reinterpret_cast<const void*>(attn_dq_kernel<D>), smem))
        return MOE_ECUDA;
    const int64_t gkv = l.max128 * n_kv_heads, gq = l.max128 * n_heads;
    p.list = 0;
    p.tiles = reinterpret_cast<const int4*>(plan + l.q128);
    p.units = n_heads;
    attn_dq_kernel<D><<<static_cast<int>(gq), 384, smem, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_dq");
    p.list = 1;
    p.tiles = reinterpret_cast<const int4*>(plan + l.kv128);
    p.units = n_kv_heads;
    attn_dkv_kernel<D><<<static_cast<int>(gkv), 384, smem, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_dkv");
    return MOE_OK;
}

}  // namespace

int64_t attention_backward_ws(int64_t T, int n_heads) { return 2 * T * n_heads * 4; }

int launch_attention_bwd(const moe_attention_t& a, const void* plan, const uint16_t* q,
                         const uint16_t* k, const uint16_t* v, const uint16_t* out,
                         const uint16_t* rest, const float* lse, const uint16_t* dout,
                         uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, int32_t* status,
                         cudaStream_t st) {
    const int D = a.head_dim;
    float* lse2 = static_cast<float*>(ws);
    float* delta = lse2 + a.T * a.n_heads;
    BwdParams p;
    memset(&p, 0, sizeof(p));
    if (attn_tensor_map(&p.mapQ, q, D, a.T, a.n_heads, a.q_t, a.q_h) ||
        attn_tensor_map(&p.mapK, k, D, a.T, a.n_kv_heads, a.k_t, a.k_h) ||
        attn_tensor_map(&p.mapV, v, D, a.T, a.n_kv_heads, a.v_t, a.v_h) ||
        attn_tensor_map(&p.mapO, dout, D, a.T, a.n_heads, a.do_t, a.do_h))
        return MOE_ECUDA;
    const AttnPlanLayout l = attn_plan_layout(a.T, a.n_seqs);
    const int64_t blocks = (a.T * a.n_heads + 31) / 32;
    if (blocks >= (1ll << 31) || l.max128 * a.n_heads >= (1ll << 31)) return MOE_EINVAL;
    DeltaParams d;
    d.T = a.T;
    d.heads = a.n_heads;
    d.D = D;
    d.o_t = a.o_t;
    d.o_h = a.o_h;
    d.do_t = a.do_t;
    d.do_h = a.do_h;
    d.out = out;
    d.rest = rest;
    d.dout = dout;
    d.lse = lse;
    d.lse2 = lse2;
    d.delta = delta;
    attn_delta_kernel<<<static_cast<int>(blocks), 256, 0, st>>>(d);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_delta");
    const uint8_t* b = static_cast<const uint8_t*>(plan);
    p.header = reinterpret_cast<const int32_t*>(b);
    p.group = a.n_heads / a.n_kv_heads;
    p.D = D;
    p.T = a.T;
    p.q_t = a.q_t;
    p.q_h = a.q_h;
    p.k_t = a.k_t;
    p.k_h = a.k_h;
    p.v_t = a.v_t;
    p.v_h = a.v_h;
    p.do_t = a.do_t;
    p.do_h = a.do_h;
    p.q = q;
    p.k = k;
    p.v = v;
    p.dout = dout;
    p.dq_t = a.dq_t;
    p.dq_h = a.dq_h;
    p.dk_t = a.dk_t;
    p.dk_h = a.dk_h;
    p.dv_t = a.dv_t;
    p.dv_h = a.dv_h;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.lse2 = lse2;
    p.delta = delta;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    p.status = status;
    return D <= 64 ? launch_pair<64>(p, l, b, a.n_heads, a.n_kv_heads, st)
                   : launch_pair<128>(p, l, b, a.n_heads, a.n_kv_heads, st);
}

}  // namespace moe
