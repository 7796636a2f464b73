// attention_bwd.cu -- gradients of the causal packed attention.
//
//   P_ij = 2^(c s_ij - lse_i log2 e)      D_i = dO_i . O_i
//   dV_j = sum_i P_ij dO_i                dS_ij = P_ij (dO_i . V_j - D_i)
//   dK_j = scale sum_i dS_ij Q_i          dQ_i = scale sum_j dS_ij K_j
//
// Two kernels.  The first, one CTA an SM working through the batch, takes 128
// query rows at a time, forms their D (from O in two bf16 parts) and walks
// their key blocks for dQ.  The second gives 128 keys of one key/value head to
// a CTA, or to a cluster of two or four where there are few, and walks the
// query blocks of all the group's heads, so dK and dV are summed in TMEM (a
// cluster's parts then in their order through shared memory) and written
// once: no atomics, the same bits every time.
// Both compute P and dP again (seven products of 128 x 128 x D a block pair
// where five are needed): the price of a fixed order without a pass over
// memory for dQ.  Warps 0-15 form P and dS (a thread holds 32 of the 128
// columns of its TMEM lane), warp 16 issues the MMAs, warp 17 the TMA loads.
// P and dS return to the columns of S and dP as bf16 A operands.
//   8192 tokens in 4 sequences, 16/4 heads of 128 (one product 25 us at a library
// product's rate): dQ 127 us, dK and dV 141 us.  dK and dV: the longest column of
// blocks is 104 rounds of 128 x 128 pairs (26 blocks, 4 heads) where an even share
// would be 82, and sets the time: about 2500 cycles a round and 8 us of start and
// end.  The products of a round are 2048 of them, and so is their operands' way
// through shared memory (computed from the tiles' bytes; no counter shows it).
// dQ: 2200 cycles a round (products 1536, operands 1750, computed likewise, and P
// and dS of a block follow each other), 6500 between two pieces of work (D, the
// store of dQ).  Head widths 72 to 120 run the products of 128: 16384 tokens in 7,
// 48/8 heads, dQ and dK/dV of 128 794 and 884 us, of 96 778 and 867, of 80 769 and
// 844, of 64 610 and 690.
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
    const uint16_t *out, *rest;
    int64_t o_t, o_h;
    const float* lse;
    float *lse2, *delta;   // [heads, T]: lse log2 e and D, written by the dQ kernel
    float scale, scale_log2;
    int32_t* status;
};

// ------------------------------------------------------------------ what rows see that is not finite

// Rows [row0, row0 + 32) of columns [c0, c0 + 32) of dQ: a column in which a key of
// the row's own block that it sees is not finite is NaN (either the row's lse
// is, or the key's weight is 0).  A column a lane.
__device__ __noinline__ void dq_visible(const BwdParams& p, int64_t start, int len, int row0, int h,
                                        int kvh, int c0) {
    const int c = c0 + (threadIdx.x & 31);
    if (c >= p.D) return;
    bool odd = false;
    for (int j = row0 & ~127; j < min(row0 + 32, len); ++j) {
        odd |= bf16_odd(p.k[(start + j) * p.k_t + kvh * p.k_h + c]);
        if (odd && j >= row0) p.dq[(start + j) * p.dq_t + h * p.dq_h + c] = 0x7FFF;
    }
}

// Key rows [row0, row0 + 32) of columns [c0, c0 + 32) of dV: adds what of the
// gradients of the queries of its own block, from the key on, is not finite.
// (dK needs nothing: such a query's lse or D is not finite, and so is its dS.)
__device__ __noinline__ void dv_visible(const BwdParams& p, int64_t start, int len, int row0, int kvh,
                                        int c0) {
    const int c = c0 + (threadIdx.x & 31);
    if (c >= p.D) return;
    float sum = 0.f;   // of what is not finite among the queries so far
    for (int i = min((row0 & ~127) + 128, len) - 1; i >= row0; --i) {
        for (int h = kvh * p.group; h < (kvh + 1) * p.group; ++h) {
            const uint16_t g = p.dout[(start + i) * p.do_t + h * p.do_h + c];
            if (bf16_odd(g)) sum += bf16_f32(g);
        }
        if (sum != 0.f && i < row0 + 32) {
            uint16_t* o = p.dv + (start + i) * p.dv_t + kvh * p.dv_h + c;
            *o = f32_bf16(bf16_f32(*o) + sum);
        }
    }
}

__device__ __forceinline__ void zero_rows(uint16_t* base, int64_t st_t, int D, int rows) {
    for (int i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
        *reinterpret_cast<uint4*>(base + (i / (D / 8)) * st_t + i % (D / 8) * 8) =
            make_uint4(0, 0, 0, 0);
}

// Columns [c0, c0 + 32) of the warp's 32 accumulator rows, times `f`, as bf16.
__device__ __forceinline__ void take_rows(uint32_t taddr, int c0, float f, uint4 (&v)[4]) {
    uint32_t a[32];
    tmem_ld32(taddr + c0, a);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = mul2(make_float2(__uint_as_float(a[8 * g + 2 * e]),
                                              __uint_as_float(a[8 * g + 2 * e + 1])),
                                  make_float2(f, f));
            w[e] = pack_bf16x2(x.x, x.y);
        }
        v[g] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Two resident tiles, a ring of ST streamed ones, NF of the rows' scalars, barriers.
template <int D, int ST, int NF>
struct BwdCfg {
    static constexpr int SCALARS = NF;
    static constexpr int TILE = 128 * D * 2;
    static constexpr int STAGES = ST;
    static constexpr int SMEM = 2 * TILE + STAGES * TILE + SCALARS * 4 + 272;
};
// Warps 0-15 form P and dS; then the MMA warp, the load warp, two idle ones.
constexpr int kBwdThreads = 640, kMmaWarp = 16, kLoadWarp = 17, kFormers = 512;
constexpr int dkv_stages(int D) { return D == 128 ? 4 : 8; }
constexpr int dq_stages(int D) { return D == 128 ? 5 : 8; }
template <int D>
using DkvCfg = BwdCfg<D, dkv_stages(D), 1024>;
template <int D>
using DqCfg = BwdCfg<D, dq_stages(D), 512>;

// Shared-memory layout and barriers of both kernels: two resident tiles, a
// ring of streamed ones.
template <class C>
struct BwdSmem {
    uint8_t *res, *ring;
    float* rows;   // scalars of query rows: dQ two blocks of 256, dK and dV 64 a warp
    uint64_t *full, *empty, *res_full, *res_empty, *s_full, *s_free, *dp_full, *p_full, *ds_full, *acc_full,
        *acc_empty, *done, *sums_there, *sums_read;
    uint32_t* tmem_slot;
    volatile int *abort_flag, *odd_flag;   // odd: a value that is not finite was met
    __device__ explicit BwdSmem(uint8_t* raw_ptr) {
        res = raw_ptr;
        ring = res + 2 * C::TILE;
        rows = reinterpret_cast<float*>(ring + C::STAGES * C::TILE);
        full = reinterpret_cast<uint64_t*>(rows + C::SCALARS);
        empty = full + C::STAGES;
        res_full = empty + C::STAGES;
        res_empty = res_full + 1;
        s_full = res_empty + 1;
        s_free = s_full + 1;
        dp_full = s_free + 1;
        p_full = dp_full + 2;
        ds_full = p_full + 1;
        acc_full = ds_full + 2;
        acc_empty = acc_full + 1;
        done = acc_empty + 1;
        sums_there = done + 1;
        sums_read = sums_there + 1;
        tmem_slot = reinterpret_cast<uint32_t*>(sums_read + 1);
        abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
        odd_flag = abort_flag + 1;
    }
    __device__ void init(int parts) {   // parts: CTAs of a cluster
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(res_full, 1);
        mbar_init(s_full, 1);
        mbar_init(s_free, 16);   // one arrival a warp
        mbar_init(&dp_full[0], 1);   // dQ: one for each dP, since the next one may be
        mbar_init(&dp_full[1], 1);   // ready before this one is looked for
        mbar_init(p_full, 16);
        mbar_init(&ds_full[0], 16);   // likewise
        mbar_init(&ds_full[1], 16);
        mbar_init(res_empty, 1);
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);
        mbar_init(done, 1);
        mbar_init(sums_there, 16 * parts);   // one arrival a warp and CTA
        mbar_init(sums_read, 16 * parts);
        *abort_flag = 0;
        *odd_flag = 0;
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

// Byte offset of 16-byte piece `q` of row `r` of a part's sums.
template <int D>
__device__ __forceinline__ uint32_t sum_at(int r, int q) {
    return r * (2 * D * 4) + ((q ^ (r & 7)) * 16);
}

template <int D, int PARTS>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dkv_kernel(const __grid_constant__ BwdParams p) {
    using C = DkvCfg<D>;
    // the CTAs of a cluster share one block of keys: a part of its query
    // blocks each, their sums joined through shared memory at the end
    const uint32_t part = PARTS > 1 ? cluster_ctarank() : 0u;
    const int item = blockIdx.x / PARTS;
    const int tile = item / p.units;
    if (tile >= p.header[p.list]) return;
    const int kvh = item - tile * p.units;
    const int4 te = p.tiles[tile];
    if (!moe_check(plan_entry_ok(te, p.T, 128), 1205)) return;
    const int64_t start = te.x;
    const int len = te.y;
    if (te.z < 0) {   // tokens of no sequence
        if (part) return;
        zero_rows(p.dk + start * p.dk_t + kvh * p.dk_h, p.dk_t, p.D, len);
        zero_rows(p.dv + start * p.dv_t + kvh * p.dv_h, p.dv_t, p.D, len);
        return;
    }
    const int nb = te.z, nblk = (len + 127) / 128;
    const int per_head = nblk - nb;          // query blocks of one head
    const int all = p.group * per_head;
    const int first = static_cast<int>(all * part / PARTS);
    const int n = static_cast<int>(all * (part + 1) / PARTS) - first;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_u32(smem_raw) & 1023u) {   // the swizzled tiles' alignment
        report_error(p.status, MOE_ECUDA);
        return;
    }
    BwdSmem<C> sm(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sm.init(PARTS);
    if (warp == kMmaWarp) {
        tmem_alloc(sm.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (PARTS > 1) cluster_sync();   // the others' barriers exist
    const uint32_t tm = *sm.tmem_slot;
    const uint32_t tmS = tm, tmP = tm + 128, tmV = tm + 256, tmK = tm + 384;

    if (warp >= kMmaWarp) {
        setmaxnreg_dec<64>();
        if (warp == kLoadWarp && lane == 0) {
            // -------------------------------------------------------- loads
            const uint32_t ar = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const int tok = static_cast<int>(start);
            if (n) {
                mbar_arrive_expect_tx(sm.res_full, 2 * C::TILE);
                load_tile<D>(ar, &p.mapK, sm.res_full, tok + nb * 128, kvh);
                load_tile<D>(ar + C::TILE, &p.mapV, sm.res_full, tok + nb * 128, kvh);
            }
            uint32_t st = 0, ph = 0, armed = 0, par = 0;
            bool ok = true;
            int h = kvh * p.group + first / per_head, i = nb + first % per_head;
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
                if (n) mbar_wait(sm.res_full, 0, &no_abort, nullptr, 20000000ull);
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait(&sm.full[s], (par >> s) & 1u, &no_abort, nullptr, 20000000ull);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMAs
            const uint32_t one = elect_lane();
            const uint32_t aK = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const uint64_t dK = desc_k(aK), dV = desc_k(aK + C::TILE);
            const auto stage = [](int it) { return static_cast<uint32_t>(it % C::STAGES); };
            const auto phase = [](int it) { return static_cast<uint32_t>(it / C::STAGES) & 1u; };
            const auto at = [&](int it) { return ag + stage(it) * C::TILE; };
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = warp_wait_short(bar, parity, sm.abort_flag, p.status);
                tc_fence_after();
                return got;
            };
            bool ok = n && wait(sm.res_full, 0) && wait(&sm.full[0], 0);
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
                mma_tokens_quarters<D>(one, tmV, tmS, desc_mn(at(io)), it > 0);
                commit(one, &sm.empty[stage(io)]);
                if (it + 1 < n) {
                    if (!(ok = wait(&sm.full[stage(iq + 2)], phase(iq + 2)))) break;
                    // runs after the product above has read P from these columns
                    mma_scores<D>(one, tmS, dK, desc_k(at(iq + 2)));
                    commit(one, sm.s_full);
                }
                if (!(ok = wait(sm.ds_full, it & 1u))) break;
                mma_tokens_quarters<D>(one, tmK, tmP, desc_mn(at(iq)), it > 0);
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
        setmaxnreg_inc<104>();
        // ------------------------------------------------------------ P and dS
        // a thread: key row r, query columns [c0, c0 + 32)
        const int quarter = warp >> 2, c0 = 32 * quarter;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmS + lane_off + c0, tp = tmP + lane_off + c0;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        // Each warp brings the lse2 and D of its 32 query columns itself, a
        // block ahead: through a barrier over all sixteen, the first to finish
        // a block waited for the last (900 of 2490 cycles).
        float* rows = sm.rows + warp * 64;
        int qb = nb + first % per_head;
        int64_t at = (kvh * p.group + first / per_head) * p.T + start + c0 + lane;   // its head's row 0
        // (Behind the sequence's end too, where they tell of the rows there.)
        const int64_t left = p.T - start;
        const auto fetch = [&](const float* src) {
            return qb * 128 + c0 + lane < left ? src[at + qb * 128] : 0.f;
        };
        float l_next = n ? fetch(p.lse2) : 0.f, d_next = n ? fetch(p.delta) : 0.f;
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            __syncwarp();
            rows[lane] = l_next;
            rows[32 + lane] = d_next;
            __syncwarp();
            const bool finite = l_next - l_next == 0.f && d_next - d_next == 0.f;
            const int limit = min(128, len - qb * 128);   // query rows in this block
            const bool diagonal = qb == nb, masked = diagonal || limit < 128;
            // columns whose Q or dO may not be finite, where hidden pairs are
            uint32_t odd = 0;
            if (masked)
                odd = __ballot_sync(0xFFFFFFFFu, !finite) & (diagonal ? ~0u : bits_from(limit - c0));
            // the columns that count: from the diagonal to the last row
            const uint32_t seen = bits_from((qb == nb ? r : 0) - c0) & ~bits_from(limit - c0);
            if (++qb == nblk) {
                qb = nb;
                at += p.T;
            }
            if (it + 1 < n) {
                l_next = fetch(p.lse2);
                d_next = fetch(p.delta);
            }

            if (odd) {   // not before S and dP are done with the tiles
                const uint32_t q = 2 * it, st0 = q % C::STAGES, st1 = (q + 1) % C::STAGES;
                if (!(ok = warp_wait(sm.s_full, it & 1u, sm.abort_flag, p.status) &&
                           warp_wait(sm.dp_full, it & 1u, sm.abort_flag, p.status) &&
                           warp_wait(&sm.full[st0], q / C::STAGES & 1u, sm.abort_flag, p.status) &&
                           warp_wait(&sm.full[st1], (q + 1) / C::STAGES & 1u, sm.abort_flag,
                                     p.status)))
                    break;
                const uint32_t ring = smem_u32(sm.ring);
                for (uint32_t m = odd; m; m &= m - 1) {
                    const int e = __ffs(m) - 1;
                    if ((e & 3) != (warp & 3)) continue;   // four warps meet these columns
                    clean_row<D>(ring + st0 * C::TILE, c0 + e);
                    clean_row<D>(ring + st1 * C::TILE, c0 + e);
                }
                fence_proxy_async_smem();
                if (lane == 0) *sm.odd_flag = 1;
            }
            if (!(ok = warp_wait(sm.s_full, it & 1u, sm.abort_flag, p.status))) break;
            tc_fence_after();
            float x[32];
            tmem_ld32_async(ts, reinterpret_cast<uint32_t*>(x));
            tmem_wait_ld();
            uint32_t pk[16];
            const float4* l4 = reinterpret_cast<const float4*>(rows);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
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
                for (int i = 0; i < 32; ++i)
                    if (!(seen >> i & 1u)) x[i] = 0.f;
            }
            // P, and dS below, as bf16: what the tensor cores take beside bf16 dO
            // and Q, with fp32's range.  A rounding of at most 2^-8 a pair.
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st16(ts, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.p_full);

            if (!(ok = warp_wait(sm.dp_full, it & 1u, sm.abort_flag, p.status))) break;
            tc_fence_after();
            float d[32];
            tmem_ld32_async(tp, reinterpret_cast<uint32_t*>(d));
            tmem_wait_ld();
            const float4* e4 = reinterpret_cast<const float4*>(rows + 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
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
                for (int i = 0; i < 32; ++i)
                    if (!(seen >> i & 1u)) d[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
            tmem_st16(tp, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.ds_full);
        }
        if (n) {
            if (ok) ok = warp_wait(sm.acc_full, 0, sm.abort_flag, p.status);
            tc_fence_after();
        }
        const int row = nb * 128 + r, row0 = row - lane;
        if constexpr (PARTS > 1) {
            // this part's sums, rows of [dV | dK], into the ring (every copy
            // into it has landed, every product has read it): 16-byte pieces,
            // swizzled by the row so that a warp's rows spread over the banks
            for (int i = quarter; i < 2 * D / 32; i += 4) {
                uint32_t a[32];
                if (n) tmem_ld32((i >= D / 32 ? tmK - D : tmV) + lane_off + 32 * i, a);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<uint4*>(sm.ring + sum_at<D>(r, 8 * i + e)) =
                        n ? make_uint4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3])
                          : make_uint4(0, 0, 0, 0);
            }
            // the parts meet at barriers in shared memory, whose waits have a
            // limit, unlike the cluster's own barrier
            __syncwarp();
            if (lane < PARTS) mbar_arrive_cluster(mapa_shared(smem_u32(sm.sums_there), lane));
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(sm.sums_there, 0, p.status)) && ok;
            // this CTA's share of the 2 D columns, 32 at a time: the parts'
            // sums in their order
            constexpr int PIECES = 2 * D / 32 / PARTS;
            static_assert(PIECES <= 4, "one piece a warp at most");
            const int at0 = (static_cast<int>(part) * PIECES + quarter) * 32;
            const int which = at0 >= D, col = at0 - which * D;   // of [dV | dK]
            if (ok && quarter < PIECES) {
                const float f = which ? p.scale : 1.0f;
                const int64_t st_t = which ? p.dk_t : p.dv_t;
                uint16_t* o = (which ? p.dk + kvh * p.dk_h : p.dv + kvh * p.dv_h) +
                              (start + row0) * st_t + col + 4 * (lane & 7);
                // eight lanes a row, four rows at a time: whole lines of the
                // other CTAs' memory (a row a lane measured four times slower)
#pragma unroll
                for (int k0 = 0; k0 < 8; k0 += 2) {
                    float4 x[PARTS][2];
#pragma unroll
                    for (int s = 0; s < PARTS; ++s)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            x[s][k] = ld_cluster4(mapa_shared(
                                smem_u32(sm.ring) + sum_at<D>(32 * (warp & 3) + 4 * (k0 + k) + lane / 8,
                                                              at0 / 4 + (lane & 7)), s));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float2 lo = make_float2(x[0][k].x, x[0][k].y);
                        float2 hi = make_float2(x[0][k].z, x[0][k].w);
#pragma unroll
                        for (int s = 1; s < PARTS; ++s) {
                            lo = add2(lo, make_float2(x[s][k].x, x[s][k].y));
                            hi = add2(hi, make_float2(x[s][k].z, x[s][k].w));
                        }
                        lo = mul2(lo, make_float2(f, f));
                        hi = mul2(hi, make_float2(f, f));
                        const int rr = 4 * (k0 + k) + lane / 8;
                        if (row0 + rr < len && col + 4 * (lane & 7) < p.D)
                            *reinterpret_cast<uint2*>(o + rr * st_t) =
                                make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(hi.x, hi.y));
                    }
                }
            }
            bool odd = false;   // any part's queries
#pragma unroll
            for (int s = 0; s < PARTS; ++s)
                odd |= ld_cluster(mapa_shared(smem_u32(const_cast<int*>(sm.odd_flag)), s)) != 0;
            // nobody leaves while its sums may still be read
            __syncwarp();   // (and a row's pieces come from eight lanes)
            if (lane < PARTS) mbar_arrive_cluster(mapa_shared(smem_u32(sm.sums_read), lane));
            mbar_wait_cluster(sm.sums_read, 0, p.status, 4 * kWaitTimeoutNs);
            __syncwarp();
            if (odd && ok && quarter < PIECES && !which) dv_visible(p, start, len, row0, kvh, col);
        } else if (ok) {   // 32 columns of [dV | dK] at a time
            for (int i = quarter; i < 2 * D / 32; i += 4) {
                const int which = i >= D / 32, col = 32 * i - which * D;
                const int64_t st_t = which ? p.dk_t : p.dv_t;
                uint16_t* o = (which ? p.dk + kvh * p.dk_h : p.dv + kvh * p.dv_h) +
                              (start + row0) * st_t;
                uint4 v[4];
                take_rows((which ? tmK : tmV) + lane_off, col, which ? p.scale : 1.0f, v);
                store_quad(v, o, st_t, len - row0, col, p.D);
                __syncwarp();   // a row's pieces come from four lanes
                if (!which && *sm.odd_flag) dv_visible(p, start, len, row0, kvh, col);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ dQ

struct DqWork {
    int64_t start;
    int len, block, h, kvh, n;   // n: key blocks
    __device__ DqWork() {}
    __device__ DqWork(const BwdParams& p, int item) {
        const int tile = item / p.units;
        const int4 te = p.tiles[tile];
        start = te.x;
        len = te.y;
        block = te.z;
        h = item - tile * p.units;
        kvh = h / p.group;
        n = block + 1;
    }
};

// D of a block of 128 query rows, D_i = dO_i . (out_i + rest_i): eight lanes a
// row, 16 bytes a load, all loads of a block under way at once.
template <int D>
struct RowDots {
    uint4 o[2][D / 64], e[2][D / 64], g[2][D / 64];
    float lse;
    __device__ void load(const BwdParams& p, const DqWork& w) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = w.block * 128 + 64 * k + (tid >> 3);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = ((tid & 7) + 8 * c) * 8;
                o[k][c] = e[k][c] = g[k][c] = make_uint4(0, 0, 0, 0);
                if (w.block <= 0 || row >= w.len || col >= p.D) continue;   // a first block's: below
                const int64_t at = (w.start + row) * p.o_t + w.h * p.o_h + col;
                o[k][c] = *reinterpret_cast<const uint4*>(p.out + at);
                e[k][c] = *reinterpret_cast<const uint4*>(p.rest + at);
                g[k][c] = *reinterpret_cast<const uint4*>(
                    p.dout + (w.start + row) * p.do_t + w.h * p.do_h + col);
            }
        }
        const int row = w.block * 128 + tid;
        lse = tid < 128 && w.block >= 0 && row < w.len ? p.lse[w.h * p.T + w.start + row] : 0.f;
    }
    // brings the rows into L2, by one warp
    __device__ static void prefetch(const BwdParams& p, const DqWork& w, int lane) {
        const int rows = w.block <= 0 ? 0 : min(128, w.len - w.block * 128);
        for (int i = lane; i < rows * (D / 64); i += 32) {   // a line of 64 channels
            const int row = w.block * 128 + i / (D / 64), col = i % (D / 64) * 64;
            const int64_t at = (w.start + row) * p.o_t + w.h * p.o_h + col;
            prefetch_l2(p.out + at);
            prefetch_l2(p.rest + at);
            prefetch_l2(p.dout + (w.start + row) * p.do_t + w.h * p.do_h + col);
        }
    }
    // D and lse log2 e of the block's rows to rows[0..127], rows[128..255] and,
    // for the dK, dV kernel, to global memory
    __device__ void finish(const BwdParams& p, const DqWork& w, float* rows) const {
        const int tid = threadIdx.x;
        const int64_t at = w.h * p.T + w.start + w.block * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const uint32_t ov[4] = {o[k][c].x, o[k][c].y, o[k][c].z, o[k][c].w};
                const uint32_t ev[4] = {e[k][c].x, e[k][c].y, e[k][c].z, e[k][c].w};
                const uint32_t gv[4] = {g[k][c].x, g[k][c].y, g[k][c].z, g[k][c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum = fma2(bf16x2_f32(gv[i]), add2(bf16x2_f32(ov[i]), bf16x2_f32(ev[i])), sum);
            }
            float d = sum.x + sum.y;
#pragma unroll
            for (int s = 4; s > 0; s >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, s);
            const int row = 64 * k + (tid >> 3);
            if ((tid & 7) == 0) {
                rows[row] = d;
                // a first block's is formed from P and dP below
                if (w.n > 1 && w.block * 128 + row < w.len) p.delta[at + row] = d;
            }
        }
        if (tid < 128) {   // (of scores that are all -infinity: weights of 0 / 0)
            const float lse2 = lse == -INFINITY ? NAN : lse * kLog2e;
            rows[128 + tid] = lse2;
            if (w.block * 128 + tid < w.len) p.lse2[at + tid] = lse2;
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dq_kernel(const __grid_constant__ BwdParams p) {
    // keys stay for dQ, a block longer than values: a ring of its own for each,
    // or the next values would wait behind them
    using C = DqCfg<D>;
    constexpr uint32_t VS = dq_stages(D) * 2 / 5, KS = dq_stages(D) - VS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_u32(smem_raw) & 1023u) {   // the swizzled tiles' alignment
        report_error(p.status, MOE_ECUDA);
        return;
    }
    report_refused(p.header, p.status);
    BwdSmem<C> sm(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sm.init(1);
    if (warp == kMmaWarp) {
        tmem_alloc(sm.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *sm.tmem_slot;
    const uint32_t tmP = tm + 128, tmQ = tm + 384;   // S at tm; dP alternates: + 128
    AttnItems items(p.header[p.list] * p.units);
    int item;
    const auto next = [&] { return items.next(item, p.tiles, p.units, p.T, 128, 1204); };

    if (warp >= kMmaWarp) {
        setmaxnreg_dec<64>();
        if (warp == kLoadWarp) {
            // -------------------------------------------------------- loads
            const uint32_t ar = smem_u32(sm.res), ag = smem_u32(sm.ring);
            uint32_t kt = 0, vt = 0, armed = 0, par = 0, done = 0;   // tiles of either ring so far
            const auto issue = [&](const DqWork& w) {   // lane 0
                const int tok = static_cast<int>(w.start);
                if (done && !mbar_wait(sm.res_empty, (done - 1) & 1u, sm.abort_flag, p.status))
                    return false;
                ++done;
                mbar_arrive_expect_tx(sm.res_full, 2 * C::TILE);
                load_tile<D>(ar, &p.mapQ, sm.res_full, tok + w.block * 128, w.h);
                load_tile<D>(ar + C::TILE, &p.mapO, sm.res_full, tok + w.block * 128, w.h);
                for (int it = 0; it < 2 * w.n; ++it) {
                    const bool isv = it & 1;
                    const uint32_t t = isv ? vt++ : kt++, ring = isv ? VS : KS;
                    const uint32_t st = t % ring + (isv ? KS : 0), ph = t / ring & 1u;
                    if (!mbar_wait(&sm.empty[st], ph ^ 1u, sm.abort_flag, p.status)) return false;
                    mbar_arrive_expect_tx(&sm.full[st], C::TILE);
                    armed |= 1u << st;
                    par = (par & ~(1u << st)) | (ph << st);
                    load_tile<D>(ag + st * C::TILE, isv ? &p.mapV : &p.mapK, &sm.full[st],
                                 tok + (it >> 1) * 128, w.kvh);
                }
                return true;
            };
            bool ok = true, more = next();
            while (ok && more) {
                const DqWork w(p, item);
                if (lane == 0 && w.block >= 0) ok = issue(w);
                ok = __all_sync(0xFFFFFFFFu, ok);
                // this item's last tiles are under way: the next one's rows,
                // which its D is formed from, into L2
                if ((more = next())) RowDots<D>::prefetch(p, DqWork(p, item), lane);
            }
            if (lane == 0 && (!ok || *sm.abort_flag)) {   // let the armed copies land before leaving
                volatile int no_abort = 0;
                if (done) mbar_wait(sm.res_full, (done - 1) & 1u, &no_abort, nullptr, 20000000ull);
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait(&sm.full[s], (par >> s) & 1u, &no_abort, nullptr, 20000000ull);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMAs
            const uint32_t one = elect_lane();
            const uint32_t aQ = smem_u32(sm.res), ag = smem_u32(sm.ring);
            const uint64_t dQ = desc_k(aQ), dO = desc_k(aQ + C::TILE);
            // key blocks whose scores, whose dS have been met, items so far
            uint32_t cs = 0, cd = 0, done = 0;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = warp_wait_short(bar, parity, sm.abort_flag, p.status);
                tc_fence_after();
                return got;
            };
            const auto landed = [&](uint32_t t, uint32_t ring, uint32_t from) {
                return wait(&sm.full[t % ring + from], t / ring & 1u);
            };
            const auto tile = [&](uint32_t st) { return ag + st * C::TILE; };
            // S and dP of the next key block, a block ahead of its dS: S once
            // the last one has been read, dP into the columns whose dS the
            // product before last has read
            const auto scores = [&](bool last) {
                if (!landed(cs, KS, 0) || (cs && !wait(sm.s_free, (cs - 1) & 1u))) return false;
                mma_scores<D>(one, tm, dQ, desc_k(tile(cs % KS)));
                commit(one, sm.s_full);
                if (!landed(cs, VS, KS)) return false;
                mma_scores<D>(one, tmP + 128 * (cs & 1u), dO, desc_k(tile(cs % VS + KS)));
                commit(one, &sm.dp_full[cs & 1u]);
                commit(one, &sm.empty[cs % VS + KS]);
                if (last) commit(one, sm.res_empty);
                ++cs;
                return true;
            };
            bool ok = true;
            while (ok && next()) {
                const DqWork w(p, item);
                if (w.block < 0) continue;
                if (!(ok = wait(sm.res_full, done++ & 1u) && scores(w.n == 1))) break;
                for (int j = 0; j < w.n; ++j) {
                    if (j + 1 < w.n && !(ok = scores(j + 2 == w.n))) break;
                    if (!(ok = wait(&sm.ds_full[cd & 1u], (cd >> 1) & 1u))) break;
                    // the last item's dQ has been read
                    if (j == 0 && done > 1 && !(ok = wait(sm.acc_empty, done & 1u))) break;
                    mma_tokens_quarters<D>(one, tmQ, tmP + 128 * (cd & 1u),
                                           desc_mn(tile(cd % KS)), j > 0);
                    commit(one, &sm.empty[cd++ % KS]);
                }
                if (ok) commit(one, sm.acc_full);
            }
            commit(one, sm.done);
            volatile int no_abort = 0;
            mbar_wait(sm.done, 0, &no_abort, p.status);
        }
    } else {
        setmaxnreg_inc<104>();
        // ------------------------------------------------------------ P and dS
        // a thread: query row r, key columns [c0, c0 + 32)
        const int quarter = warp >> 2, c0 = 32 * quarter;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tm + lane_off + c0;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        uint32_t blocks = 0, done = 0;   // key blocks and items so far
        // a warp that has given up (ok false) still meets the others at every
        // barrier, and does nothing else
        bool ok = true;
        DqWork w;
        while (next()) {
            w = DqWork(p, item);
            if (w.block < 0) {   // tokens of no sequence
                uint16_t* o = p.dq + w.start * p.dq_t + w.h * p.dq_h;
                for (int i = threadIdx.x; i < w.len * (p.D / 8); i += kFormers)
                    *reinterpret_cast<uint4*>(o + (i / (p.D / 8)) * p.dq_t + i % (p.D / 8) * 8) =
                        make_uint4(0, 0, 0, 0);
                // dK and dV take it that these rows may hold anything
                for (int i = threadIdx.x; i < w.len; i += kFormers)
                    p.lse2[w.h * p.T + w.start + i] = NAN;
                continue;
            }
            float* rows = sm.rows + (done & 1u) * 256;
            {
                RowDots<D> dots;
                dots.load(p, w);
                dots.finish(p, w, rows);
            }
            named_bar_sync(1, kFormers);
            float delta = rows[r];
            const float lse2 = rows[128 + r];
            const int row = w.block * 128 + r, row0 = row - lane, n = w.n;
            const bool valid = row < w.len;
            const float2 nl = make_float2(-lse2, -lse2);
            for (int j = 0; j < n; ++j, ++blocks) {
                const uint32_t tp = tmP + 128 * (blocks & 1u) + lane_off + c0;
                bool odd = false;
                const uint32_t kst = blocks % KS;
                if (j == n - 1) {   // the diagonal block's K
                    ok = ok && warp_wait(&sm.full[kst], blocks / KS & 1u, sm.abort_flag, p.status);
                    odd = ok && odd_tile<D>(smem_u32(sm.ring) + kst * C::TILE, threadIdx.x, kFormers);
                }
                if (!(ok = ok && warp_wait(sm.s_full, blocks & 1u, sm.abort_flag, p.status))) {
                    for (int i = 0; n == 1 && i < 2; ++i) named_bar_sync(1, kFormers);
                    break;
                }
                tc_fence_after();
                float x[32];
                tmem_ld32_async(ts, reinterpret_cast<uint32_t*>(x));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.s_free);
                if (odd) {   // S is done with K, dQ still to come
                    clean_tile<D>(smem_u32(sm.ring) + kst * C::TILE, threadIdx.x, kFormers);
                    *sm.odd_flag = 1;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 a = fma2(make_float2(x[2 * i], x[2 * i + 1]), c2, nl);
                    x[2 * i] = exp2_fast(a.x);
                    x[2 * i + 1] = exp2_fast(a.y);
                }
                if (!(ok = warp_wait(&sm.dp_full[blocks & 1u], (blocks >> 1) & 1u, sm.abort_flag,
                                     p.status))) {
                    for (int i = 0; n == 1 && i < 2; ++i) named_bar_sync(1, kFormers);
                    break;
                }
                tc_fence_after();
                float d[32];
                tmem_ld32_async(tp, reinterpret_cast<uint32_t*>(d));
                tmem_wait_ld();
                if (n == 1) {
                    // the first 128 tokens of a sequence: the whole row is
                    // here, so D_i = sum_j P_ij dP_ij without the rounding of
                    // P that O's product carries, which weighs most in short
                    // rows (it falls as 1 / sqrt(row)); the dK, dV kernel
                    // reads it too
                    float part = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) part += c0 + i <= r ? x[i] * d[i] : 0.f;
                    float* sum = sm.rows + (~done & 1u) * 256;   // the idle buffer
                    if (quarter < 2) sum[quarter * 128 + r] = part;
                    named_bar_sync(1, kFormers);
                    if (quarter >= 2) sum[(quarter - 2) * 128 + r] += part;
                    named_bar_sync(1, kFormers);
                    delta = sum[r] + sum[128 + r];
                    if (valid && quarter == 0) p.delta[w.h * p.T + w.start + row] = delta;
                }
                const float2 nd = make_float2(-delta, -delta);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 a = mul2(make_float2(x[2 * i], x[2 * i + 1]),
                                          add2(make_float2(d[2 * i], d[2 * i + 1]), nd));
                    d[2 * i] = a.x;
                    d[2 * i + 1] = a.y;
                }
                if (j == n - 1) {   // the diagonal block; a hidden pair may hold anything
                    const uint32_t hidden = bits_from(r + 1 - c0);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (hidden >> i & 1u) d[i] = 0.f;
                }
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
                tmem_st16(tp, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ds_full[blocks & 1u]);
            }
            ok = ok && warp_wait(sm.acc_full, done & 1u, sm.abort_flag, p.status);
            ++done;
            if (ok) {
                tc_fence_after();
                uint4 v[4];
                if (c0 < D) take_rows(tmQ + lane_off, c0, p.scale, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.acc_empty);
                if (c0 < D)
                    store_quad(v, p.dq + (w.start + row0) * p.dq_t + w.h * p.dq_h, p.dq_t,
                               w.len - row0, c0, p.D);
                __syncwarp();   // a row's pieces come from four lanes
                if (*sm.odd_flag) dq_visible(p, w.start, w.len, row0, w.h, w.kvh, c0);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

template <int D, int PARTS>
int launch_dkv(const BwdParams& p, int64_t items, cudaStream_t st) {
    const auto kern = attn_dkv_kernel<D, PARTS>;
    const int smem = DkvCfg<D>::SMEM;
    if (ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return MOE_ECUDA;
    if (items * PARTS >= (1ll << 31)) return MOE_EINVAL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items * PARTS), 1, 1);
    cfg.blockDim = dim3(kBwdThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PARTS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_dkv");
    return MOE_OK;
}

// CTAs that share a block of keys.  The first keys of a sequence meet every
// query block of the group's heads, so one CTA would run 2 / (T / 128 + 1) of
// a head's work alone, against 1 / SMs of all the work for an even share.
// Measured with 1, 2 and 4 CTAs a block, 16/4 heads: 8192 tokens in four sequences
// 141, 148, 197 us, in one 336, 320, 371; 4096 in four 74, 51, 76, in one 166,
// 94, 119; 1024 in one 49, 33, 25; 8/1 heads, 1024 in four 51, 33, 25.  The host
// knows the tokens, not the sequences (they stay on the device): 8192 tokens get
// one CTA a block, right for four sequences and 5 % too slow for one.
int dkv_parts(int64_t T, int group, int n_kv_heads, int sms) {
    const int64_t blocks = (T + 127) / 128;
    const double share = 2.0 * sms / (static_cast<double>(n_kv_heads) * (blocks + 1));
    int parts = share > 4.0 ? 4 : share > 1.5 ? 2 : 1;
    while (parts > 1 && group * blocks < 4 * parts) parts /= 2;   // too few to share
    return parts;
}

template <int D>
int launch_pair(BwdParams& p, const AttnPlanLayout& l, const uint8_t* plan, int n_heads,
                int n_kv_heads, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    const int smem = DqCfg<D>::SMEM;
    if (ensure_smem_attr(reinterpret_cast<const void*>(attn_dq_kernel<D>), smem)) return MOE_ECUDA;
    const int64_t items = l.max128 * n_heads;
    if (items >= (1ll << 31) - 1024) return MOE_EINVAL;
    p.list = 0;
    p.tiles = reinterpret_cast<const int4*>(plan + l.q128);
    p.units = n_heads;
    attn_dq_kernel<D><<<static_cast<int>(items < sms ? items : sms), kBwdThreads, smem, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_dq");
    p.list = 1;
    p.tiles = reinterpret_cast<const int4*>(plan + l.kv128);
    p.units = n_kv_heads;
    const int parts = dkv_parts(p.T, p.group, n_kv_heads, sms);
    const int64_t kv_items = l.max128 * n_kv_heads;
    return parts == 4   ? launch_dkv<D, 4>(p, kv_items, st)
           : parts == 2 ? launch_dkv<D, 2>(p, kv_items, st)
                        : launch_dkv<D, 1>(p, kv_items, st);
}

}  // namespace

int check_status_attention_bwd() { return moe_check_read_reset(); }

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
    p.out = out;
    p.rest = rest;
    p.o_t = a.o_t;
    p.o_h = a.o_h;
    p.lse = lse;
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
