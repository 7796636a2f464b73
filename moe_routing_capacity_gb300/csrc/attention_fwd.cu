// attention_fwd.cu -- causal attention over packed sequences, forward, and
// the plan of work lists that forward and backward share.
//
// One CTA an SM works through the batch, heaviest work first.  A piece of
// work is two tiles of 128 query rows that read the same key/value head of
// the same sequence (two query heads of a group, or two blocks of rows when
// the group is odd), over the sequence's key blocks of 128:
//   S = Q K^T (tcgen05, fp32 in TMEM); m, l = running maximum and sum;
//   P = 2^(c S - c m) as bf16 back into S's columns; O += P V (A from TMEM).
// Warps 0-3 and 4-7 run the softmax of the two tiles, a thread a row, so that
// no two threads have to meet (two threads a row took 491 us where this takes
// 479); warp 8 issues the MMAs, warp 9 the TMA loads, warp 10 looks at V where
// keys are hidden.  While one tile's softmax runs, the tensor cores work on the
// other's products.  TMEM: two S and two O of 128 columns, all 512.
//   16384 tokens in 7 sequences, 48/8 heads of 128 (0.69 TFLOP): 498 us, 1.39
// PFLOP/s (a library product reaches 1.88), 487 without the look at V.  32768
// tokens in one sequence, 8/2 heads: 1.28 ms, 1.72 PFLOP/s.  Ten calls each; run for
// seconds, both meet the power limit (530 us, 1.38 ms).  Heads of 96, 80 and 64 at
// the first size: 492, 490, 438 us.
// What bounds it: S waits for the product that reads P from
// its columns, so a tile's softmax (about 1500 cycles) and its products (1024)
// follow each other and two tiles do not quite fill the tensor cores; beside
// that Q and K from shared memory take its whole bandwidth while S is formed,
// and a piece of work starts and ends with 4000 cycles without products.
// (A MMA warp for each tile: 701 us, products of two issuers interleave; softmax
// loops rolled over halves of the keys, to be shorter: 507 us.)
#include <cstring>

#include "attention.cuh"
#include "internal.h"

namespace moe {

namespace {

struct FwdParams {
    CUtensorMap mapQ, mapK, mapV;   // {head_dim, T, heads}, box {64, 128, 1}
    const int4* tiles;
    const int32_t* header;
    int list;                        // which header word counts the tiles
    int units;                       // CTAs of one tile
    int pair_heads;                  // 1: tiles are two heads; 0: two row blocks
    int group;
    int D;
    int64_t T;
    int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    const uint16_t *q, *k, *v;
    uint16_t *out, *rest;
    float* lse;
    float scale, scale_log2;
    int32_t* status;
};

// Warps 0-3 and 4-7 the softmax of the two tiles, a thread a row; then the MMA
// warp, the load warp, the value warp (diagonal blocks of V), an idle one.
constexpr int kFwdThreads = 384, kFwdMmaWarp = 8, kFwdLoadWarp = 9, kFwdValueWarp = 10;

template <int D>
struct FwdCfg {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int SMEM = 2 * TILE + STAGES * TILE + 320;
};

// Adds to the warp's rows [row0, row0 + 32) of out what of the values from key
// `from` on, which were set to 0 for the product, they see: infinities and NaN,
// whose weights are above 0.  Four channels a lane; a row whose lse is not finite
// is NaN throughout.
__device__ __noinline__ void fwd_visible(const FwdParams& p, int64_t start, int len, int from,
                                         int row0, int h, int kvh, float lse) {
    const int lane = threadIdx.x & 31, c = 4 * lane;
    const bool in = c < p.D;
    const uint16_t* v = p.v + start * p.v_t + kvh * p.v_h + c;
    float sum[4] = {0, 0, 0, 0};   // of what is not finite among the keys so far
    for (int j = from; j < min(row0 + 32, len); ++j) {
        const uint2 w = in ? *reinterpret_cast<const uint2*>(v + j * p.v_t) : make_uint2(0, 0);
        const uint32_t x[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (bf16_odd(x[e])) sum[e] += bf16_f32(static_cast<uint16_t>(x[e]));
        const float l = __shfl_sync(0xFFFFFFFFu, lse, j & 31);
        if (j < row0 || !(l - l == 0.f)) continue;
        const int64_t o = (start + j) * p.o_t + h * p.o_h + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (sum[e] != 0.f) {
                p.out[o + e] = f32_bf16(bf16_f32(p.out[o + e]) + sum[e]);
                if (p.rest) p.rest[o + e] = 0x7FFF;
            }
    }
}

// One piece of work: two tiles of query rows over one key/value head.
struct FwdWork {
    int64_t start;
    int len, kvh, block;
    int h[2], m0[2], n[2];   // query head, first row, key blocks (0: no tile)
    __device__ FwdWork(const FwdParams& p, int item) {
        const int tile = item / p.units, u = item - tile * p.units;
        const int4 te = p.tiles[tile];
        start = te.x;
        len = te.y;
        block = te.z;
        if (p.pair_heads) {
            const int half = p.group / 2;
            kvh = u / half;
            h[0] = kvh * p.group + 2 * (u - kvh * half);
            h[1] = h[0] + 1;
            m0[0] = m0[1] = block * 128;
        } else {
            h[0] = h[1] = u;
            kvh = u / p.group;
            m0[0] = block * 256;
            m0[1] = m0[0] + 128;
        }
        n[0] = m0[0] / 128 + 1;
        n[1] = m0[1] < len ? m0[1] / 128 + 1 : 0;
    }
    // key block j holds a tile's diagonal
    __device__ bool diagonal(int j) const { return j == n[0] - 1 || j == n[1] - 1; }
};

// f(work) for each of this CTA's items; false ends the walk.
template <class F>
__device__ __forceinline__ void each_item(const FwdParams& p, F f) {
    AttnItems items(p.header[p.list] * p.units);
    int item;
    while (items.next(item, p.tiles, p.units, p.T, p.pair_heads ? 128 : 256, 1203))
        if (!f(FwdWork(p, item))) return;
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdParams p) {
    using C = FwdCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_u32(smem_raw) & 1023u) {   // the swizzled tiles' alignment
        report_error(p.status, MOE_ECUDA);
        return;
    }
    report_refused(p.header, p.status);
    uint8_t* sQ = smem_raw;
    uint8_t* sKV = sQ + 2 * C::TILE;
    uint64_t* full = reinterpret_cast<uint64_t*>(sKV + C::STAGES * C::TILE);
    uint64_t* empty = full + C::STAGES;
    uint64_t* q_full = empty + C::STAGES;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;   // [2] scores of a tile ready
    uint64_t* p_full = s_full + 2;    // [2][2] a half of its P written
    uint64_t* o_full = p_full + 4;    // [2] its product with V done
    uint64_t* o_empty = o_full + 2;   // [2] its O read by the epilogue
    uint64_t* done = o_empty + 2;
    uint64_t* v_full = done + 1;      // [STAGES] a diagonal block's V, before the value warp
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_full + C::STAGES);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* odd_flag = abort_flag + 1;   // a value that is not finite was met

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&v_full[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[2 * t], 4);   // one arrival a warp
            mbar_init(&p_full[2 * t + 1], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&o_empty[t], 4);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        *odd_flag = 0;
        fence_mbar_init();
    }
    if (warp == kFwdMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;
    const uint32_t tmS = tm, tmO = tm + 256;   // tile t: + 128 t

    if (warp >= kFwdMmaWarp) {
        setmaxnreg_dec<64>();
        if (warp == kFwdLoadWarp && lane == 0) {
            // -------------------------------------------------------- loads
            tma_prefetch_map(&p.mapQ);
            tma_prefetch_map(&p.mapK);
            tma_prefetch_map(&p.mapV);
            const uint32_t aq = smem_u32(sQ), akv = smem_u32(sKV);
            uint32_t st = 0, ph = 0, armed = 0, par = 0, items = 0;
            uint32_t via = 0, v_ph = 0;   // stages filled for the value warp; its phases
            bool ok = true;
            each_item(p, [&](const FwdWork& w) {
                if (w.block < 0) return true;
                const int tiles = w.n[1] ? 2 : 1, blocks = max(w.n[0], w.n[1]);
                const int tok = static_cast<int>(w.start);
                if (items && !(ok = mbar_wait(q_empty, (items - 1) & 1u, abort_flag, p.status)))
                    return false;
                ++items;
                mbar_arrive_expect_tx(q_full, tiles * C::TILE);
                for (int t = 0; t < tiles; ++t)
                    for (int b = 0; b < D / 64; ++b)
                        tma_load_3d(aq + t * C::TILE + b * kBoxBytes, &p.mapQ, q_full, b * 64,
                                    tok + w.m0[t], w.h[t]);
                for (int it = 0; it < 2 * blocks; ++it) {
                    if (!(ok = mbar_wait(&empty[st], ph ^ 1u, abort_flag, p.status))) return false;
                    const bool v = (it & 1) && w.diagonal(it >> 1);
                    uint64_t* landed = v ? &v_full[st] : &full[st];
                    mbar_arrive_expect_tx(landed, C::TILE);
                    armed |= 1u << st;
                    par = (par & ~(1u << st)) | ((v ? v_ph >> st & 1u : ph) << st);
                    via = (via & ~(1u << st)) | (static_cast<uint32_t>(v) << st);
                    if (v) v_ph ^= 1u << st;
                    for (int b = 0; b < D / 64; ++b)
                        tma_load_3d(akv + st * C::TILE + b * kBoxBytes,
                                    (it & 1) ? &p.mapV : &p.mapK, landed, b * 64,
                                    tok + (it >> 1) * 128, w.kvh);
                    if (++st == C::STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                return true;
            });
            if (!ok || *abort_flag) {   // let the armed copies land before leaving
                volatile int no_abort = 0;
                if (items) mbar_wait(q_full, (items - 1) & 1u, &no_abort, nullptr, 20000000ull);
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait(via >> s & 1u ? &v_full[s] : &full[s], (par >> s) & 1u, &no_abort,
                                  nullptr, 20000000ull);
            }
        } else if (warp == kFwdValueWarp) {
            // -------------------------------------------------------- diagonal blocks of V
            const uint32_t akv = smem_u32(sKV);
            uint32_t st = 0, v_ph = 0;
            each_item(p, [&](const FwdWork& w) {
                if (w.block < 0) return true;
                for (int it = 0; it < 2 * max(w.n[0], w.n[1]); ++it) {
                    if ((it & 1) && w.diagonal(it >> 1)) {
                        if (!warp_wait(&v_full[st], v_ph >> st & 1u, abort_flag, p.status))
                            return false;
                        v_ph ^= 1u << st;
                        if (odd_tile<D>(akv + st * C::TILE, lane, 32)) {
                            clean_tile<D>(akv + st * C::TILE, lane, 32);
                            *odd_flag = 1;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[st]);
                    }
                    if (++st == C::STAGES) st = 0;
                }
                return true;
            });
        } else if (warp == kFwdMmaWarp) {
            // -------------------------------------------------------- MMAs
            const uint32_t one = elect_lane();
            const uint32_t aq = smem_u32(sQ), akv = smem_u32(sKV);
            uint32_t st = 0, ph = 0;        // next tile of the ring
            uint32_t items = 0, ps[2] = {0, 0}, tiles[2] = {0, 0};
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = warp_wait_short(bar, parity, abort_flag, p.status);
                tc_fence_after();
                return got;
            };
            const auto next = [&] {         // its stage, once it has landed; then the one after
                const uint32_t s = st;
                if (!wait(&full[st], ph)) return ~0u;
                if (++st == C::STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
                return s;
            };
            each_item(p, [&](const FwdWork& w) {
                if (w.block < 0) return true;
                const int blocks = max(w.n[0], w.n[1]);
                if (!wait(q_full, items++ & 1u)) return false;
                uint32_t sk = next();
                if (sk == ~0u) return false;
                for (int t = 0; t < 2; ++t)
                    if (w.n[t]) {
                        mma_scores<D>(one, tmS + 128 * t, desc_k(aq + t * C::TILE),
                                      desc_k(akv + sk * C::TILE));
                        commit(one, &s_full[t]);
                    }
                commit(one, &empty[sk]);
                if (blocks == 1) commit(one, q_empty);
                for (int j = 0; j < blocks; ++j) {
                    const uint32_t sv = next();
                    if (sv == ~0u) return false;
                    const uint64_t dv = desc_mn(akv + sv * C::TILE);
                    bool have_k = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j >= w.n[t]) continue;
                        const uint32_t dS = tmS + 128 * t, dO = tmO + 128 * t;
                        // the last item's O has been read
                        if (j == 0 && tiles[t]++ && !wait(&o_empty[t], (tiles[t] - 2) & 1u))
                            return false;
                        if (!wait(&p_full[2 * t], ps[t] & 1u)) return false;
                        mma_tokens<D>(one, dO, dS, dv, 0, j > 0);
                        if (!wait(&p_full[2 * t + 1], ps[t]++ & 1u)) return false;
                        mma_tokens<D>(one, dO, dS, dv, 1, true);
                        commit(one, &o_full[t]);
                        if (j + 1 < w.n[t]) {
                            if (!have_k && (sk = next()) == ~0u) return false;
                            have_k = true;
                            // runs after the product above has read P from these columns
                            mma_scores<D>(one, dS, desc_k(aq + t * C::TILE),
                                          desc_k(akv + sk * C::TILE));
                            commit(one, &s_full[t]);
                        }
                    }
                    commit(one, &empty[sv]);
                    if (have_k) commit(one, &empty[sk]);
                    if (j == blocks - 2) commit(one, q_empty);   // its last scores are issued
                }
                return true;
            });
            // nothing of this CTA is in flight when it leaves
            commit(one, done);
            volatile int no_abort = 0;
            mbar_wait(done, 0, &no_abort, p.status);
        }
    } else {
        setmaxnreg_inc<216>();
        // ------------------------------------------------------------ softmax
        // a thread: row r of tile t
        const int t = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmS + 128 * t + lane_off, to = tmO + 128 * t + lane_off;
        const float c = p.scale_log2;
        const float slack = 8.0f / c;   // P may reach 2^8 before O is rescaled
        uint32_t blocks = 0;            // key blocks of this tile so far
        bool ok = true;
        each_item(p, [&](const FwdWork& w) {
            const int h = t ? w.h[1] : w.h[0], n = t ? w.n[1] : w.n[0];
            if (w.block < 0) {   // tokens of no sequence
                if (t && !p.pair_heads) return true;
                for (int i = r; i < w.len * (p.D / 8); i += 128) {
                    const int64_t o = (w.start + i / (p.D / 8)) * p.o_t + h * p.o_h + i % (p.D / 8) * 8;
                    *reinterpret_cast<uint4*>(p.out + o) = make_uint4(0, 0, 0, 0);
                    if (p.rest) *reinterpret_cast<uint4*>(p.rest + o) = make_uint4(0, 0, 0, 0);
                }
                for (int i = r; i < w.len; i += 128) p.lse[h * p.T + w.start + i] = -INFINITY;
                return true;
            }
            if (!n) return true;
            // l: sum of P, for lse; lb: sum of P as rounded to bf16, which
            // divides O: a row that is nearly one key's then gives that key's
            // v, not v times its weight's rounding error, and D_i of the
            // backward depends on it
            float m = -INFINITY, l = 0.f, lb = 0.f;
            for (int j = 0; j < n; ++j, ++blocks) {
                if (!(ok = warp_wait(&s_full[t], blocks & 1u, abort_flag, p.status))) return false;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmem_ld32_async(ts + 32 * i, reinterpret_cast<uint32_t*>(s) + 32 * i);
                tmem_wait_ld();
                if (j == n - 1) {   // the diagonal block: keys after the row are hidden
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t hidden = bits_from(r + 1 - 32 * i);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (hidden >> e & 1u) s[32 * i + e] = -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[e] = max3(s[e], s[8 + e], s[16 + e]);
#pragma unroll
                for (int i = 24; i < 120; i += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 8 + e]);
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], s[120 + e]);
                const float top = fmaxf(max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[4]),
                                        max3(mx[5], mx[6], mx[7]));
                // O keeps an older maximum until a row's rises by 2^8: sums in
                // fp32 hold the larger terms, and rescaling is rare
                const bool rise = top > m + slack;
                if (j == 0) {
                    m = top;
                } else if (__any_sync(0xFFFFFFFFu, rise)) {
                    if (!(ok = warp_wait(&o_full[t], (blocks - 1) & 1u, abort_flag, p.status)))
                        return false;
                    const float f = rise ? exp2_fast((m - top) * c) : 1.0f;
                    if (rise) m = top;
                    l *= f;
                    lb *= f;
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * i, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(to + 16 * i, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                // (no key with a weight so far: -inf - -inf would be NaN)
                const float from = m == -INFINITY ? 0.f : -m * c;
                const float2 c2 = make_float2(c, c), neg = make_float2(from, from);
                // half the keys: their product with V runs while the others
                // are formed.  P as bf16: what the tensor cores take beside a
                // bf16 V, with fp32's range; the roundings (2^-8 at most a
                // key) average out over a row's keys
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float* x = s + 64 * half;
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int e = 16 * i; e < 16 * i + 16; ++e) {
                            const float2 v = fma2(make_float2(x[2 * e], x[2 * e + 1]), c2, neg);
                            x[2 * e] = exp2_fast(v.x);
                            x[2 * e + 1] = exp2_fast(v.y);
                            pk[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
                        }
                        tmem_st16(ts + 32 * half + 16 * i, pk + 16 * i);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
                    // the sums, while the products run
                    float2 sum = make_float2(0.f, 0.f), sumb = sum;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        sum = add2(sum, make_float2(x[2 * e], x[2 * e + 1]));
                        sumb = add2(sumb, bf16x2_f32(pk[e]));
                    }
                    l += sum.x + sum.y;
                    lb += sumb.x + sumb.y;
                }
            }
            // ------------------------------------------------------------ output
            if (!(ok = warp_wait(&o_full[t], (blocks - 1) & 1u, abort_flag, p.status))) return false;
            tc_fence_after();
            const int row = (t ? w.m0[1] : w.m0[0]) + r, row0 = row - lane;
            const bool valid = row < w.len;
            const float inv = 1.0f / lb;
            const float lse = m * p.scale + logf(l);
            const int64_t o = (w.start + row0) * p.o_t + h * p.o_h;
            // out, and for the backward what the rounding took: 16 bits of O
            // together, since D from the 8 of out alone is off by as much as dS
            // where a row is nearly one key's
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t a[32];
                tmem_ld32(to + 32 * i, a);
                if (i == D / 32 - 1) {   // O may be overwritten from here on
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_empty[t]);
                }
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = mul2(make_float2(__uint_as_float(a[2 * e]),
                                                      __uint_as_float(a[2 * e + 1])),
                                          make_float2(inv, inv));
                    hi[e] = pack_bf16x2(x.x, x.y);
                    lo[e] = pack_bf16x2(x.x - bf16_lo(hi[e]), x.y - bf16_hi(hi[e]));
                }
                uint4 v[4];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    v[g] = make_uint4(hi[4 * g], hi[4 * g + 1], hi[4 * g + 2], hi[4 * g + 3]);
                store_quad(v, p.out + o, p.o_t, w.len - row0, 32 * i, p.D);
                if (p.rest) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        v[g] = make_uint4(lo[4 * g], lo[4 * g + 1], lo[4 * g + 2], lo[4 * g + 3]);
                    store_quad(v, p.rest + o, p.o_t, w.len - row0, 32 * i, p.D);
                }
            }
            if (valid) p.lse[h * p.T + w.start + row] = lse;
            __syncwarp();    // a row's pieces come from four lanes
            if (*odd_flag)   // (of two row blocks, the second meets the first's diagonal too)
                fwd_visible(p, w.start, w.len, w.m0[0], row0, h, w.kvh, lse);
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kFwdMmaWarp) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ the plan
// Weight w = blocks a query block reads (its number + 1), or that read a key
// block.  Entries with weight >= w of a list of sequences with b_s blocks:
// a counting sort, heaviest first; sequence s has one entry of each weight
// 1 .. b_s in either list.  One CTA, bound by the latency of its loads and
// atomics one behind the other; once a batch.  5 sequences of 301 tokens 6.3 us,
// 7 of 16384 7.7, one of 65536 12, 1024 of 16384 50, 4096 of 262144 185.

__global__ void __launch_bounds__(1024, 1)
    attn_plan_kernel(const int32_t* cu, int n_seqs, int64_t T, int4* q128, int4* kv128, int4* q256,
                     int32_t* header, int32_t* cursor, int bins, int most128, int most256,
                     int32_t* status) {
    __shared__ int part[32];
    __shared__ int carry, bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int s = tid; s <= n_seqs; s += 1024) {
        const int lo = s ? cu[s - 1] : 0;
        if (cu[s] < lo || cu[s] > T) bad = 1;
    }
    __syncthreads();
    if (bad) {
        if (tid < 8) header[tid] = tid == kPlanRefused;
        if (tid == 0) report_error(status, MOE_EINVAL);
        return;
    }
    if (tid == 0) header[kPlanRefused] = 0;
    for (int pass = 0; pass < 2; ++pass) {
        const int bs = pass ? 256 : 128;
        for (int i = tid; i < bins; i += 1024) cursor[i] = 0;
        if (tid == 0) carry = 0;
        __syncthreads();
        for (int s = tid; s < n_seqs; s += 1024) {
            const int nb = (cu[s + 1] - cu[s] + bs - 1) / bs;
            if (nb) atomicAdd(&cursor[nb], 1);
        }
        __syncthreads();
        // sequences with at least w blocks (a suffix sum), then the first
        // entry of weight w: the entries heavier than w
        for (int what = 0; what < 2; ++what) {
            if (tid == 0) carry = 0;
            __syncthreads();
            for (int base = bins - 1; base >= 0; base -= 1024) {
                const int w = base - tid;
                const int v = w >= 0 ? cursor[w] : 0;
                int x = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) part[warp] = x;
                __syncthreads();
                if (warp == 0) {
                    int y = part[lane];
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int z = __shfl_up_sync(0xFFFFFFFFu, y, o);
                        if (lane >= o) y += z;
                    }
                    part[lane] = y;
                }
                __syncthreads();
                const int incl = carry + x + (warp ? part[warp - 1] : 0);
                if (w >= 0) cursor[w] = what ? incl - v : incl;
                __syncthreads();
                if (tid == 1023) carry = incl;
                __syncthreads();
            }
            if (what == 0) {
                if (tid == 0) cursor[0] = 0;   // no entry has weight 0
                __syncthreads();
            }
        }
        const int total = carry;
        for (int s = warp; s < n_seqs; s += 32) {
            const int first = cu[s], len = cu[s + 1] - first, nb = (len + bs - 1) / bs;
            for (int w = lane + 1; w <= nb; w += 32) {
                const int at = atomicAdd(&cursor[w], 1);
                if (!moe_check(at >= 0 && at < (pass ? most256 : most128), 1201)) continue;
                if (pass) {
                    q256[at] = make_int4(first, len, w - 1, 0);
                } else {
                    q128[at] = make_int4(first, len, w - 1, 0);
                    kv128[at] = make_int4(first, len, nb - w, 0);
                }
            }
        }
        // tokens outside every sequence, in blocks
        const int head = cu[0], tail = static_cast<int>(T) - cu[n_seqs];
        const int nh = (head + bs - 1) / bs, nt = (tail + bs - 1) / bs;
        for (int i = tid; i < nh + nt; i += 1024) {
            const int in = i < nh ? i : i - nh;
            const int first = (i < nh ? 0 : cu[n_seqs]) + in * bs;
            const int len = min(bs, (i < nh ? head : static_cast<int>(T)) - first);
            const int4 e = make_int4(first, len, -1, 0);
            if (!moe_check(total + i < (pass ? most256 : most128), 1202)) continue;
            if (pass) {
                q256[total + i] = e;
            } else {
                q128[total + i] = e;
                kv128[total + i] = e;
            }
        }
        if (tid == 0) {
            if (pass) {
                header[2] = total + nh + nt;
            } else {
                header[0] = header[1] = total + nh + nt;
            }
        }
        __syncthreads();
    }
}

}  // namespace

int check_status_attention_fwd() { return moe_check_read_reset(); }

int64_t attention_plan_bytes(int64_t T, int n_seqs) { return attn_plan_layout(T, n_seqs).total; }

int launch_attention_plan(int64_t T, int n_seqs, const int32_t* cu, void* plan, int32_t* status,
                          cudaStream_t st) {
    const AttnPlanLayout l = attn_plan_layout(T, n_seqs);
    uint8_t* b = static_cast<uint8_t*>(plan);
    attn_plan_kernel<<<1, 1024, 0, st>>>(
        cu, n_seqs, T, reinterpret_cast<int4*>(b + l.q128), reinterpret_cast<int4*>(b + l.kv128),
        reinterpret_cast<int4*>(b + l.q256), reinterpret_cast<int32_t*>(b),
        reinterpret_cast<int32_t*>(b + l.cursor), static_cast<int>(l.bins),
        static_cast<int>(l.max128), static_cast<int>(l.max256), status);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_plan");
    return MOE_OK;
}

// {channels, tokens, heads} of a strided tensor in boxes of 64 x 128 x 1
// with the 128-byte swizzle; channels past D and tokens past T read as zero.
int attn_tensor_map(CUtensorMap* m, const void* base, int D, int64_t T, int heads, int64_t st_t,
                    int64_t st_h) {
    // an extent of one has no stride of its own: any valid one will do
    if (T == 1) st_t = D;
    if (heads == 1) st_h = D;
    return tensor_map_bf16_3d(m, base, D, T, heads, st_t, st_h, 128);
}

int launch_attention_fwd(const moe_attention_t& a, const void* plan, const uint16_t* q,
                         const uint16_t* k, const uint16_t* v, uint16_t* out, uint16_t* rest,
                         float* lse, int32_t* status, cudaStream_t st) {
    FwdParams p;
    memset(&p, 0, sizeof(p));
    const int D = a.head_dim;
    if (attn_tensor_map(&p.mapQ, q, D, a.T, a.n_heads, a.q_t, a.q_h) ||
        attn_tensor_map(&p.mapK, k, D, a.T, a.n_kv_heads, a.k_t, a.k_h) ||
        attn_tensor_map(&p.mapV, v, D, a.T, a.n_kv_heads, a.v_t, a.v_h))
        return MOE_ECUDA;
    const AttnPlanLayout l = attn_plan_layout(a.T, a.n_seqs);
    const uint8_t* b = static_cast<const uint8_t*>(plan);
    p.group = a.n_heads / a.n_kv_heads;
    // Two heads of an even group read the same keys in the same blocks; of an odd
    // group, two blocks of rows, of which the second meets a block more.  Rows
    // instead of heads at 48/8 heads: 516 us against 493 (16384 tokens), at 16/4
    // 86 against 84 (8192 tokens), 14.3 against 16.4 (301 tokens).
    p.pair_heads = p.group % 2 == 0;
    p.header = reinterpret_cast<const int32_t*>(b);
    p.list = p.pair_heads ? 0 : 2;
    p.tiles = reinterpret_cast<const int4*>(b + (p.pair_heads ? l.q128 : l.q256));
    p.units = p.pair_heads ? a.n_heads / 2 : a.n_heads;
    p.D = D;
    p.T = a.T;
    p.q_t = a.q_t;
    p.q_h = a.q_h;
    p.k_t = a.k_t;
    p.k_h = a.k_h;
    p.v_t = a.v_t;
    p.v_h = a.v_h;
    p.o_t = a.o_t;
    p.o_h = a.o_h;
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.rest = rest;
    p.lse = lse;
    p.scale = a.scale;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = status;
    // one CTA an SM, or fewer where the batch has less work than that
    const int64_t most = (p.pair_heads ? l.max128 : l.max256) * p.units;
    if (most >= (1ll << 31) - 1024) return MOE_EINVAL;
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    const int grid = static_cast<int>(most < sms ? most : sms);
    if (D <= 64) {
        if (ensure_smem_attr(reinterpret_cast<const void*>(attn_fwd_kernel<64>), FwdCfg<64>::SMEM))
            return MOE_ECUDA;
        attn_fwd_kernel<64><<<grid, kFwdThreads, FwdCfg<64>::SMEM, st>>>(p);
    } else {
        if (ensure_smem_attr(reinterpret_cast<const void*>(attn_fwd_kernel<128>),
                             FwdCfg<128>::SMEM))
            return MOE_ECUDA;
        attn_fwd_kernel<128><<<grid, kFwdThreads, FwdCfg<128>::SMEM, st>>>(p);
    }
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "attn_fwd");
    return MOE_OK;
}

}  // namespace moe
