// head_norm_rotary.cu -- norm of every query and key head and its rotation to the
// token's position in one pass, and the gradient of both.
//
// Forward, a head row x of D channels:  r = (mean(x^2) + eps)^-1/2, y = R(pos) (w x r).
// Backward, with dn = R^T dy and u = w dn:
//     dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of dn x r
// so one look at x and dy gives both means, and nothing of the forward is kept.
//
// A head row is a group of G lanes, each with 16 channels: both chunks of 8 that a
// rotation pairs, or 16 channels behind the rotated ones, so that turning a pair and both
// means stay within a lane and log2 G exchanges.  The grid fills the machine once; a group
// walks over items (a token and a share of its heads) with a few rows under way that each
// lane copies for itself (no barrier).  The forward folds weights and angles of an item
// into four factors a pair, and steps pointers from row to row.
//   Forward, 16384 x (48 + 8) x 128: 77 us, floor 69; 8192 x (16 + 4) x 128: 17.4 us, floor
// 12.4: some 180 instructions a warp's four rows, of which the 16 warps of an SM issue 45 %
// of the time, the start, and uneven shares (24576 items of 8, 8 and 4 heads over 9728 groups
// give 5120 of them 20 rows, 1536 16 and the others 12, where 16.8 is even).  Items of all their rows
// in registers without a ring took 20.6 and 92, rows of weights and angles not folded 21.5
// and 80.
//   Backward, 65536 x (48 + 8) x 128: 444 us, floor 415, 6.3 TB/s: memory.  8192 x (16 + 4):
// 31.8, floor 18.5: the same shares, here CTA by CTA, so that whole CTAs have 20 or 12 rows a
// group.  The forward's stepped pointers would spill here (492 and 34).
#include "common.cuh"
#include "early.cuh"
#include "head_split.h"
#include "internal.h"

namespace moe {

namespace {

struct Rows {   // heads of a tensor: elements between tokens and heads
    const uint16_t* base;
    int64_t t, h;
};

struct HeadParams {
    int64_t T, table_rows;
    int hq, hk, D, units, rot_units, half;   // units: 16-channel pieces of a head
    int q_splits, k_splits;                  // parts of a token's query heads, key heads
    int q_each, k_each;                      // heads of a part, the last one's fewer (forward)
    int64_t q_items, items;                  // tokens times parts: the query heads', all
    Rows x_q, x_k, dy_q, dy_k, y_q, y_k;     // inputs, upstream gradients, outputs
    const uint16_t *w_q, *w_k;
    const float* table;
    const int32_t* pos;
    float* part;
    int32_t* status;
    float eps, inv_d;
};

constexpr int kThreads = 256;
constexpr int kBlocks = 2;     // resident on an SM
constexpr int kStages = 4;     // head rows that a lane of the gradient has under way
constexpr int kAhead = 3;      // and of the forward

// Where this lane's two chunks of 8 channels stand in a head: half the rotated width
// apart, or half of the rest, so that neighbouring lanes read neighbouring chunks whichever
// channels make a pair.
struct Place {
    int c0, c1;
    bool rot, one, two;   // rotated; the first chunk exists; the second does
    __device__ Place(const HeadParams& p, int u) {
        rot = u < p.rot_units;
        const int rest = p.units - p.rot_units;
        c0 = rot ? 8 * u : 2 * p.half + 8 * (u - p.rot_units);
        c1 = c0 + (rot ? p.half : 8 * rest);
        one = u < p.units;
        two = one && c1 < p.D;
    }
};

// 16 channels of a lane as pairs of floats: f[0..3] the first chunk, f[4..7] the second.
__device__ __forceinline__ void unpack(const uint4& a, const uint4& b, float2 (&f)[8]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = bf16x2_f32(w[i]);
}

__device__ __forceinline__ uint4 pack4(const float2* f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                      pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}

// Turns the 8 pairs of a lane's 16 channels by the angles {c, s}.
template <bool PAIRS>
__device__ __forceinline__ void turn(float2 (&f)[8], const float2 (&c)[4], const float2 (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PAIRS) {   // words 2 i and 2 i + 1 are pairs 2 i and 2 i + 1
            const float2 u = f[2 * i], v = f[2 * i + 1];
            f[2 * i] = make_float2(fmaf(-u.y, s[i].x, u.x * c[i].x), fmaf(u.x, s[i].x, u.y * c[i].x));
            f[2 * i + 1] = make_float2(fmaf(-v.y, s[i].y, v.x * c[i].y), fmaf(v.x, s[i].y, v.y * c[i].y));
        } else {       // words i and i + 4 hold pairs 2 i and 2 i + 1
            const float2 u = f[i], v = f[i + 4], uc = mul2(u, c[i]);
            f[i] = make_float2(fmaf(-v.x, s[i].x, uc.x), fmaf(-v.y, s[i].y, uc.y));
            f[i + 4] = fma2(u, s[i], mul2(v, c[i]));
        }
    }
}

// A lane's angles of 8 pairs in four vectors of two: the pairs' order is that of the first
// chunk's words and then the second's where pairs are neighbours, else of the chunks' channels.
template <bool PAIRS>
__device__ __forceinline__ const float* angle(const HeadParams& p, int64_t pos, int u, int e) {
    const int pair = PAIRS ? 4 * u + 2 * (e & 1) + (e >> 1) * (p.half / 2) : 8 * u + 2 * e;
    return p.table + (pos * p.half + pair) * 2;
}

// The angles that turn back.
template <bool PAIRS>
__device__ __forceinline__ void load_angles(const HeadParams& p, int64_t pos, int u, float2 (&c)[4],
                                            float2 (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(angle<PAIRS>(p, pos, u, e));
        c[e] = make_float2(v.x, v.z);
        s[e] = make_float2(-v.y, -v.w);
    }
}

// The steps of a group of lanes: items (a token and some of its query heads, behind all
// of those a token and some of its key heads) in strides over the grid, head by head.
struct Walk {
    int64_t item, t;
    int h;
    bool keys, first;   // the step is its item's first
    __device__ __forceinline__ bool more(const HeadParams& p) const { return item < p.items; }
    __device__ __forceinline__ void enter(const HeadParams& p) {
        keys = item >= p.q_items;
        const int splits = keys ? p.k_splits : p.q_splits;
        const int64_t i = keys ? item - p.q_items : item;
        if (splits == 1) {
            t = i;
            h = 0;
        } else if (p.items < (1ll << 31)) {   // a 32-bit division where it does
            const uint32_t q = static_cast<uint32_t>(i) / static_cast<uint32_t>(splits);
            t = q;
            h = static_cast<int>(static_cast<uint32_t>(i) - q * splits);
        } else {
            t = i / splits;
            h = static_cast<int>(i - t * splits);
        }
        first = true;
    }
    __device__ __forceinline__ void next(const HeadParams& p, int64_t stride) {
        h += keys ? p.k_splits : p.q_splits;
        first = false;
        if (h >= (keys ? p.hk : p.hq)) {
            item += stride;
            if (more(p)) enter(p);
        }
    }
    __device__ __forceinline__ const uint16_t* row(const Rows& q, const Rows& k) const {
        const Rows& r = keys ? k : q;
        return r.base + t * r.t + h * r.h;
    }
};

// Each lane copies the chunks of x and dy that it will read itself, so that a stage needs
// no barrier.
struct Ring {
    static constexpr int kSlots = 4;
    uint4* mine;   // slot k of stage s: mine[(s * kSlots + k) * kThreads]
    __device__ __forceinline__ uint4* at(int stage, int k) const { return mine + (stage * kSlots + k) * kThreads; }

    // Starts the copies of a step.  Chunks that a head does not have stay as they are (zero).
    __device__ __forceinline__ void issue(const HeadParams& p, const Place& pl, const Walk& w, int stage) const {
        const uint16_t *x = w.row(p.x_q, p.x_k), *dy = w.row(p.dy_q, p.dy_k);
        if (pl.one) cp_async_16(smem_u32(at(stage, 0)), x + pl.c0, 16);
        if (pl.two) cp_async_16(smem_u32(at(stage, 1)), x + pl.c1, 16);
        if (pl.one) cp_async_16(smem_u32(at(stage, 2)), dy + pl.c0, 16);
        if (pl.two) cp_async_16(smem_u32(at(stage, 3)), dy + pl.c1, 16);
    }
};

__device__ __forceinline__ void load_weights(const uint16_t* w, int c0, int c1, bool one, bool two,
                                             float2 (&f)[8]) {
    const uint4 none = make_uint4(0, 0, 0, 0);
    unpack(one ? *reinterpret_cast<const uint4*>(w + c0) : none,
           two ? *reinterpret_cast<const uint4*>(w + c1) : none, f);
}

// One pass over the heads: the gradients, and the block's part of dw.
template <bool PAIRS, int G>
__global__ void __launch_bounds__(kThreads, kBlocks) head_norm_bwd_kernel(const __grid_constant__ HeadParams p) {
    extern __shared__ __align__(16) uint4 smem[];
    wait_earlier();
    const int lane = threadIdx.x & 31, u = lane & (G - 1), group = threadIdx.x / G;
    const unsigned mask = (G == 32 ? 0xffffffffu : ((1u << G) - 1u)) << (lane & ~(G - 1));
    const Place pl(p, u);
    if (!moe_check((!pl.one || pl.c0 + 8 <= p.D) && (!pl.two || pl.c1 + 8 <= p.D), 1601)) return;
    const Ring ring{smem + threadIdx.x};
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / G);
    Walk in, at;   // what is copied next, what is worked on
    in.item = at.item = static_cast<int64_t>(blockIdx.x) * (kThreads / G) + group;
    auto fill = [&](int stage) {
        if (in.more(p)) {
            ring.issue(p, pl, in, stage);
            in.next(p, stride);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i)   // chunks that a head does not have
#pragma unroll
        for (int k = 0; k < Ring::kSlots; ++k)
            if (!(k & 1 ? pl.two : pl.one)) *ring.at(i, k) = make_uint4(0, 0, 0, 0);
    float2 w[8], c[4], s[4], dw[8];
    if (in.more(p)) {
        in.enter(p);
        at.enter(p);
        load_weights(at.keys ? p.w_k : p.w_q, pl.c0, pl.c1, pl.one, pl.two, w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = make_float2(0.0f, 0.0f);
    // the group's part of dw_q and dw_k, behind the ring
    float2* red = reinterpret_cast<float2*>(smem + kStages * Ring::kSlots * kThreads) + threadIdx.x;
    const bool only_keys = at.more(p) && at.keys;
    bool mine = only_keys, gone = false;
#pragma unroll
    for (int i = 0; i < kStages; ++i) fill(i);
    for (int stage = 0; at.more(p); stage = stage + 1 == kStages ? 0 : stage + 1) {
        cp_async_wait<kStages - 1>();
        if (at.keys != mine) {   // the first key heads
            load_weights(p.w_k, pl.c0, pl.c1, pl.one, pl.two, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                red[i * kThreads] = dw[i];
                dw[i] = make_float2(0.0f, 0.0f);
            }
            mine = true;
        }
        if (at.first && p.table) {
            const int64_t pos = p.pos ? p.pos[at.t] : at.t;
            gone = pos < 0 || pos >= p.table_rows;
            if (gone)
                report_error(p.status, MOE_EINVAL);
            else if (pl.rot)
                load_angles<PAIRS>(p, pos, u, c, s);
        }
        float2 f[8], ss = make_float2(0.0f, 0.0f);
        unpack(*ring.at(stage, 0), *ring.at(stage, 1), f);
        uint16_t* o = const_cast<uint16_t*>(at.row(p.y_q, p.y_k));
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma2(f[i], f[i], ss);
        float sum = ss.x + ss.y;
        float2 d[8], dot = make_float2(0.0f, 0.0f);
        unpack(*ring.at(stage, 2), *ring.at(stage, 3), d);
        if (pl.rot) turn<PAIRS>(d, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fma2(mul2(w[i], d[i]), f[i], dot);
        float along = dot.x + dot.y;
#pragma unroll
        for (int q = G / 2; q > 0; q >>= 1) {
            sum += __shfl_xor_sync(mask, sum, q);
            along += __shfl_xor_sync(mask, along, q);
        }
        const float r = rsqrtf(fmaf(sum, p.inv_d, p.eps)), back = -along * p.inv_d * r * r;
        const float2 r2 = make_float2(r, r), back2 = make_float2(back, back);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!gone) dw[i] = fma2(d[i], mul2(f[i], r2), dw[i]);
            f[i] = mul2(fma2(f[i], back2, mul2(w[i], d[i])), r2);
        }
        if (pl.one && !gone) *reinterpret_cast<uint4*>(o + pl.c0) = pack4(f);
        if (pl.two && !gone) *reinterpret_cast<uint4*>(o + pl.c1) = pack4(f + 4);
        fill(stage);
        at.next(p, stride);
    }
    cp_async_wait<0>();
    const int other = 8 * kThreads;
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // a group that has met no key heads adds nothing to them
        red[(mine ? other : 0) + i * kThreads] = dw[i];
        if (!mine) red[other + i * kThreads] = make_float2(0.0f, 0.0f);
    }
    if (only_keys) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[i * kThreads] = make_float2(0.0f, 0.0f);
    }
    __syncthreads();
    // the block's sums, its groups in their order
    const float2* all = reinterpret_cast<const float2*>(smem + kStages * Ring::kSlots * kThreads);
    for (int e = threadIdx.x; e < 2 * p.units * 8; e += kThreads) {
        const int kind = e / (p.units * 8), unit = e / 8 % p.units, i = e % 8;
        if (kind == 1 && !p.hk) break;
        const Place q(p, unit);
        if (i >= 4 && !q.two) continue;
        float2 sum = make_float2(0.0f, 0.0f);
        for (int g = 0; g < kThreads / G; ++g) sum = add2(sum, all[kind * other + i * kThreads + g * G + unit]);
        const int ch = i < 4 ? q.c0 + 2 * i : q.c1 + 2 * (i - 4);
        *reinterpret_cast<float2*>(p.part + (static_cast<int64_t>(blockIdx.x) * 2 + kind) * p.D + ch) = sum;
    }
}

// What a lane does with its 16 channels x1, x2 (pairs of pairs): r (a x1 + b x2) and
// r (c x1 + d x2), weights and angles in one.
struct Coefs {
    float2 a[4], b[4], c[4], d[4];
};

// 16 channels as the first and the second of 8 pairs, two pairs to a float2.
template <bool PAIRS>
__device__ __forceinline__ void split(const uint4& p, const uint4& q, float2 (&x1)[4], float2 (&x2)[4]) {
    const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PAIRS) {
            x1[i] = make_float2(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
            x2[i] = make_float2(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
        } else {
            x1[i] = bf16x2_f32(w[i]);
            x2[i] = bf16x2_f32(w[i + 4]);
        }
    }
}

template <bool PAIRS>
__device__ __forceinline__ void join(const float2 (&y1)[4], const float2 (&y2)[4], uint4* p, uint4* q) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PAIRS) {
            w[2 * i] = pack_bf16x2(y1[i].x, y2[i].x);
            w[2 * i + 1] = pack_bf16x2(y1[i].y, y2[i].y);
        } else {
            w[i] = pack_bf16x2(y1[i].x, y1[i].y);
            w[i + 4] = pack_bf16x2(y2[i].x, y2[i].y);
        }
    }
    *p = make_uint4(w[0], w[1], w[2], w[3]);
    *q = make_uint4(w[4], w[5], w[6], w[7]);
}

// A group's item: a run of a token's query heads, behind all of those a run of its key
// heads.  The lane's first chunk of the run's first head, the elements between heads, the
// heads left.
struct Run {
    int64_t item, step;
    const uint16_t* x;
    int left;
    int64_t pos;   // asked for a row ahead of its use
    template <bool OUT>
    __device__ __forceinline__ void enter(const HeadParams& p, int c0) {
        const bool keys = item >= p.q_items;
        const int splits = keys ? p.k_splits : p.q_splits, each = keys ? p.k_each : p.q_each;
        const int64_t i = keys ? item - p.q_items : item;
        int part = 0;
        int64_t t = i;
        if (splits > 1) {
            if (p.items < (1ll << 31)) {   // a 32-bit division where it does
                const uint32_t q = static_cast<uint32_t>(i) / static_cast<uint32_t>(splits);
                t = q;
                part = static_cast<int>(static_cast<uint32_t>(i) - q * splits);
            } else {
                t = i / splits;
                part = static_cast<int>(i - t * splits);
            }
        }
        int h = part * each, n = (keys ? p.hk : p.hq) - h;
        if (!moe_check(n > 0, 1603)) {   // the walk ends where left comes to zero
            h = 0;
            n = 1;
        }
        const Rows& r = OUT ? (keys ? p.y_k : p.y_q) : (keys ? p.x_k : p.x_q);
        left = n < each ? n : each;
        step = r.h;
        x = r.base + t * r.t + h * r.h + c0;
        if (!OUT && p.table) pos = p.pos ? p.pos[t] : t;
    }
};

// One pass over the heads: the norms, turned.  Each lane copies the chunks, and with an
// item's first row the angles, that it will read itself.
template <bool PAIRS, int G>
__global__ void __launch_bounds__(kThreads, kBlocks) head_norm_fwd_kernel(const __grid_constant__ HeadParams p) {
    extern __shared__ __align__(16) uint4 smem[];
    wait_earlier();
    constexpr int N = kThreads, kSlots = 6;
    const int lane = threadIdx.x & 31, u = lane & (G - 1);
    const unsigned mask = (G == 32 ? 0xffffffffu : ((1u << G) - 1u)) << (lane & ~(G - 1));
    const Place pl(p, u);
    if (!moe_check((!pl.one || pl.c0 + 8 <= p.D) && (!pl.two || pl.c1 + 8 <= p.D), 1602)) return;
    const int apart = pl.c1 - pl.c0;
    uint4* const mine = smem + threadIdx.x;   // slot k of stage s: mine[(s * kSlots + k) * N]
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (N / G);
    Run in, at;   // what is copied next, what is worked on
    // a warp's groups side by side, the CTAs' warps in turn: the last items go to all CTAs
    in.item = at.item = (static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * (32 / G) + lane / G;
    if (in.item >= p.items) return;
    in.enter<false>(p, pl.c0);
    at.enter<true>(p, pl.c0);
    bool fresh = true, more = true;   // what is copied next begins an item; there is something
    uint32_t skip = 0;                // bit s: stage s begins an item without a place
    auto fill = [&](int stage) {
        if (more) {
            uint4* to = mine + stage * (kSlots * N);
            if (pl.one) cp_async_16(smem_u32(to), in.x, 16);
            if (pl.two) cp_async_16(smem_u32(to + N), in.x + apart, 16);
            if (fresh && p.table) {
                const int64_t pos = in.pos;
                skip &= ~(1u << stage);
                if (pos < 0 || pos >= p.table_rows) {
                    report_error(p.status, MOE_EINVAL);
                    skip |= 1u << stage;
                } else if (pl.rot) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) cp_async_16(smem_u32(to + (2 + e) * N), angle<PAIRS>(p, pos, u, e), 16);
                }
            }
            in.x += in.step;
            fresh = --in.left == 0;
            if (fresh) {
                in.item += stride;
                more = in.item < p.items;
                if (more) in.enter<false>(p, pl.c0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)   // chunks that a head does not have
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (!(k ? pl.two : pl.one)) mine[(i * kSlots + k) * N] = make_uint4(0, 0, 0, 0);
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 wa, wb;
    auto weights = [&](bool keys) {
        const uint16_t* w = keys ? p.w_k : p.w_q;
        wa = pl.one ? *reinterpret_cast<const uint4*>(w + pl.c0) : none;
        wb = pl.two ? *reinterpret_cast<const uint4*>(w + pl.c1) : none;
    };
    bool keys = at.item >= p.q_items, gone = false;
    weights(keys);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fill(i);
    Coefs k;
    bool first = true;
    for (int stage = 0;; stage = stage + 1 == kAhead ? 0 : stage + 1) {
        cp_async_wait<kAhead - 1>();
        const uint4* from = mine + stage * (kSlots * N);
        if (first) {
            gone = skip >> stage & 1;
            float2 w1[4], w2[4];
            split<PAIRS>(wa, wb, w1, w2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (pl.rot) {
                    const float4 v = *reinterpret_cast<const float4*>(from + (2 + e) * N);
                    const float2 c = make_float2(v.x, v.z), s = make_float2(v.y, v.w);
                    k.a[e] = mul2(w1[e], c);
                    k.b[e] = mul2(w2[e], make_float2(-s.x, -s.y));
                    k.c[e] = mul2(w1[e], s);
                    k.d[e] = mul2(w2[e], c);
                } else {
                    k.a[e] = w1[e];
                    k.d[e] = w2[e];
                }
            }
        }
        float2 x1[4], x2[4], ss = make_float2(0.0f, 0.0f);
        split<PAIRS>(from[0], from[N], x1, x2);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(x1[i], x1[i], fma2(x2[i], x2[i], ss));
        float sum = ss.x + ss.y;
#pragma unroll
        for (int q = G / 2; q > 0; q >>= 1) sum += __shfl_xor_sync(mask, sum, q);
        const float r = rsqrtf(fmaf(sum, p.inv_d, p.eps));
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z1 = mul2(x1[i], r2), z2 = mul2(x2[i], r2);
            if (pl.rot) {
                x1[i] = fma2(z1, k.a[i], mul2(z2, k.b[i]));
                x2[i] = fma2(z1, k.c[i], mul2(z2, k.d[i]));
            } else {
                x1[i] = mul2(z1, k.a[i]);
                x2[i] = mul2(z2, k.d[i]);
            }
        }
        uint4 ya, yb;
        join<PAIRS>(x1, x2, &ya, &yb);
        uint16_t* o = const_cast<uint16_t*>(at.x);
        if (pl.one && !gone) *reinterpret_cast<uint4*>(o) = ya;
        if (pl.two && !gone) *reinterpret_cast<uint4*>(o + apart) = yb;
        fill(stage);
        at.x += at.step;
        first = --at.left == 0;
        if (first) {
            at.item += stride;
            if (at.item >= p.items) return;
            at.enter<true>(p, pl.c0);
            if (!keys && at.item >= p.q_items) {
                keys = true;
                weights(true);
            }
        }
    }
}

template <bool PAIRS, int G>
int begin_forward(const HeadParams& p, int sms, cudaStream_t st) {
    constexpr int kBytes = kAhead * 6 * kThreads * 16;
    const auto kern = head_norm_fwd_kernel<PAIRS, G>;
    if (const int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), kBytes)) return rc;
    const int64_t need = (p.items * G + kThreads - 1) / kThreads, most = static_cast<int64_t>(sms) * kBlocks;
    return launch_early(kern, need < most ? need : most, kThreads, kBytes, st, p);
}

int begin_forward_any(const HeadParams& p, bool pairs, int lanes, int sms, cudaStream_t st) {
    switch (lanes) {
        case 4: return pairs ? begin_forward<true, 4>(p, sms, st) : begin_forward<false, 4>(p, sms, st);
        case 8: return pairs ? begin_forward<true, 8>(p, sms, st) : begin_forward<false, 8>(p, sms, st);
        case 16: return pairs ? begin_forward<true, 16>(p, sms, st) : begin_forward<false, 16>(p, sms, st);
        default: return pairs ? begin_forward<true, 32>(p, sms, st) : begin_forward<false, 32>(p, sms, st);
    }
}

// dw_q, dw_k: the blocks' sums, 32 runs of blocks side by side and then their 32 sums.
__global__ void __launch_bounds__(1024) head_norm_sums_kernel(const float* part, int blocks, int D,
                                                              float* dw_q, float* dw_k) {
    __shared__ float red[32][33];
    wait_earlier();   // the partials are complete
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    const bool there = c < (dw_k ? 2 : 1) * D;
    if (there)
        for (int b = run; b < blocks; b += 32) s += __ldcg(part + static_cast<int64_t>(b) * 2 * D + c);   // past L1, as it started early
    red[run][lane] = s;
    __syncthreads();
    if (run == 0 && there) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        if (c < D)
            dw_q[c] = s;
        else
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
    p.eps = c.eps;
    p.inv_d = 1.0f / static_cast<float>(c.D);
    return p;
}

int lanes_of(int units) { return units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32; }

void set_items(HeadParams* p) {
    p->q_items = p->T * p->q_splits;
    p->items = p->q_items + p->T * p->k_splits;
}

// The parts of a token's heads: of each kind every q_splits-th, k_splits-th head (the
// gradient).
void head_strides(HeadParams* p, int lanes, int sms) {
    const HeadParts parts = head_parts(p->T, p->hq, p->hk, lanes, static_cast<int64_t>(sms) * kBlocks * kThreads);
    p->q_splits = parts.q;
    p->k_splits = parts.k;
    set_items(p);
}

// Runs of neighbours (the forward).
void head_neighbours(HeadParams* p, int lanes, int sms) {
    const HeadParts parts = head_parts(p->T, p->hq, p->hk, lanes, static_cast<int64_t>(sms) * kBlocks * kThreads);
    const HeadRuns q = head_runs(p->hq, parts.q), k = head_runs(p->hk, parts.k);
    p->q_splits = q.runs;
    p->q_each = q.each;
    p->k_splits = k.runs;
    p->k_each = k.each;
    set_items(p);
}

constexpr int kMaxParts = kBlocks * 160;   // blocks of a backward launch, on a device of 160 SMs at most

template <bool PAIRS, int G>
int begin_backward(const HeadParams& p, int sms, int* grid, cudaStream_t st) {
    constexpr int kBytes = kStages * Ring::kSlots * kThreads * 16 + kThreads * 128;
    const auto kern = head_norm_bwd_kernel<PAIRS, G>;
    if (const int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), kBytes)) return rc;
    const int64_t need = (p.items * G + kThreads - 1) / kThreads;
    int64_t most = static_cast<int64_t>(sms) * kBlocks;
    if (most > kMaxParts) most = kMaxParts;
    *grid = static_cast<int>(need < most ? need : most);
    return launch_early(kern, *grid, kThreads, kBytes, st, p);
}

int begin_backward_any(const HeadParams& p, bool pairs, int lanes, int sms, int* grid, cudaStream_t st) {
    switch (lanes) {
        case 4: return pairs ? begin_backward<true, 4>(p, sms, grid, st) : begin_backward<false, 4>(p, sms, grid, st);
        case 8: return pairs ? begin_backward<true, 8>(p, sms, grid, st) : begin_backward<false, 8>(p, sms, grid, st);
        case 16: return pairs ? begin_backward<true, 16>(p, sms, grid, st) : begin_backward<false, 16>(p, sms, grid, st);
        default: return pairs ? begin_backward<true, 32>(p, sms, grid, st) : begin_backward<false, 32>(p, sms, grid, st);
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
    p.x_q = {q, c.q_t, c.q_h};
    p.x_k = {k, c.k_t, c.k_h};
    p.y_q = {q_out, c.qo_t, c.qo_h};
    p.y_k = {k_out, c.ko_t, c.ko_h};
    p.w_q = w_q;
    p.w_k = w_k;
    p.table = c.rot_dim ? table : nullptr;
    p.pos = pos;
    p.status = status;
    const int lanes = lanes_of(p.units);
    head_neighbours(&p, lanes, sms);
    if (const int rc = begin_forward_any(p, c.interleaved, lanes, sms, st)) return rc;
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
    p.x_q = {q, c.q_t, c.q_h};
    p.x_k = {k, c.k_t, c.k_h};
    p.dy_q = {dq, c.dq_t, c.dq_h};
    p.dy_k = {dk, c.dk_t, c.dk_h};
    p.y_q = {dq_out, c.qo_t, c.qo_h};
    p.y_k = {dk_out, c.ko_t, c.ko_h};
    p.w_q = w_q;
    p.w_k = w_k;
    p.table = c.rot_dim ? table : nullptr;
    p.pos = pos;
    p.part = static_cast<float*>(ws);
    p.status = status;
    const int lanes = lanes_of(p.units);
    head_strides(&p, lanes, sms);
    int grid = 0;
    if (const int rc = begin_backward_any(p, c.interleaved, lanes, sms, &grid, st)) return rc;
    trace_after(st, "head_norm_rotary_bwd");
    if (const int rc = launch_early(head_norm_sums_kernel, (2 * c.D + 31) / 32, 1024, 0, st, p.part,
                                    grid, c.D, dw_q, dw_k))
        return rc;
    trace_after(st, "head_norm_rotary_sums");
    return MOE_OK;
}

}  // namespace moe
