// router_select.cu -- the choice of a token's experts from its router logits, and the
// gradient of its weights.
//
// Scores s are sigmoid(l) or softmax(l); the choice goes by v = s + bias: the groups of
// experts with the largest value (the sum of their one or two largest v) are kept, and of
// their experts the k with the largest v.  The order is that of the exact real values,
// equal ones by the lower index; the weights are s / sum(s) or s, times a factor.
//
// A warp takes a token.  The lanes are split evenly over the groups, so that a group's
// value is a matter of its own lanes.  Scores are computed in fp32 together with a bound
// of their error; where the bound leaves a comparison that matters open (about one token
// in a thousand), the token is done again in 64 bits.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

struct SelectParams {
    int64_t T;
    int E, k, groups, kept, per, lanes;   // per: experts a group, lanes: of a warp a group
    int softmax, top2, renorm;
    float scale;
    const float *logits, *bias;
    int32_t* idx;
    float* w;
};

// The order of v as an unsigned key: a larger value, a larger key (-0 as +0); 0 is below
// every key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Two largest of (a1 >= a2) and (b1 >= b2).
template <typename F>
__device__ __forceinline__ void merge2(F& a1, F& a2, F b1, F b2) {
    if (b1 > a1) {
        a2 = a1 > b2 ? a1 : b2;
        a1 = b1;
    } else if (b1 > a2) {
        a2 = b1;
    }
}

// The choice in 64 bits; lane j < k returns the j-th expert.
template <int PER>
__device__ __noinline__ int choose64(const SelectParams& p, int64_t t) {
    const int lane = threadIdx.x & 31, grp = lane / p.lanes, sub = lane - grp * p.lanes;
    const float* row = p.logits + t * p.E;
    double v[PER];
    uint32_t open = 0;   // entries that may still be chosen
    double m = -INFINITY;
    for (int i = 0; i < PER; ++i) {
        const int in = sub + p.lanes * i;
        v[i] = -INFINITY;
        if (grp < p.groups && in < p.per) {
            open |= 1u << i;
            v[i] = row[grp * p.per + in];
            m = fmax(m, v[i]);
        }
    }
    double sum = 0;
    if (p.softmax) {
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
        for (int i = 0; i < PER; ++i)
            if (open >> i & 1) sum += exp(v[i] - m);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    double b1 = -INFINITY, b2 = -INFINITY;
    for (int i = 0; i < PER; ++i) {
        if (!(open >> i & 1)) continue;
        const double s = p.softmax ? exp(v[i] - m) / sum : 1 / (1 + exp(-v[i]));
        const double x = p.bias ? s + p.bias[grp * p.per + sub + p.lanes * i] : s;
        v[i] = x != x ? -INFINITY : x;
        merge2(b1, b2, v[i], static_cast<double>(-INFINITY));
    }
    if (p.kept < p.groups) {
        for (int o = 1; o < p.lanes; o <<= 1)
            merge2(b1, b2, __shfl_xor_sync(kAll, b1, o), __shfl_xor_sync(kAll, b2, o));
        double value = p.top2 ? b1 + b2 : b1;
        if (value != value) value = -INFINITY;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double other = __shfl_sync(kAll, value, g * p.lanes);
            rank += other > value || (other == value && g < grp);
        }
        if (rank >= p.kept) open = 0;
    }
    int mine = 0;
    for (int j = 0; j < p.k; ++j) {
        double best = -INFINITY;
        int e = 0x7fffffff;
        for (int i = 0; i < PER; ++i) {
            const int ei = grp * p.per + sub + p.lanes * i;
            if ((open >> i & 1) && (v[i] > best || (v[i] == best && ei < e))) {
                best = v[i];
                e = ei;
            }
        }
        const int own = e;
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, best, o);
            const int oe = __shfl_xor_sync(kAll, e, o);
            if (ov > best || (ov == best && oe < e)) {
                best = ov;
                e = oe;
            }
        }
        if (lane == j) mine = e;
        if (own == e) open &= ~(1u << ((e - grp * p.per) / p.lanes));
    }
    return mine;
}

// Relative error of a fast score: 2^-20 for a sigmoid and 2^-18 for a softmax (the fast
// exponential, the division or the sum over the row), and the rounding of the exponent's
// argument; the sum with the bias rounds once more.  What underflows is below 1e-36.
__device__ __forceinline__ float score_error(float s, float arg, float v, bool softmax) {
    const float rel = (softmax ? 3.8147e-6f : 9.5368e-7f) + fabsf(arg) * 1.1921e-7f;
    return fmaf(s, rel, fmaf(fabsf(v), 1.1921e-7f, 1e-36f));
}

__device__ __forceinline__ float fast_score(float l, float m, float inv, bool softmax) {
    return softmax ? __expf(l - m) * inv : __fdividef(1.0f, 1.0f + __expf(-l));
}

template <int PER>
__global__ void __launch_bounds__(kThreads) router_select_kernel(const SelectParams p) {
    const int lane = threadIdx.x & 31, grp = lane / p.lanes, sub = lane - grp * p.lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const float* row = p.logits + t * p.E;
    const int first = grp * p.per + sub;                     // this lane's first expert
    const int count = grp < p.groups && sub < p.per ? (p.per - sub + p.lanes - 1) / p.lanes : 0;
    if (!moe_check(count <= PER && first + (count - 1) * p.lanes < p.E, 1611)) return;
    const bool sm = p.softmax != 0, by_groups = p.kept < p.groups;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < count ? __ldg(row + first + p.lanes * i) : -INFINITY;
    // a row of one value (padding) leaves the choice to the bias, and needs no score
    const float l0 = __shfl_sync(kAll, v[0], 0);
    bool same = true;
#pragma unroll
    for (int i = 0; i < PER; ++i) same = same && (i >= count || v[i] == l0);
    same = __all_sync(kAll, same);
    float m = 0.0f, inv = 1.0f;
    if (sm && (p.bias || by_groups || !p.renorm)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = fmaxf(m, v[i]);
        m = warp_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += i < count ? __expf(v[i] - m) : 0.0f;
        inv = 1.0f / warp_sum(sum);
    }
    // Without a bias the logits' own order is the scores'; a group's two largest scores
    // add up all the same.
    const bool exact = !p.bias || same;
    bool open_question = false;
    float b1 = -INFINITY, b2 = -INFINITY, worst = 0.0f;   // two largest; the largest error
    if (p.bias || (by_groups && p.top2)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i >= count) continue;
            const float l = v[i], s = same ? 0.0f : fast_score(l, m, inv, sm);
            float x = p.bias ? s + __ldg(p.bias + first + p.lanes * i) : s;
            x = x != x ? -INFINITY : x;
            if (by_groups) {
                if (!same) worst = fmaxf(worst, score_error(s, sm ? l - m : l, x, sm));
                merge2(b1, b2, x, -INFINITY);
            }
            v[i] = p.bias ? x : l != l ? -INFINITY : l;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = v[i] != v[i] ? -INFINITY : v[i];
            b1 = fmaxf(b1, v[i]);
        }
    }
    bool keep = grp < p.groups;
    if (by_groups) {
        for (int o = 1; o < p.lanes; o <<= 1) {
            merge2(b1, b2, __shfl_xor_sync(kAll, b1, o), __shfl_xor_sync(kAll, b2, o));
            worst = fmaxf(worst, __shfl_xor_sync(kAll, worst, o));
        }
        float value = p.top2 ? b1 + b2 : b1;
        value = value != value ? -INFINITY : value;
        // whichever experts the value comes from, no error in the group is larger
        const float err = p.top2 ? fmaf(2.0f, worst, fabsf(value) * 1.1921e-7f) : worst;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl_sync(kAll, value, g * p.lanes);
            rank += other > value || (other == value && g < grp);
        }
        keep = keep && rank < p.kept;
        if (__any_sync(kAll, err > 0.0f)) {
            // the lowest that a kept group may be, the highest that another may
            const uint32_t low = __reduce_min_sync(
                kAll, keep ? order_key(value - err) : 0xffffffffu);
            const uint32_t high = __reduce_max_sync(
                kAll, !keep && grp < p.groups ? order_key(value + err) : 0u);
            open_question = low <= high;
        }
    }
    // Rounds of selection: each lane's two first entries in routing order, the largest key
    // over the warp, the lowest expert that holds it.
    uint32_t hk = 0, sk = 0, used = 0;
    int hi = -1, si = -1;
    if (keep) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i < count) {
                const uint32_t key = order_key(v[i]);
                if (key > hk) {
                    sk = hk; si = hi;
                    hk = key; hi = i;
                } else if (key > sk) {
                    sk = key; si = i;
                }
            }
        }
    }
    int mine = 0, next = -1;   // lane j holds the j-th expert; the one behind the last
    const int there = p.kept * p.per;
    const int rounds = p.k < there ? p.k + 1 : p.k;
    for (int rd = 0; rd < rounds; ++rd) {
        const uint32_t top = __reduce_max_sync(kAll, hk);
        const int he = first + p.lanes * hi;
        const uint32_t e = __reduce_min_sync(kAll, hi >= 0 && hk == top ? static_cast<uint32_t>(he) : 0xffffffffu);
        if (rd == p.k) {
            next = static_cast<int>(e);
        } else if (lane == rd) {
            mine = static_cast<int>(e);
        }
        if (hi >= 0 && static_cast<uint32_t>(he) == e) {
            used |= 1u << hi;
            if (si >= 0) {
                hk = sk; hi = si;
                sk = 0; si = -1;
            } else {
                hk = 0; hi = -1;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (i < count && !(used >> i & 1u)) {
                        const uint32_t key = order_key(v[i]);
                        if (key > hk) {
                            hk = key; hi = i;
                        }
                    }
                }
            }
        }
    }
    if (!moe_check(lane >= p.k || (mine >= 0 && mine < p.E), 1612)) mine = 0;
    float l = lane < p.k ? __ldg(row + mine) : 0.0f;
    if (!exact) {
        // neighbours in the order whose bounds meet
        auto bounds = [&](int e, float le, float& x, float& err) {
            const float s = fast_score(le, m, inv, sm);
            x = s + __ldg(p.bias + e);
            err = score_error(s, sm ? le - m : le, x, sm);
            x = x != x ? -INFINITY : x;
        };
        float x = 0.0f, err = 0.0f, nx = 0.0f, nerr = 0.0f;
        if (lane < p.k) bounds(mine, l, x, err);
        if (next >= 0) bounds(next, __ldg(row + next), nx, nerr);
        float ox = __shfl_down_sync(kAll, x, 1), oerr = __shfl_down_sync(kAll, err, 1);
        if (lane == p.k - 1) {
            ox = nx;
            oerr = nerr;
        }
        const bool pair = lane < p.k - 1 || (lane == p.k - 1 && next >= 0);
        open_question |= __any_sync(kAll, pair && !(x - ox > err + oerr));
    }
    if (open_question) {
        mine = choose64<PER>(p, t);
        l = lane < p.k ? __ldg(row + mine) : 0.0f;
    }
    float s;
    if (sm && p.renorm) {   // the softmax of the chosen
        const float top = warp_max(lane < p.k ? l : -INFINITY);
        s = lane < p.k ? expf(l - top) : 0.0f;
    } else if (sm) {
        s = expf(l - m) * inv;
    } else {
        s = lane < p.k ? 1.0f / (1.0f + expf(-l)) : 0.0f;
    }
    if (p.renorm) {
        const float sum = warp_sum(s);
        s = sum == 0.0f ? 0.0f : s / sum;
    }
    if (lane < p.k) {
        p.idx[t * p.k + lane] = mine;
        p.w[t * p.k + lane] = s * p.scale;
    }
}

// ------------------------------------------------------------------ gradient

struct SelectBwdParams {
    int64_t T;
    int E, k, softmax, renorm;
    float scale;
    const float *logits, *dw;
    const int32_t* idx;
    void* dlogits;
};

__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(uint16_t* o, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *o = *reinterpret_cast<const uint16_t*>(&b);
}

// A warp a token: its row is put together in shared memory, and the block's rows, which
// stand side by side in memory, are written as one run of 16-byte pieces.
template <typename Out>
__global__ void __launch_bounds__(kThreads) router_select_bwd_kernel(const SelectBwdParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Out* rows = reinterpret_cast<Out*>(smem);
    constexpr int W = kThreads / 32;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * W, t = t0 + wid;
    if (t < p.T) {
        Out* mine = rows + static_cast<int64_t>(wid) * p.E;
        const float* row = p.logits + t * p.E;
        int e = -1;
        float g = 0.0f, l = -INFINITY;
        if (lane < p.k) {
            e = p.idx[t * p.k + lane];
            if (e < 0 || e >= p.E) e = -1;
            if (e >= 0) {
                g = p.dw[t * p.k + lane] * p.scale;
                l = __ldg(row + e);
            }
        }
        float d;   // gradient of the lane's chosen logit
        if (p.softmax && !p.renorm) {
            float m = -INFINITY, sum = 0.0f;
            for (int i = lane; i < p.E; i += 32) m = fmaxf(m, __ldg(row + i));
            m = warp_max(m);
            for (int i = lane; i < p.E; i += 32) sum += __expf(__ldg(row + i) - m);
            const float inv = 1.0f / warp_sum(sum);
            const float s = e >= 0 ? expf(l - m) * inv : 0.0f;
            const float all = warp_sum(e >= 0 ? g * s : 0.0f);
            for (int i = lane; i < p.E; i += 32) put(mine + i, -(expf(__ldg(row + i) - m) * inv) * all);
            d = s * (g - all);
        } else {
            for (int i = lane; i < p.E; i += 32) put(mine + i, 0.0f);
            float s, gate = 1.0f;   // ds/dl = s gate
            if (p.softmax) {
                const float top = warp_max(l);
                s = e >= 0 ? expf(l - top) : 0.0f;
            } else {
                const float x = expf(-l);
                s = e >= 0 ? 1.0f / (1.0f + x) : 0.0f;
                gate = x > 3e38f ? 1.0f : x / (1.0f + x);   // 1 - s, without the difference
            }
            if (p.renorm) {
                const float sum = warp_sum(s);
                const float n = sum == 0.0f ? 0.0f : s / sum;
                d = n * gate * (g - warp_sum(e >= 0 ? g * n : 0.0f));
            } else {
                d = s * gate * g;
            }
        }
        __syncwarp();
        if (e >= 0) put(mine + e, d);
    }
    __syncthreads();
    const int64_t n = (p.T - t0 < W ? p.T - t0 : W) * p.E * static_cast<int64_t>(sizeof(Out));
    uint8_t* to = static_cast<uint8_t*>(p.dlogits) + t0 * p.E * static_cast<int64_t>(sizeof(Out));
    const int full = static_cast<int>(n / 16);
    for (int i = threadIdx.x; i < full; i += kThreads)
        reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(smem)[i];
    for (int i = full * 16 / static_cast<int>(sizeof(Out)) + threadIdx.x;
         i < static_cast<int>(n / static_cast<int64_t>(sizeof(Out))); i += kThreads)
        reinterpret_cast<Out*>(to)[i] = rows[i];
}

}  // namespace

int check_status_router_select() { return moe_check_read_reset(); }

int router_select_lanes(int groups) {
    int pow2 = 1;
    while (pow2 < groups) pow2 *= 2;
    return 32 / pow2;
}

int launch_router_select(const moe_routing_t& c, const float* logits, const float* bias,
                         int32_t* idx, float* w, cudaStream_t st) {
    SelectParams p;
    p.T = c.T;
    p.E = c.n_experts;
    p.k = c.top_k;
    p.groups = c.groups_kept < c.n_groups ? c.n_groups : 1;
    p.kept = c.groups_kept < c.n_groups ? c.groups_kept : 1;
    p.per = p.E / p.groups;
    p.lanes = router_select_lanes(p.groups);
    p.softmax = c.score == 0;
    p.top2 = c.group_top == 2;
    p.renorm = c.renorm;
    p.scale = c.scale;
    p.logits = logits;
    p.bias = bias;
    p.idx = idx;
    p.w = w;
    const int64_t grid = (c.T + kThreads / 32 - 1) / (kThreads / 32);
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    const int need = (p.per + p.lanes - 1) / p.lanes;
    void (*kern)(SelectParams) = need <= 2    ? router_select_kernel<2>
                                 : need <= 4  ? router_select_kernel<4>
                                 : need <= 8  ? router_select_kernel<8>
                                 : need <= 12 ? router_select_kernel<12>
                                 : need <= 16 ? router_select_kernel<16>
                                              : router_select_kernel<32>;
    kern<<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "router_select");
    return MOE_OK;
}

int launch_router_select_backward(const moe_routing_t& c, const float* logits, const int32_t* idx,
                                  const float* dw, void* dlogits, cudaStream_t st) {
    SelectBwdParams p;
    p.T = c.T;
    p.E = c.n_experts;
    p.k = c.top_k;
    p.softmax = c.score == 0;
    p.renorm = c.renorm;
    p.scale = c.scale;
    p.logits = logits;
    p.dw = dw;
    p.idx = idx;
    p.dlogits = dlogits;
    const int64_t grid = (c.T + kThreads / 32 - 1) / (kThreads / 32);
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    const int bytes = kThreads / 32 * p.E * (c.grad_f32 ? 4 : 2);   // at most 32 KB
    if (c.grad_f32)
        router_select_bwd_kernel<float><<<static_cast<unsigned>(grid), kThreads, bytes, st>>>(p);
    else
        router_select_bwd_kernel<uint16_t><<<static_cast<unsigned>(grid), kThreads, bytes, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "router_select_bwd");
    return MOE_OK;
}

}  // namespace moe
