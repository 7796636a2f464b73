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
// of their error; where the bound leaves a comparison that matters open, the few experts
// that it hangs on are valued in 64 bits, and the whole row where they are many.
//   16384 tokens of 384 experts in 8 groups, 8 chosen, sigmoid with bias: 18.8 us; the
// bytes are 3.9 us; some 1000 instructions a token bound it.  With k rounds of a warp-wide
// maximum it took 70 us.  Without groups and bias 10 us.
//   Gradient, 65536 x 384 in bf16, softmax of the row: 24.4 us, 22.9 of them memory's (the
// logits in, the gradient out); the chosen ones looked up behind the row, 31.5.
#include "common.cuh"
#include "early.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 128;      // 256: 19.2 and 25.8 us in place of 18.9 and 25.1
constexpr int kRowThreads = 256;   // eight rows start on 16 bytes, whatever their length
constexpr float kSmall = -60.0f;   // below it sigmoid(l) is e^l to 2^-86
constexpr float kNone = -709.78f;  // below it 1 / (1 + e^-l) is 0 in 64 bits
constexpr unsigned kAll = 0xffffffffu;

struct SelectParams {
    int64_t T;
    int E, k, groups, kept, per;   // per: experts a group
    int lanes, log_lanes;          // lanes of a warp that share a group
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
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

// A lane's experts: entry i is expert first + of(i) of the group, those with of(i) < room
// are there.  U neighbours at a time, so that U = 4 loads 16 bytes.
template <int U>
struct Entries {
    int first, room, lanes;
    __device__ __forceinline__ Entries(const SelectParams& p, int grp, int sub)
        : first(grp * p.per + U * sub), room(grp < p.groups ? p.per - U * sub : 0), lanes(p.lanes) {}
    __device__ __forceinline__ int of(int i) const { return i / U * U * lanes + i % U; }
    __device__ __forceinline__ bool has(int i) const { return of(i / U * U) < room; }   // in whole U
    __device__ __forceinline__ int expert(int i) const { return first + of(i); }
};

template <int U, int PER>
__device__ __forceinline__ void load(float (&v)[PER], const float* from, const Entries<U>& at) {
#pragma unroll
    for (int i = 0; i < PER; i += U) {
        if constexpr (U == 4) {
            float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at.has(i)) q = *reinterpret_cast<const float4*>(from + at.expert(i));
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        } else {
            v[i] = at.has(i) ? from[at.expert(i)] : -INFINITY;
        }
    }
}

// The order of x (NaN as the smallest) as a signed key.
__device__ __forceinline__ long long order_key64(double x) {
    long long b = __double_as_longlong(x + 0.0);
    if ((b & 0x7fffffffffffffffll) > 0x7ff0000000000000ll) b = 0xfff0000000000000ll;
    return b < 0 ? b ^ 0x7fffffffffffffffll : b;
}

// The choice in 64 bits; lane j < k returns the j-th expert.  A row of one value (padding)
// leaves the choice to the bias.
template <int PER, int U>
__device__ __noinline__ int choose64(const SelectParams& p, int64_t t) {
    const int lane = threadIdx.x & 31, grp = lane >> p.log_lanes, sub = lane & (p.lanes - 1);
    const float* row = p.logits + t * p.E;
    const Entries<U> at(p, grp, sub);
    const float l0 = *row;
    bool same = true, even = true;
    uint32_t open = 0;   // entries that may still be chosen
    float m = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < PER; ++i) {
        if (!at.has(i)) continue;
        open |= 1u << i;
        const float l = row[at.expert(i)];
        same = same && l == l0;
        even = even && (!p.bias || p.bias[at.expert(i)] == *p.bias);
        m = fmaxf(m, l);
    }
    same = __all_sync(kAll, same);
    if (same && __all_sync(kAll, even)) return lane;   // nothing to choose by: the first experts
    m = warp_max(m);
    double sum = 1;
    if (p.softmax && !same) {
        sum = 0;
        for (int i = 0; i < PER; ++i)
            if (open >> i & 1) sum += exp(static_cast<double>(row[at.expert(i)]) - m);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    long long key[PER], k1 = order_key64(-INFINITY), k2 = k1;
    double b1 = -INFINITY, b2 = -INFINITY;
    for (int i = 0; i < PER; ++i) {
        key[i] = 0;
        if (!(open >> i & 1)) continue;
        const double l = row[at.expert(i)];
        double x = same ? 0 : p.softmax ? exp(l - m) / sum : 1 / (1 + exp(-l));
        if (p.bias)
            x += p.bias[at.expert(i)];
        else if (!p.top2 && !same)
            x = l;   // the scores' order, without their rounding: for the groups' largest as well
        key[i] = order_key64(x);
        if (key[i] > k1) {
            k2 = k1; b2 = b1;
            k1 = key[i]; b1 = x;
        } else if (key[i] > k2) {
            k2 = key[i]; b2 = x;
        }
        if (!p.bias && !same) key[i] = order_key64(l);
    }
    if (p.kept < p.groups) {
        for (int o = 1; o < p.lanes; o <<= 1) {
            const double o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            const long long q1 = order_key64(o1), q2 = order_key64(o2);
            if (q1 > k1) {
                if (k1 > q2) {
                    k2 = k1; b2 = b1;
                } else {
                    k2 = q2; b2 = o2;
                }
                k1 = q1; b1 = o1;
            } else if (q1 > k2) {
                k2 = q1; b2 = o1;
            }
        }
        const long long value = order_key64(p.top2 ? b1 + b2 : b1);
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const long long other = __shfl_sync(kAll, value, g << p.log_lanes);
            rank += other > value || (other == value && g < grp);
        }
        if (rank >= p.kept) open = 0;
    }
    int mine = 0;
    for (int j = 0; j < p.k; ++j) {
        long long best = 0;
        int e = 0x7fffffff, which = -1;
        for (int i = 0; i < PER; ++i) {   // experts ascend with i
            if ((open >> i & 1) && (which < 0 || key[i] > best)) {
                best = key[i];
                which = i;
                e = at.expert(i);
            }
        }
        const int own = e;
        for (int o = 16; o > 0; o >>= 1) {
            const long long ob = __shfl_xor_sync(kAll, best, o);
            const int oe = __shfl_xor_sync(kAll, e, o);
            if (oe != 0x7fffffff && (e == 0x7fffffff || ob > best || (ob == best && oe < e))) {
                best = ob;
                e = oe;
            }
        }
        if (lane == j) mine = e;
        if (own == e) open &= ~(1u << which);
    }
    return mine;
}

// The largest logit and the sum of the exponentials of a row, in 64 bits.
template <int PER, int U>
__device__ __noinline__ double row_sum64(const SelectParams& p, int64_t t, float* largest) {
    const int lane = threadIdx.x & 31, grp = lane >> p.log_lanes, sub = lane & (p.lanes - 1);
    const float* row = p.logits + t * p.E;
    const Entries<U> at(p, grp, sub);
    float m = -INFINITY;
    for (int i = 0; i < PER; ++i)
        if (at.has(i)) m = fmaxf(m, row[at.expert(i)]);
    m = warp_max(m);
    double sum = 0;
#pragma unroll 4
    for (int i = 0; i < PER; ++i)
        if (at.has(i)) sum += exp(static_cast<double>(row[at.expert(i)]) - m);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    *largest = m;
    return sum;
}

// What expert e goes by, in 64 bits.
__device__ __noinline__ double value64(const SelectParams& p, int64_t t, int e, float m, double sum) {
    const double l = p.logits[t * p.E + e];
    const double s = p.softmax ? exp(l - m) / sum : 1 / (1 + exp(-l));
    return p.bias ? s + p.bias[e] : s;
}

// The rank of a lane's expert e among n, softmax's with bias, in 64 bits but for the row's
// sum, which is fp32's, off by fewer than 64 steps: a difference of two values is off by that
// part of their scores' difference (*open: one that matters may be).  The sum in 64 bits is 384
// exponentials where this is n (16384 tokens of 384 experts: 25.1 -> 19.2 us).
__device__ __noinline__ int rank_rough(const SelectParams& p, int64_t t, int e, int n, float m, float inv,
                                       const int* list, double* values, double* scores, bool* open) {
    const int lane = threadIdx.x & 31;
    double value = -INFINITY, score = 0;
    if (lane < n) {
        value = value64(p, t, e, m, 1.0 / inv);
        value = value != value ? -INFINITY : value;
        score = value - p.bias[e];
    }
    __syncwarp();
    values[lane] = value;
    scores[lane] = score;
    __syncwarp();
    int rank = 0;
    bool near = false;
    for (int j = 0; j < n; ++j) {
        const double o = values[j], apart = fabs(scores[j] - score);
        rank += o > value || (o == value && list[j] < e);
        // a score is known to 2^-52 of what it was taken from
        near |= !(fabs(o - value) > 0x1p-18 * apart || apart <= 0x1p-50 * fabs(value));
    }
    *open = __any_sync(kAll, lane < n && rank < p.k && near);
    return rank;
}

// The experts of the set bits, one a lane, in list (at most 32; their number).
template <int U>
__device__ __forceinline__ int collect(uint32_t bits, const Entries<U>& at, int* list) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    while (const unsigned who = __ballot_sync(kAll, bits != 0)) {
        const int to = n + __popc(who & ((1u << lane) - 1u));
        if (bits && to < 32) list[to] = at.expert(__ffs(bits) - 1);
        bits &= bits - 1;
        n += __popc(who);
        if (n > 32) break;
    }
    __syncwarp();
    return n;
}

constexpr float kStep = 5.9604645e-8f;   // 2^-24

// Bound of a fast score's error.  arg is the exponential's argument: its product with
// log2(e) is off by 1.5 steps of |arg|, the exponential by 4, the sum and the division by
// 3, the sum of a softmax's row by fewer than 48 (rounded up for both); what underflows is
// below 1e-36.  Of a logit of -infinity, whose score is 0, that alone is left, and not NaN.
__device__ __forceinline__ float score_error(float s, float arg, bool softmax) {
    return fmaf(s, (softmax ? 64.0f : 8.0f) * kStep + 1.5f * kStep * fminf(fabsf(arg), 3e38f), 1e-36f);
}

// 1 / x for 1 <= x, infinity among them, off by a step.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_score(float l, float m, float inv, bool softmax) {
    return softmax ? __expf(l - m) * inv : reciprocal(1.0f + __expf(-l));
}

// Steps: values and each lane's two largest; the groups; a value that k experts reach for
// certain, from the lanes' largest; the few experts that reach it (11 of 384 for k = 8 on average),
// one a lane, whose ranks the lanes count.  Where a step's bounds leave it open, the few
// experts that it hangs on are valued in 64 bits, one a lane; choose64 where they are many.
template <int PER, int U>
__global__ void __launch_bounds__(kThreads) router_select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ int lists[kThreads / 32][32];      // the experts left
    __shared__ __align__(16) double values[kThreads / 32][32];   // their values, in fp32 where that does
    wait_earlier();
    __shared__ float open[kThreads / 32][32 * PER];
    __shared__ double scores[kThreads / 32][32];
    const int lane = threadIdx.x & 31, grp = lane >> p.log_lanes, sub = lane & (p.lanes - 1);
    int* list = lists[threadIdx.x >> 5];
    double* wide = values[threadIdx.x >> 5];
    float* few = reinterpret_cast<float*>(wide);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const float* row = p.logits + t * p.E;
    const Entries<U> at(p, grp, sub);
    const bool sm = p.softmax != 0, by_groups = p.kept < p.groups;
    float v[PER];
    load<U>(v, row, at);
    float m = 0.0f, inv = 1.0f, top = -INFINITY;   // top: the lane's largest logit
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, v[i]);
    if (sm && (p.bias || by_groups || !p.renorm)) {
        m = warp_max(top);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += __expf(v[i] - m);   // no expert: 0
        inv = 1.0f / warp_sum(sum);
    }
    // Without a bias the logits' own order is the scores'; a group's two largest scores
    // add up all the same.
    float b1 = -INFINITY, b2 = -INFINITY;   // the lane's two largest of what the groups go by
    if (p.bias) {
        float b[PER];
        load<U>(b, p.bias, at);
#pragma unroll
        for (int i = 0; i < PER; ++i)   // NaN as the smallest; -infinity where there is no expert
            v[i] = fmaxf(fast_score(v[i], m, inv, sm) + b[i], -INFINITY);
        if (by_groups && p.top2) {
#pragma unroll
            for (int i = 0; i < PER; ++i) merge2(b1, b2, v[i], -INFINITY);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) b1 = fmaxf(b1, v[i]);
        }
    } else if (by_groups && p.top2) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = fmaxf(v[i], -INFINITY);
            merge2(b1, b2, v[i], -INFINITY);
        }
    } else {
        b1 = top;
    }
    bool keep = grp < p.groups, all = false;   // all: the whole row in 64 bits
    const float high = b1;                     // the lane's largest value
    double sum64 = 0;
    if (by_groups) {
        float big = top;
        for (int o = 1; o < p.lanes; o <<= 1) {
            merge2(b1, b2, __shfl_xor_sync(kAll, b1, o), __shfl_xor_sync(kAll, b2, o));
            big = fmaxf(big, __shfl_xor_sync(kAll, big, o));
        }
        const float second = b2;   // without a bias, a logit
        if (!p.bias && p.top2) {
            b1 = fast_score(b1, m, inv, sm);
            b2 = fast_score(b2, m, inv, sm);
        }
        const float value = fmaxf(p.top2 ? b1 + b2 : b1, -INFINITY);
        // s |arg| grows with s where |arg| > 1, so the group's largest score bounds the errors
        // of whichever experts its value comes from
        float err = 0.0f;
        if (p.bias || p.top2) {
            const float arg = sm ? big - m : big;
            err = score_error(fast_score(big, m, inv, sm), fmaxf(1.0f, fabsf(arg)), sm);
            err = p.top2 ? fmaf(fabsf(value) + fabsf(b1) + fabsf(b2), kStep, 2.0f * err)
                         : fmaf(fabsf(value), kStep, err);
        }
        int rank = 0;
        for (int g0 = 0; g0 < p.groups; g0 += p.lanes) {   // a group's lanes share the others
            const int g = g0 + sub;
            const float other = __shfl_sync(kAll, value, (g << p.log_lanes) & 31);
            rank += g < p.groups && (other > value || (other == value && g < grp));
        }
        for (int o = 1; o < p.lanes; o <<= 1) rank += __shfl_xor_sync(kAll, rank, o);
        bool open_question = false;
        if (p.bias || p.top2) {
            // the lowest that a kept group may be, the highest that another may
            const uint32_t low = __reduce_min_sync(kAll, keep && rank < p.kept ? order_key(value - err) : 0xffffffffu);
            const uint32_t over = __reduce_max_sync(kAll, keep && rank >= p.kept ? order_key(value + err) : 0u);
            open_question = !(low > over);
        }
        if (open_question) {
            // the experts that may be among a group's largest
            const float from = p.bias ? (p.top2 ? b2 : b1) - 4.0f * err : second;
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) bits |= at.has(i) && !(v[i] < from) ? 1u << i : 0u;
            const int n = collect<U>(bits, at, list);
            all = n > 32;
            if (!all) {
                if (sm) sum64 = row_sum64<PER, U>(p, t, &m);
                if (lane < n) wide[lane] = value64(p, t, list[lane], m, sum64);
                __syncwarp();
                double w1 = -INFINITY, w2 = -INFINITY;
                for (int j = 0; j < n; ++j) {
                    const double x = wide[j];
                    if (list[j] / p.per != grp) continue;
                    if (x > w1) {
                        w2 = w1;
                        w1 = x;
                    } else if (x > w2) {
                        w2 = x;
                    }
                }
                const double exact = p.top2 ? w1 + w2 : w1;
                rank = 0;
                for (int g = 0; g < p.groups; ++g) {
                    const double other = __shfl_sync(kAll, exact, g << p.log_lanes);
                    rank += other > exact || (!(exact > other) && g < grp);
                }
                __syncwarp();
            }
        }
        keep = keep && rank < p.kept;
    }
    // A value that k experts reach: the k-th largest of the lanes' largest (equal ones go
    // together, which only lowers it).  Of 2 k lanes and more it leaves 1.4 k experts on
    // average; with fewer, or so many that more than 32 may be left, the lanes' largest two
    // decide, which leave 1.1 k (16 of 384 experts, 16384 tokens: 36.0 -> 19.1 us), spread
    // over the warp first where few lanes have experts (7 of 2 of 8 groups of 55, softmax with
    // bias, 26467 tokens: 63.6 -> 49.2 us); and of 25 and more a lane goes on to its next
    // value.
    uint32_t key = keep && at.room > 0 ? order_key(high) : 0u, reach = 0;
    const int some = __popc(__ballot_sync(kAll, key != 0));
    if (2 * p.k <= some && p.k <= 10) {
        for (int j = 0; j < p.k; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, key);
            reach = best ? best : reach;
            key = key == best ? 0u : key;
        }
    } else if (p.k <= 24) {
        float h1 = -INFINITY, h2 = -INFINITY;
        uint32_t next;
        if (4 * p.k <= 3 * some) {
#pragma unroll
            for (int i = 0; i < PER; ++i) merge2(h1, h2, v[i], -INFINITY);
            next = key && at.has(1) ? order_key(h2) : 0u;
        } else {   // the open groups' values over all lanes
            const int slot = __popc(__ballot_sync(kAll, key != 0) & ((1u << lane) - 1u)), n = some * PER;
            float* all_open = open[threadIdx.x >> 5];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key) all_open[i * some + slot] = v[i];
            __syncwarp();
            for (int i = lane; i < n; i += 32) merge2(h1, h2, all_open[i], -INFINITY);
            key = lane < n ? order_key(h1) : 0u;
            next = lane + 32 < n ? order_key(h2) : 0u;
        }
        for (int j = 0; j < p.k; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, key);
            reach = best ? best : reach;
            if (key == best) {
                key = next;
                next = 0u;
            }
        }
    } else {
        for (int j = 0; j < p.k; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, key);
            reach = best ? best : reach;
            if (key != best) continue;
            key = 0u;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t k2 = at.has(i) ? order_key(v[i]) : 0u;
                key = k2 < best && k2 > key ? k2 : key;
            }
        }
    }
    const float least = __uint_as_float(reach & 0x80000000u ? reach & 0x7fffffffu : ~reach);
    float from = least;
    if (p.bias) {   // by how much values may be off
        const float big = warp_max(keep ? top : -INFINITY);
        const float arg = sm ? big - m : big;
        const float off = score_error(fast_score(big, m, inv, sm), fmaxf(1.0f, fabsf(arg)), sm);
        from = least - 4.0f * fmaf(fabsf(least), kStep, off);
    }
    // (absent experts are at -infinity: where that, or NaN, would do, choose64 does)
    all = all || !(from > -INFINITY);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (v[i] >= from) bits |= 1u << i;
    if (!keep) bits = 0;
    const int n = collect<U>(bits, at, list);
    int e = 0, rank = 32;
    float l = 0.0f;
    if (n > 32 || n < p.k) {
        all = true;
    } else if (!all) {
        float x = -INFINITY, err = 0.0f;
        if (lane < n) {
            e = list[lane];
            if (!moe_check(e >= 0 && e < p.E, 1611)) e = 0;
            l = row[e];
            x = fmaxf(l, -INFINITY);
            if (p.bias) {
                const float s = fast_score(l, m, inv, sm);
                x = fmaxf(s + p.bias[e], -INFINITY);
                err = fmaf(fabsf(x), kStep, score_error(s, sm ? l - m : l, sm));
            }
        }
        few[lane] = x;   // -infinity behind the last
        // both of two neighbours within the largest error: their order is open
        const float apart = p.bias ? 2.0f * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(fminf(err, 3e38f))))
                                   : 0.0f;
        __syncwarp();
        rank = 0;
        int close = 0;   // how many are that near, itself among them
        for (int j = 0; j < n; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(few + j);
            rank += (o.x > x) + (o.y > x) + (o.z > x) + (o.w > x);
            close += (fabsf(o.x - x) <= apart) + (fabsf(o.y - x) <= apart) + (fabsf(o.z - x) <= apart) +
                     (fabsf(o.w - x) <= apart);
        }
        if (__any_sync(kAll, lane < n && rank < p.k && close != 1)) {
            if (!p.bias) {   // equal logits, or infinite ones: the lower expert first
                rank = 0;
                for (int j = 0; j < n; ++j) rank += few[j] > x || (few[j] == x && list[j] < e);
            } else {
                bool open_still = true;
                if (sm && sum64 == 0) {
                    rank = rank_rough(p, t, e, n, m, inv, list, wide, scores[threadIdx.x >> 5], &open_still);
                    if (open_still) sum64 = row_sum64<PER, U>(p, t, &m);
                }
                if (open_still) {
                    double exact = -INFINITY;
                    if (lane < n) {
                        exact = value64(p, t, e, m, sum64);
                        exact = exact != exact ? -INFINITY : exact;
                    }
                    __syncwarp();
                    wide[lane] = exact;
                    __syncwarp();
                    rank = 0;
                    for (int j = 0; j < n; ++j) rank += wide[j] > exact || (wide[j] == exact && list[j] < e);
                }
            }
        }
        if (lane >= n) rank = 32;
    }
    if (all) {
        rank = lane < p.k ? lane : 32;
        e = choose64<PER, U>(p, t);
        if (!moe_check(lane >= p.k || (e >= 0 && e < p.E), 1612)) e = 0;
        l = lane < p.k ? row[e] : 0.0f;
    }
    const bool chosen = rank < p.k;
    float s;
    // shares of the chosen: softmax's, and sigmoid's of small logits only, are those of e^l
    if (p.renorm && (sm || !__any_sync(kAll, chosen && !(l < kSmall)))) {
        const float big = warp_max(chosen ? l : -INFINITY);
        s = sm || big > kNone ? __expf(l - big) : 0.0f;
    } else {
        s = fast_score(l, m, inv, sm);
    }
    if (p.renorm) {
        const float sum = warp_sum(chosen ? s : 0.0f);
        s = sum == 0.0f ? 0.0f : __fdividef(s, sum);
    }
    if (chosen) {
        p.idx[t * p.k + rank] = e;
        p.w[t * p.k + rank] = s * p.scale;
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

// A lane's chosen expert (-1: none), the gradient of its weight and its logit.  Asked for
// before the row and, as the logit waits for the expert, behind it: the waits overlap
// (65536 x 384: 24.4 us, asked for together 26.6).
struct Chosen {
    int e = -1;
    float g = 0.0f, l = -INFINITY;
    __device__ __forceinline__ void ask(const SelectBwdParams& p, int64_t t) {
        const int lane = threadIdx.x & 31;
        if (lane >= p.k) return;
        e = p.idx[t * p.k + lane];
        g = p.dw[t * p.k + lane] * p.scale;
    }
    __device__ __forceinline__ void logit(const SelectBwdParams& p, int64_t t) {
        if (e < 0 || e >= p.E)
            e = -1;
        else
            l = p.logits[t * p.E + e];
    }
};

// The chosen logit's own part of the gradient, and for softmax without renormalisation
// what the whole row is made from: dl_e = s_e (g_e - all).
__device__ __forceinline__ float chosen_grad(const SelectBwdParams& p, const Chosen& c, float m, float inv,
                                             float* all) {
    if (p.softmax && !p.renorm) {
        const float s = c.e >= 0 ? __expf(c.l - m) * inv : 0.0f;
        *all = warp_sum(c.e >= 0 ? c.g * s : 0.0f);
        return s * (c.g - *all);
    }
    float s, gate = 1.0f;   // ds/dl = s gate
    if (p.renorm && (p.softmax || !__any_sync(kAll, c.e >= 0 && !(c.l < kSmall)))) {   // as the forward
        const float top = warp_max(c.l);
        s = c.e >= 0 && (p.softmax || top > kNone) ? expf(c.l - top) : 0.0f;
    } else {
        const float x = expf(-c.l);
        s = c.e >= 0 ? 1.0f / (1.0f + x) : 0.0f;
        gate = x > 3e38f ? 1.0f : x / (1.0f + x);   // 1 - s, without the difference
    }
    if (!p.renorm) return s * gate * c.g;
    const float sum = warp_sum(s);
    const float n = sum == 0.0f ? 0.0f : s / sum;
    return n * gate * (c.g - warp_sum(c.e >= 0 ? c.g * n : 0.0f));
}

__device__ __forceinline__ void put4(float* o, const float (&v)[4]) {
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put4(uint16_t* o, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// A warp a token, four neighbouring experts a lane at a time; the chosen experts' places
// are written again behind the row.
template <int Q, typename Out>
__global__ void __launch_bounds__(kThreads) router_select_bwd4_kernel(const SelectBwdParams p) {
    wait_earlier();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    Out* to = static_cast<Out*>(p.dlogits) + t * p.E;
    const int quads = p.E / 4;
    float m = 0.0f, inv = 0.0f, all = 0.0f, d;
    Chosen c;
    c.ask(p, t);
    if (p.softmax && !p.renorm) {
        float4 v[Q];
        const float4* row = reinterpret_cast<const float4*>(p.logits + t * p.E);
#pragma unroll
        for (int i = 0; i < Q; ++i)
            v[i] = lane + 32 * i < quads ? row[lane + 32 * i]
                                         : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        c.logit(p, t);
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < Q; ++i) m = fmaxf(m, fmaxf(fmaxf(v[i].x, v[i].y), fmaxf(v[i].z, v[i].w)));
        m = warp_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            v[i] = make_float4(__expf(v[i].x - m), __expf(v[i].y - m), __expf(v[i].z - m), __expf(v[i].w - m));
            sum += (v[i].x + v[i].y) + (v[i].z + v[i].w);
        }
        inv = 1.0f / warp_sum(sum);
        d = chosen_grad(p, c, m, inv, &all);
        const float f = -inv * all;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const float o[4] = {v[i].x * f, v[i].y * f, v[i].z * f, v[i].w * f};
            if (lane + 32 * i < quads) put4(to + 4 * (lane + 32 * i), o);
        }
    } else {
        const float o[4] = {};
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (lane + 32 * i < quads) put4(to + 4 * (lane + 32 * i), o);
        c.logit(p, t);
        d = chosen_grad(p, c, m, inv, &all);
    }
    __syncwarp();   // the row is written
    if (c.e >= 0) put(to + c.e, d);
}

// The same for rows that are not in whole fours, where only the chosen have a gradient: the
// block's rows, which stand side by side in memory, are written as one run of zeros in
// 16-byte pieces, the chosen experts' places behind it (22824 x 302 in fp32: 7.2 us, put
// together in shared memory 19.6; for whole fours a row a warp is as fast or faster).
template <typename Out>
__global__ void __launch_bounds__(kRowThreads) router_select_sparse_kernel(const SelectBwdParams p) {
    constexpr int W = kRowThreads / 32;
    wait_earlier();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * W, t = t0 + (threadIdx.x >> 5);
    Chosen c;
    if (t < p.T) c.ask(p, t);
    Out* to = static_cast<Out*>(p.dlogits) + t0 * p.E;
    const int n = static_cast<int>(p.T - t0 < W ? p.T - t0 : W) * p.E, each = 16 / static_cast<int>(sizeof(Out));
    for (int i = threadIdx.x; i < n / each; i += kRowThreads)
        reinterpret_cast<uint4*>(to)[i] = make_uint4(0, 0, 0, 0);
    for (int i = n / each * each + threadIdx.x; i < n; i += kRowThreads) put(to + i, 0.0f);
    if (t < p.T) c.logit(p, t);
    const float d = chosen_grad(p, c, 0.0f, 0.0f, nullptr);
    __syncthreads();   // the zeros are written
    if (c.e >= 0) put(to + (t - t0) * p.E + c.e, d);
}

// And for the softmax of the whole row, PER experts a lane: a row is put together in shared
// memory, and the block's rows are written as one run (65536 x 383: 33 us, the row read
// three times instead of held 50).
template <int PER, typename Out>
__global__ void __launch_bounds__(kRowThreads) router_select_bwd_kernel(const SelectBwdParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    wait_earlier();
    Out* rows = reinterpret_cast<Out*>(smem);
    constexpr int W = kRowThreads / 32;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * W, t = t0 + wid;
    if (t < p.T) {
        Out* mine = rows + static_cast<int64_t>(wid) * p.E;
        const float* row = p.logits + t * p.E;
        Chosen c;
        c.ask(p, t);
        float v[PER], m = -INFINITY, sum = 0.0f, all;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = lane + 32 * i < p.E ? row[lane + 32 * i] : -INFINITY;
        c.logit(p, t);
#pragma unroll
        for (int i = 0; i < PER; ++i) m = fmaxf(m, v[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = __expf(v[i] - m);
            sum += v[i];
        }
        const float inv = 1.0f / warp_sum(sum), d = chosen_grad(p, c, m, inv, &all), f = -inv * all;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < p.E) put(mine + lane + 32 * i, v[i] * f);
        __syncwarp();
        if (c.e >= 0) put(mine + c.e, d);
    }
    __syncthreads();
    const int64_t n = (p.T - t0 < W ? p.T - t0 : W) * p.E * static_cast<int64_t>(sizeof(Out));
    uint8_t* to = static_cast<uint8_t*>(p.dlogits) + t0 * p.E * static_cast<int64_t>(sizeof(Out));
    const int full = static_cast<int>(n / 16);
    for (int i = threadIdx.x; i < full; i += kRowThreads)
        reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(smem)[i];
    for (int i = full * 16 / static_cast<int>(sizeof(Out)) + threadIdx.x;
         i < static_cast<int>(n / static_cast<int64_t>(sizeof(Out))); i += kRowThreads)
        reinterpret_cast<Out*>(to)[i] = rows[i];
}

template <typename Out>
int start_backward(const SelectBwdParams& p, cudaStream_t st) {
    const bool four = p.E % 4 == 0, dense = p.softmax && !p.renorm;
    const int need = (p.E / 4 + 31) / 32, threads = four ? kThreads : kRowThreads;
    const int64_t grid = (p.T + threads / 32 - 1) / (threads / 32);
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    void (*kern)(SelectBwdParams) =
        !four       ? (!dense         ? router_select_sparse_kernel<Out>
                       : p.E <= 256 ? router_select_bwd_kernel<8, Out>
                       : p.E <= 512 ? router_select_bwd_kernel<16, Out>
                                    : router_select_bwd_kernel<32, Out>)
        : need <= 1 ? router_select_bwd4_kernel<1, Out>
        : need <= 2 ? router_select_bwd4_kernel<2, Out>
        : need <= 3 ? router_select_bwd4_kernel<3, Out>
        : need <= 4 ? router_select_bwd4_kernel<4, Out>
                    : router_select_bwd4_kernel<8, Out>;
    return launch_early(kern, grid, threads, four || !dense ? 0 : threads / 32 * p.E * sizeof(Out), st, p);   // 32 KB at most
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
    p.log_lanes = 0;
    while (1 << p.log_lanes < p.lanes) ++p.log_lanes;
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
    // four neighbours a lane where the groups and the rows are in whole fours
    const bool four = p.per % 4 == 0;
    const int unit = four ? 4 : 1, units = p.per / unit;
    const int need = (units + p.lanes - 1) / p.lanes * unit;
    void (*kern)(SelectParams) =
        four ? (need <= 4    ? router_select_kernel<4, 4>
                : need <= 8  ? router_select_kernel<8, 4>
                : need <= 12 ? router_select_kernel<12, 4>
                : need <= 16 ? router_select_kernel<16, 4>
                             : router_select_kernel<32, 4>)
             : (need <= 4    ? router_select_kernel<4, 1>
                : need <= 8  ? router_select_kernel<8, 1>
                : need <= 16 ? router_select_kernel<16, 1>
                             : router_select_kernel<32, 1>);
    if (const int rc = launch_early(kern, grid, kThreads, 0, st, p)) return rc;
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
    if (const int rc = c.grad_f32 ? start_backward<float>(p, st) : start_backward<uint16_t>(p, st)) return rc;
    trace_after(st, "router_select_bwd");
    return MOE_OK;
}

}  // namespace moe
