// distill.cu -- loss of a student's logits z against a teacher's top logits y, and its
// gradient.
//
//     p = softmax(y / tau) over a token's given entries,  q = softmax(z / tau) over all V
//     loss = scale w tau^2 sum_k p_k (log p_k - log q_{i_k})
//     dz_v = scale w tau (q_v - sum over k with i_k = v of p_k)
//
// A team of threads takes a row.  One pass over it carries the running maximum and the sum
// of exponentials (in base 2, the temperature folded into the factor), while one more warp
// brings the entries; the gradient is a second pass, which writes q, and the entries' places
// are written again behind that.  A row of up to 2 KB stays in a warp's registers between
// the passes; of one of more than 64 KB shared memory keeps a part; else the second pass
// reads L2.
//   Forward of 4096 x 131072 bf16 (1.07 GB): 149 us, 7.2 TB/s; of 10172 x 12288: 46, floor
// 37.  Gradient alone of 15258 x 8192: 75, floor 74.  Loss and gradient of 8192 x 131072, a
// tenth of the rows without weight: 671 us, 6.1 TB/s of the 4.1 GB that have to move; the
// exponentials alone (two a logit) are 460 us at 16 a cycle and SM, and the second reading
// of the row is L2's.  A ring of chunks in the shared memory of a cluster, filled and
// drained by bulk copies, moved nothing twice and took 950: a CTA's two passes and the
// meeting between them follow each other, and only one fits on an SM.  Rows of 12 to 64 KB
// kept in the registers of 128 to 480 threads took 10 to 45 % more than read again.
#include "common.cuh"
#include "early.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxEntries = MOE_DISTILL_MAX_ENTRIES;   // of a token
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kForward = 0, kStep = 1, kBackward = 2 };

struct DistillParams {
    int64_t T, V, z_ld, dz_ld;
    int K, teacher_f32;
    float c, loss_f, grad_f;   // log2(e) / tau, scale tau^2, scale tau
    const void *z, *teacher;
    const int32_t* ids;
    const float* weight;
    float *loss, *lse;
    void* dz;
    int32_t* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(uint16_t* o, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *o = *reinterpret_cast<const uint16_t*>(&b);
}

// The 16 bytes of a vector as floats.
__device__ __forceinline__ void spread(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void spread(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 gather(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 gather(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Running maximum and sum of 2^(x - maximum).  Every operation is written out, so that
// what is contracted does not hang on what a kernel does besides.
struct Run {
    float m = -INFINITY, s = 0.0f;
    // raises the maximum to at least v; what to subtract from the exponents
    __device__ __forceinline__ float raise(float v) {
        if (v > m) {
            s = __fmul_rn(s, exp2_fast(__fsub_rn(m, v)));
            m = v;
        }
        return m == -INFINITY ? 0.0f : m;
    }
    // the exponent x c in one rounding with the maximum, which for the sum is what it is
    __device__ __forceinline__ void add(float x, float c) {
        const float b = raise(__fmul_rn(x, c));
        s = __fadd_rn(s, exp2_fast(__fmaf_rn(x, c, -b)));
    }
    __device__ __forceinline__ void join(float om, float os) {
        const float b = raise(om);
        s = __fmaf_rn(os, exp2_fast(__fsub_rn(om, b)), s);
    }
};

// TEAM threads over a row; a CTA's team has a warp for the entries besides.
template <int TEAM>
struct Team {
    int tid;
    float* red;   // [2][TEAM / 32], TEAM > 32
    __device__ __forceinline__ void sync() const {
        if (TEAM == 32) __syncwarp();
        else __syncthreads();
    }
    // A meeting of all; what the entries' warp brings is not used.
    __device__ __forceinline__ Run join(Run r) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            r.join(__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o));
        if (TEAM == 32) return r;
        if ((tid & 31) == 0 && tid < TEAM) {
            red[tid >> 5] = r.m;
            red[TEAM / 32 + (tid >> 5)] = r.s;
        }
        __syncthreads();
        Run all;
        for (int i = 0; i < TEAM / 32; ++i) all.join(red[i], red[TEAM / 32 + i]);
        return all;
    }
};

constexpr int kUnroll = 4;   // vectors that a thread has under way

// A token's entries, by one warp: the teacher's distribution, and the student's exponents
// at the entries' words.  The arrays end in whole fours, without words behind the last.
struct Entries {
    int* id;        // [K] the word, -1: not there
    float *p, *x;   // [K] probability, the student's logit
    float* y;       // [K] the teacher's logit, then log2 of its probability
    float* total;   // [K] p of all entries of the word, at its first; -1 at others
};

// False where the row has none.
template <typename Z>
__device__ __forceinline__ bool load_entries(const DistillParams& p, int64_t t, const Z* z, const Entries& e) {
    const int lane = threadIdx.x & 31;
    Run ty;
    for (int k = lane; k < (p.K + 3) / 4 * 4; k += 32) {
        const int i = k < p.K ? p.ids[t * p.K + k] : -1;
        const bool ok = i >= 0 && i < p.V;
        if (!ok && i != -1) report_error(p.status, MOE_EINVAL);
        float y = -INFINITY;
        if (ok)
            y = p.teacher_f32 ? static_cast<const float*>(p.teacher)[t * p.K + k]
                              : to_float(static_cast<const uint16_t*>(p.teacher)[t * p.K + k]);
        e.id[k] = ok ? i : -1;
        e.y[k] = y;
        e.x[k] = ok ? to_float(z[i]) : 0.0f;
        if (ok) ty.add(y, p.c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ty.join(__shfl_xor_sync(0xffffffffu, ty.m, o), __shfl_xor_sync(0xffffffffu, ty.s, o));
    if (ty.m == -INFINITY && ty.s == 0.0f) return false;
    const float inv = 1.0f / ty.s, logs = log2f(ty.s);
    for (int k = lane; k < (p.K + 3) / 4 * 4; k += 32) {
        const float y = e.y[k], a = __fmaf_rn(y, p.c, -ty.m);
        e.p[k] = y == -INFINITY ? 0.0f : __fmul_rn(exp2_fast(a), inv);
        e.y[k] = __fsub_rn(a, logs);
    }
    return true;
}

// Words that several entries name: their first entry stands for all.
__device__ __forceinline__ void total_entries(const DistillParams& p, const Entries& e) {
    for (int k = threadIdx.x & 31; k < p.K; k += 32) {
        const int id = e.id[k];
        float sum = 0.0f;
        bool first = id >= 0;
        for (int j = 0; first && j < p.K; j += 4) {
            const int4 o = *reinterpret_cast<const int4*>(e.id + j);
            const float4 q = *reinterpret_cast<const float4*>(e.p + j);
            first = !((o.x == id && j < k) || (o.y == id && j + 1 < k) || (o.z == id && j + 2 < k) || (o.w == id && j + 3 < k));
            sum += (o.x == id ? q.x : 0.0f) + (o.y == id ? q.y : 0.0f) + (o.z == id ? q.z : 0.0f) + (o.w == id ? q.w : 0.0f);
        }
        e.total[k] = first ? sum : -1.0f;
    }
}

// sum_k p_k (log2 p_k - log2 q_k), by one warp; log2 q = (x c - m) - logs, from the row's
// maximum and not from lse, so that a word near it loses nothing to the size of the logits.
__device__ __forceinline__ float entries_loss(const DistillParams& p, const Entries& e, float m, float logs) {
    float loss = 0.0f;
    for (int k = threadIdx.x & 31; k < p.K; k += 32)
        if (e.p[k] != 0.0f) loss = __fmaf_rn(e.p[k], __fsub_rn(e.y[k], __fsub_rn(__fmaf_rn(e.x[k], p.c, -m), logs)), loss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    return loss;
}

// The lowest value of a type, in every place of a vector: its exponentials are 0.
template <typename Z>
__device__ __forceinline__ uint4 nothing() {
    const uint32_t w = sizeof(Z) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// Zeros for a row without weight or entries.
template <typename Z, int TEAM>
__device__ __forceinline__ void clear_row(Z* dz, int64_t V, int tid) {
    constexpr int E = 16 / static_cast<int>(sizeof(Z));
    const int64_t to_vec = ((16 - (reinterpret_cast<uintptr_t>(dz) & 15)) & 15) / sizeof(Z);
    const int64_t h = to_vec < V ? to_vec : V, n = (V - h) / E;
    for (int64_t i = tid; i < h; i += TEAM) put(dz + i, 0.0f);
    for (int64_t i = tid; i < n; i += TEAM) __stcs(reinterpret_cast<uint4*>(dz + h) + i, make_uint4(0, 0, 0, 0));
    for (int64_t i = h + n * E + tid; i < V; i += TEAM) put(dz + i, 0.0f);
}

// HELD: vectors a thread, where the team's registers keep the row between the passes; else
// 0, and STASH vectors a thread are kept in shared memory.  BLOCKS: CTAs on an SM.  The
// entries are brought by a warp of their own while the others are in the first pass (a warp
// that is the whole team brings them itself).
template <typename Z, int TEAM, int MODE, int HELD, int STASH, int BLOCKS>
__global__ void __launch_bounds__(TEAM == 32 ? 256 : TEAM + 32, BLOCKS) distill_kernel(const DistillParams p) {
    static_assert(STASH % kUnroll == 0, "in whole groups");
    constexpr int kTeams = TEAM == 32 ? 8 : 1;
    constexpr int E = 16 / static_cast<int>(sizeof(Z));
    constexpr bool HOLD = HELD > 0;
    extern __shared__ __align__(16) uint4 stash[];   // and behind it the entries' arrays
    __shared__ float s_red[TEAM == 32 ? 1 : TEAM / 16];
    __shared__ int s_none;
    wait_earlier();
    const int which = TEAM == 32 ? static_cast<int>(threadIdx.x >> 5) : 0;
    Team<TEAM> team{static_cast<int>(TEAM == 32 ? threadIdx.x & 31 : threadIdx.x), s_red};
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + which;
    if (t >= p.T) return;
    const int tid = team.tid;
    const bool works = TEAM == 32 || tid < TEAM, brings = TEAM == 32 || tid >= TEAM;
    const int width = (p.K + 3) / 4 * 4;
    float* arrays = reinterpret_cast<float*>(stash + STASH * TEAM) + which * 5 * width;
    const Entries en{reinterpret_cast<int*>(arrays), arrays + width, arrays + 2 * width, arrays + 3 * width,
                     arrays + 4 * width};
    const Z* z = static_cast<const Z*>(p.z) + t * p.z_ld;
    Z* dz = static_cast<Z*>(p.dz) + t * p.dz_ld;
    // the row's run of whole vectors
    const int64_t to_vec = ((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(Z);
    const int64_t head = to_vec < p.V ? to_vec : p.V;
    const int64_t nvec = (p.V - head) / E, tail = head + nvec * E;
    const uint4* zv = reinterpret_cast<const uint4*>(z + head);
    const int groups = static_cast<int>((nvec + kUnroll * TEAM - 1) / (kUnroll * TEAM));
    const int full = static_cast<int>(nvec / (kUnroll * TEAM));   // without a vector behind the row's last

    uint4 held[HOLD ? HELD : 1];
    if (HOLD && works) {   // before the weight is known: a short row's time is latency
#pragma unroll
        for (int j = 0; j < HELD; ++j) held[j] = tid + j * TEAM < nvec ? zv[tid + j * TEAM] : nothing<Z>();
    }
    const float w = p.weight ? p.weight[t] : 1.0f;
    if (w == 0.0f) {
        if (MODE != kBackward && tid == 0) {
            p.loss[t] = 0.0f;
            p.lse[t] = 0.0f;
        }
        if (MODE != kForward && works) clear_row<Z, TEAM>(dz, p.V, tid);
        return;
    }
    bool none = false;   // no entry
    if (brings) {
        none = !load_entries(p, t, z, en);
        if (TEAM > 32 && (tid & 31) == 0) s_none = none;
        if (MODE != kForward) {
            __syncwarp();
            total_entries(p, en);
        }
    }
    float m, inv = 1.0f;   // q = 2^(x c - m) inv; the gradient alone has log2 of the sum for m
    // the gradient alone goes on at once, unless it takes the place of logits that the
    // entries' warp may still be reading
    const bool meets = MODE != kBackward || static_cast<const void*>(z) == static_cast<void*>(dz);
    if (MODE == kBackward) {
        m = p.lse[t] * kLog2e;
        if (meets) {
            team.sync();
            if (TEAM > 32) none = s_none;
        }
    } else {
        Run r;
        if (works) {
            for (int64_t i = tid; i < head; i += TEAM) r.add(to_float(z[i]), p.c);
            for (int64_t q = tail + tid; q < p.V; q += TEAM) r.add(to_float(z[q]), p.c);
            auto take = [&](const uint4& v) {
                float f[E];
                spread(v, f);
                float top = f[0];
#pragma unroll
                for (int e = 1; e < E; ++e) top = fmaxf(top, f[e]);
                const float b = r.raise(__fmul_rn(top, p.c));
#pragma unroll
                for (int e = 0; e < E; ++e) r.s = __fadd_rn(r.s, exp2_fast(__fmaf_rn(f[e], p.c, -b)));
            };
            if (HOLD) {
#pragma unroll
                for (int j = 0; j < HELD; ++j)
                    if (tid + j * TEAM < nvec) take(held[j]);
            } else {
                for (int g = 0; g < groups; ++g) {
                    const int64_t i = tid + static_cast<int64_t>(g) * kUnroll * TEAM;
                    uint4 v[kUnroll];
                    if (g < full) {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) v[j] = zv[i + j * TEAM];
                    } else {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) v[j] = i + j * TEAM < nvec ? zv[i + j * TEAM] : nothing<Z>();
                    }
                    if (g < STASH / kUnroll) {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) stash[i + j * TEAM] = v[j];
                    }
#pragma unroll
                    for (int j = 0; j < kUnroll; ++j) take(v[j]);
                }
            }
        }
        r = team.join(r);
        m = r.m;
        inv = 1.0f / r.s;
        if (TEAM > 32) none = s_none;
        if (brings) {
            const float logs = log2f(r.s), loss = none ? 0.0f : entries_loss(p, en, m, logs);
            if ((tid & 31) == 0) {
                p.loss[t] = none ? 0.0f : loss * kLn2 * (w * p.loss_f);
                p.lse[t] = none ? 0.0f : __fadd_rn(m, logs) * kLn2;
            }
        }
    }
    if (MODE == kForward) return;
    const float f = w * p.grad_f, fq = f * inv;
    if (works && !none) {
        auto grad = [&](float x) { return fq * exp2_fast(fmaf(x, p.c, -m)); };
        for (int64_t i = tid; i < head; i += TEAM) put(dz + i, grad(to_float(z[i])));
        auto give = [&](const uint4& v) {
            float g[E];
            spread(v, g);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = grad(g[e]);
            return gather(g);
        };
        if (((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0) {
            uint4* dv = reinterpret_cast<uint4*>(dz + head);
            if (HOLD) {
#pragma unroll
                for (int j = 0; j < HELD; ++j)
                    if (tid + j * TEAM < nvec) __stcs(dv + tid + j * TEAM, give(held[j]));
            } else {
                // What the first pass read last is in L2 most surely, so the second goes
                // backwards, past L2's other lines (streaming loads and stores), and ends
                // with what shared memory holds.
                for (int g = groups - 1; g >= 0; --g) {
                    const int64_t i = tid + static_cast<int64_t>(g) * kUnroll * TEAM;
                    uint4 v[kUnroll];
                    if (g < STASH / kUnroll) {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) v[j] = stash[i + j * TEAM];
                    } else if (g < full) {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) v[j] = MODE == kStep ? __ldcs(zv + i + j * TEAM) : zv[i + j * TEAM];
                    } else {
#pragma unroll
                        for (int j = 0; j < kUnroll; ++j) v[j] = i + j * TEAM < nvec ? zv[i + j * TEAM] : nothing<Z>();
                    }
#pragma unroll
                    for (int j = 0; j < kUnroll; ++j) {
                        if (g >= full && i + j * TEAM >= nvec) continue;
                        if (MODE == kStep) __stcs(dv + i + j * TEAM, give(v[j]));
                        else dv[i + j * TEAM] = give(v[j]);
                    }
                }
            }
        } else {   // rows that start at different places within 16 bytes
            for (int64_t i = head + tid; i < tail; i += TEAM) put(dz + i, grad(to_float(z[i])));
        }
        for (int64_t i = tail + tid; i < p.V; i += TEAM) put(dz + i, grad(to_float(z[i])));
    }
    team.sync();
    if (TEAM > 32) none = s_none;
    if (none) {
        if (works) clear_row<Z, TEAM>(dz, p.V, tid);
        return;
    }
    // the entries' words, behind the row
    for (int k = tid; k < p.K; k += TEAM) {
        const float total = en.total[k];
        if (works && en.id[k] >= 0 && !(total < 0.0f)) put(dz + en.id[k], f * (exp2_fast(fmaf(en.x[k], p.c, -m)) * inv - total));
    }
}

// The sum of all tokens' losses, in a fixed order.
__global__ void __launch_bounds__(1024) distill_total_kernel(const float* loss, int64_t T,
                                                             float* total) {
    __shared__ float red[32];
    wait_earlier();   // the losses are complete
    float s = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += 1024) s += __ldcg(loss + t);   // past L1, as it started early
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = red[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) *total = s;
    }
}

template <typename Z, int TEAM, int MODE, int HELD, int STASH, int BLOCKS>
int start_team(const DistillParams& p, cudaStream_t st) {
    const int64_t grid = TEAM == 32 ? (p.T + 7) / 8 : p.T;
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    const auto kern = distill_kernel<Z, TEAM, MODE, HELD, STASH, BLOCKS>;
    const int most = STASH * TEAM * 16 + (TEAM == 32 ? 8 : 1) * 5 * 4 * kMaxEntries;
    const int bytes = STASH * TEAM * 16 + (TEAM == 32 ? 8 : 1) * 5 * 4 * ((p.K + 3) / 4 * 4);
    if (const int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), most)) return rc;
    return launch_early(kern, grid, TEAM == 32 ? 256 : TEAM + 32, static_cast<size_t>(bytes), st, p);
}

template <typename Z, int MODE>
int start(const DistillParams& p, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    const int64_t bytes = p.V * static_cast<int64_t>(sizeof(Z)), vectors = bytes / 16;
    if (vectors <= 32 * 4) return start_team<Z, 32, MODE, 4, 0, 4>(p, st);   // a warp's registers hold the row
    // Few threads a row leave little to a row's own waits and meetings, many keep the rows
    // that are under way few, so that what is read again is still near.  (250 MB of bf16 rows of 8,
    // 24, 64 KB: forward with 32, 128, 256, 512 threads 28, 37, 69, 153 us; 46, 46, 60, 97;
    // 47, 44, 44, 53.  Loss and gradient 52, 60, 101, 225; 115, 83, 97, 155; 126, 105, 87, 88.)
    constexpr int64_t K = 1024;
    constexpr int64_t kWarp = MODE == kForward ? 20 * K : MODE == kBackward ? 6 * K : 8 * K;
    constexpr int64_t kSmall = MODE == kForward ? 48 * K : MODE == kBackward ? 14 * K : 28 * K;
    constexpr int64_t kMiddle = MODE == kForward ? int64_t{1} << 62 : MODE == kBackward ? 48 * K : 64 * K;
    int team = bytes <= kWarp ? 32 : bytes <= kSmall ? 128 : bytes <= kMiddle ? 256 : 512;
    // as many as there is room for where the rows are few, with four vectors each (5 rows of 8
    // KB, forward, 128 threads 2.6 us, 512 3.4)
    const int room = p.T <= 3 * sms ? 512 : p.T <= 7 * sms ? 256 : p.T <= 12 * sms ? 128 : 32;
    const int most = vectors >= 2048 ? 512 : vectors >= 1024 ? 256 : vectors >= 256 || p.T <= 4 * sms ? 128 : 32;
    const int wide = room < most ? room : most;
    team = team < wide ? wide : team;
    if (team == 32) return start_team<Z, 32, MODE, 0, 0, 5>(p, st);
    if (team == 128) return start_team<Z, 128, MODE, 0, 0, 12>(p, st);
    if (team == 256) return start_team<Z, 256, MODE, 0, 0, 7>(p, st);
    if constexpr (MODE == kStep) {
        // as many rows at once as half of L2 holds, and more of a longer row in shared memory
        // (8192 rows of 128 KB: 355 us with two CTAs an SM, 313 with three; of 256 KB: 668, 742)
        if (bytes * 3 * sms <= (64ll << 20)) return start_team<Z, 480, MODE, 0, 4, 3>(p, st);
        return start_team<Z, 512, MODE, 0, 8, 2>(p, st);
    } else {
        return start_team<Z, 512, MODE, 0, 0, 3>(p, st);
    }
}

DistillParams distill_params(const moe_distill_t& c, const void* z, const int32_t* ids,
                             const void* teacher, const float* weight) {
    DistillParams p = {};
    p.T = c.T;
    p.V = c.V;
    p.z_ld = c.z_ld;
    p.dz_ld = c.dz_ld;
    p.K = c.K;
    p.teacher_f32 = c.teacher_f32;
    p.c = static_cast<float>(1.4426950408889634074 / c.temperature);
    p.loss_f = c.scale * c.temperature * c.temperature;
    p.grad_f = c.scale * c.temperature;
    p.z = z;
    p.ids = ids;
    p.teacher = teacher;
    p.weight = weight;
    return p;
}

}  // namespace

int check_status_distill() { return moe_check_read_reset(); }

int launch_distill(const moe_distill_t& c, const void* z, const int32_t* ids, const void* teacher,
                   const float* weight, float* loss, float* lse, float* total, void* dz,
                   int32_t* status, cudaStream_t st) {
    DistillParams p = distill_params(c, z, ids, teacher, weight);
    p.loss = loss;
    p.lse = lse;
    p.dz = dz;
    p.status = status;
    const int rc = c.z_f32 ? (dz ? start<float, kStep>(p, st) : start<float, kForward>(p, st))
                           : (dz ? start<uint16_t, kStep>(p, st) : start<uint16_t, kForward>(p, st));
    if (rc) return rc;
    trace_after(st, "distill");
    if (!total) return MOE_OK;
    if (const int rc = launch_early(distill_total_kernel, 1, 1024, 0, st, loss, c.T, total)) return rc;
    trace_after(st, "distill_total");
    return MOE_OK;
}

int launch_distill_backward(const moe_distill_t& c, const void* z, const int32_t* ids,
                            const void* teacher, const float* weight, const float* lse, void* dz,
                            int32_t* status, cudaStream_t st) {
    DistillParams p = distill_params(c, z, ids, teacher, weight);
    p.lse = const_cast<float*>(lse);
    p.dz = dz;
    p.status = status;
    const int rc = c.z_f32 ? start<float, kBackward>(p, st) : start<uint16_t, kBackward>(p, st);
    if (rc == MOE_OK) trace_after(st, "distill_bwd");
    return rc;
}

}  // namespace moe
