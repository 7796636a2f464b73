// embedding.cu -- lookup of table rows with scaling, and the gradient of the table by
// sorted tokens.
//
// The gradient of a word's row is the sum of its tokens' gradients in the tokens' order, so
// that it does not hang on the order in which anything runs.  A plan (one launch of one
// cluster) groups the tokens by word and cuts each word's tokens into pieces of at most
// kPiece; a warp sums a piece over 1024 channels.  Words of one piece are written at once,
// the others' pieces go to scratch and are added up in their order by a second launch.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ lookup

struct LookupParams {
    int64_t T, V, total;
    int chunks;   // of 8 channels
    const void* table;
    const int32_t* ids;
    void* out;
    int32_t* status;
    float scale;
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

constexpr int kLook = 4;   // chunks that a thread has under way

template <typename Tab, typename Out>
__global__ void __launch_bounds__(256) embedding_kernel(const LookupParams p) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 * kLook + threadIdx.x;
    float f[kLook][8];
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const int64_t i = i0 + j * 256;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = 0.0f;
        if (i >= p.total) continue;
        const int64_t t = i / p.chunks;
        const int c = static_cast<int>(i - t * p.chunks);
        const int id = __ldg(p.ids + t);
        if (id >= 0 && id < p.V)
            load8(static_cast<const Tab*>(p.table) + (static_cast<int64_t>(id) * p.chunks + c) * 8, f[j]);
        else if (id != -1)
            report_error(p.status, MOE_EINVAL);
    }
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const int64_t i = i0 + j * 256;
        if (i >= p.total) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] *= p.scale;
        store8(static_cast<Out*>(p.out) + i * 8, f[j]);
    }
}

// ------------------------------------------------------------------ plan

constexpr int kPiece = 64;       // tokens of a piece
constexpr int kCluster = 8;      // CTAs that group the tokens
constexpr int kPlanThreads = 1024;
constexpr int kShort = 128;      // words of at most so many tokens are put in order by counting
constexpr int kWindow = 1 << 18; // tokens whose bits a CTA holds at once

struct PlanView {
    int32_t* head;    // [0] tokens placed, [1] pieces, [2] scratch rows, [3] words of several
                      // pieces, [4] words past kShort
    int32_t* count;   // [V]
    int32_t* start;   // [V] where a word's tokens begin in order
    int32_t* rank;    // [T] a token's place among its word's as they came
    int32_t* mixed;   // [T] the tokens by word, as they came
    int32_t* order;   // [T] the tokens by word, ascending
    int4* pieces;     // [T] {word, first place, tokens, scratch row or -1}
    int4* joins;      // [T / kPiece] {word, first scratch row, rows, 0}
    int32_t* longs;   // [T / kShort] words past kShort
    float* part;      // scratch rows [2 T / kPiece][d]
};

int64_t up(int64_t n) { return (n + 127) & ~int64_t{127}; }

int64_t plan_layout(int64_t T, int64_t V, int d, uint8_t* base, PlanView* v) {
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        uint8_t* p = base + o;
        o += up(bytes);
        return p;
    };
    PlanView w;
    w.head = reinterpret_cast<int32_t*>(take(64));
    w.count = reinterpret_cast<int32_t*>(take(V * 4));
    w.start = reinterpret_cast<int32_t*>(take(V * 4));
    w.rank = reinterpret_cast<int32_t*>(take(T * 4));
    w.mixed = reinterpret_cast<int32_t*>(take(T * 4));
    w.order = reinterpret_cast<int32_t*>(take(T * 4));
    w.pieces = reinterpret_cast<int4*>(take(T * 16));
    w.joins = reinterpret_cast<int4*>(take((T / kPiece + 1) * 16));
    w.longs = reinterpret_cast<int32_t*>(take((T / kShort + 1) * 4));
    w.part = reinterpret_cast<float*>(take((2 * (T / kPiece) + 1) * d * 4));
    if (v) *v = w;
    return o;
}

__device__ __forceinline__ int lanemask_lt_count(unsigned m) {
    unsigned lt;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(lt));
    return __popc(m & lt);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1)
    embedding_plan_kernel(const PlanView v, const int32_t* ids, int64_t T, int64_t V,
                          int32_t* status) {
    extern __shared__ uint32_t bits[];
    __shared__ int warp_sum[32];
    const int64_t me = static_cast<int64_t>(cluster_ctarank()) * kPlanThreads + threadIdx.x;
    const int64_t all = kCluster * kPlanThreads;
    for (int64_t i = me; i < (V + 3) / 4; i += all)
        reinterpret_cast<int4*>(v.count)[i] = make_int4(0, 0, 0, 0);   // the array is padded
    if (me < 16) v.head[me] = 0;
    __threadfence();
    cluster_sync();
    for (int64_t t = me; t < T; t += all) {
        const int id = __ldg(ids + t);
        int r = -1;
        if (id >= 0 && id < V)
            r = atomicAdd(v.count + id, 1);
        else if (id != -1)
            report_error(status, MOE_EINVAL);
        v.rank[t] = r;
    }
    __threadfence();
    cluster_sync();
    // a word's first token gives it its place and its pieces
    for (int64_t t = me; t < T; t += all) {
        if (v.rank[t] != 0) continue;
        const int id = __ldg(ids + t);
        const int n = __ldcg(v.count + id), np = (n + kPiece - 1) / kPiece;
        const int at = atomicAdd(v.head, n);
        const int pc = atomicAdd(v.head + 1, np);
        if (!moe_check(at + n <= T && pc + np <= T, 1621)) continue;
        v.start[id] = at;
        int row = -1;
        if (np > 1) {
            row = atomicAdd(v.head + 2, np);
            v.joins[atomicAdd(v.head + 3, 1)] = make_int4(id, row, np, 0);
        }
        if (n > kShort) v.longs[atomicAdd(v.head + 4, 1)] = id;
        for (int j = 0; j < np; ++j)
            v.pieces[pc + j] = make_int4(id, at + j * kPiece, n - j * kPiece < kPiece ? n - j * kPiece : kPiece,
                                         row < 0 ? -1 : row + j);
    }
    __threadfence();
    cluster_sync();
    for (int64_t t = me; t < T; t += all) {
        const int r = v.rank[t];
        if (r < 0) continue;
        const int id = __ldg(ids + t);
        const int at = __ldcg(v.start + id) + r;
        if (!moe_check(at < T, 1622)) continue;
        v.mixed[at] = static_cast<int32_t>(t);
    }
    __threadfence();
    cluster_sync();
    // in order: a token of a short word counts those before it
    for (int64_t t = me; t < T; t += all) {
        if (v.rank[t] < 0) continue;
        const int id = __ldg(ids + t);
        const int n = __ldcg(v.count + id), at = __ldcg(v.start + id);
        if (n > kShort) continue;
        int before = 0;
        for (int j = 0; j < n; ++j) before += __ldcg(v.mixed + at + j) < t;
        if (!moe_check(at + before < T, 1623)) continue;
        v.order[at + before] = static_cast<int32_t>(t);
    }
    // a long word's tokens are bits of a window of the batch, read out from its front
    const int longs = __ldcg(v.head + 4), lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int words = static_cast<int>((T < kWindow ? T : kWindow) + 31) / 32;
    for (int l = static_cast<int>(cluster_ctarank()); l < longs; l += kCluster) {
        const int id = __ldcg(v.longs + l), n = __ldcg(v.count + id), at = __ldcg(v.start + id);
        int done = 0;
        for (int64_t w0 = 0; w0 < T; w0 += kWindow) {
            for (int i = threadIdx.x; i < words; i += kPlanThreads) bits[i] = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < n; j += kPlanThreads) {
                const int64_t b = __ldcg(v.mixed + at + j) - w0;
                if (b >= 0 && b < kWindow && moe_check(b / 32 < words, 1624))
                    atomicOr(bits + b / 32, 1u << (b & 31));
            }
            __syncthreads();
            for (int i0 = 0; i0 < words; i0 += kPlanThreads) {
                const int i = i0 + threadIdx.x;
                uint32_t b = i < words ? bits[i] : 0;
                int incl = __popc(b);
                const int own = incl;
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (lane == 31) warp_sum[wid] = incl;
                __syncthreads();
                int base = done, total = 0;
                for (int w = 0; w < 32; ++w) {
                    if (w < wid) base += warp_sum[w];
                    total += warp_sum[w];
                }
                int to = at + base + incl - own;
                while (b) {
                    if (moe_check(to < at + n, 1625))
                        v.order[to] = static_cast<int32_t>(w0 + 32ll * i + __ffs(b) - 1);
                    ++to;
                    b &= b - 1;
                }
                done += total;
                __syncthreads();
            }
        }
    }
}

// ------------------------------------------------------------------ gradient

struct GradParams {
    PlanView v;
    int64_t T, V;
    int d, chunks, spans;   // chunks of 8 channels; spans of 1024 channels a row
    int accumulate;
    float scale;
    const void* dout;
    void* dtable;
};

constexpr int kSpan = 4;    // chunks a lane of a warp's 1024 channels

template <typename Tab>
__device__ __forceinline__ void finish(const GradParams& p, Tab* row, int c, float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] *= p.scale;
    if (p.accumulate) {
        float old[8];
        load8(row + 8 * c, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += old[e];
    }
    store8(row + 8 * c, s);
}

// Warps over the pieces' spans, then over the rows of words that do not occur.
template <typename In, typename Tab>
__global__ void __launch_bounds__(256) embedding_bwd_kernel(const GradParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t items = static_cast<int64_t>(p.v.head[1]) * p.spans;
    const In* dout = static_cast<const In*>(p.dout);
    Tab* dtable = static_cast<Tab*>(p.dtable);
    for (int64_t it = me; it < items; it += warps) {
        const int64_t pc = it / p.spans;
        const int c0 = static_cast<int>(it - pc * p.spans) * 32 * kSpan + lane;
        const int4 q = __ldg(p.v.pieces + pc);
        if (!moe_check(q.x >= 0 && q.x < p.V && q.y + q.z <= p.T, 1626)) continue;
        float s[kSpan][8];
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[j][e] = 0.0f;
        for (int r = 0; r < q.z; ++r) {
            const int64_t t = __ldg(p.v.order + q.y + r);
            const In* row = dout + t * p.d;
            float f[kSpan][8];
#pragma unroll
            for (int j = 0; j < kSpan; ++j)
                if (c0 + 32 * j < p.chunks) load8(row + 8 * (c0 + 32 * j), f[j]);
#pragma unroll
            for (int j = 0; j < kSpan; ++j)
                if (c0 + 32 * j < p.chunks)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[j][e] += f[j][e];
        }
#pragma unroll
        for (int j = 0; j < kSpan; ++j) {
            const int c = c0 + 32 * j;
            if (c >= p.chunks) continue;
            if (q.w >= 0)
                store8(p.v.part + static_cast<int64_t>(q.w) * p.d + 8 * c, s[j]);
            else
                finish(p, dtable + static_cast<int64_t>(q.x) * p.d, c, s[j]);
        }
    }
    if (p.accumulate) return;
    const float zero[8] = {};
    for (int64_t id = me; id < p.V; id += warps) {
        if (__ldg(p.v.count + id) != 0) continue;
        Tab* row = dtable + id * p.d;
        for (int c = lane; c < p.chunks; c += 32) store8(row + 8 * c, zero);
    }
}

// Words of several pieces: 32 threads over 256 channels, 8 runs of pieces side by side.
template <typename Tab>
__global__ void __launch_bounds__(256) embedding_join_kernel(const GradParams p) {
    __shared__ float red[8][32][8];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the pieces' sums are complete
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int wide = (p.chunks + 31) / 32;
    const int64_t items = static_cast<int64_t>(p.v.head[3]) * wide;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t w = it / wide;
        const int c = static_cast<int>(it - w * wide) * 32 + lane;
        const int4 q = __ldg(p.v.joins + w);
        float s[8] = {};
        if (c < p.chunks)
            for (int j = run; j < q.z; j += 8) {
                const float* r = p.v.part + static_cast<int64_t>(q.y + j) * p.d + 8 * c;
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] += r[e];
            }
#pragma unroll
        for (int e = 0; e < 8; ++e) red[run][lane][e] = s[e];
        __syncthreads();
        if (run == 0 && c < p.chunks) {
            for (int k = 1; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] += red[k][lane][e];
            finish(p, static_cast<Tab*>(p.dtable) + static_cast<int64_t>(q.x) * p.d, c, s);
        }
        __syncthreads();
    }
}

}  // namespace

int check_status_embedding() { return moe_check_read_reset(); }

int64_t embedding_plan_bytes(int64_t T, int64_t V, int d) {
    return plan_layout(T, V, d, nullptr, nullptr);
}

int launch_embedding(const moe_embedding_t& c, const void* table, const int32_t* ids, void* out,
                     int32_t* status, cudaStream_t st) {
    LookupParams p;
    p.T = c.T;
    p.V = c.V;
    p.chunks = c.d / 8;
    p.total = c.T * p.chunks;
    p.table = table;
    p.ids = ids;
    p.out = out;
    p.status = status;
    p.scale = c.scale;
    const int64_t grid = (p.total + 256 * kLook - 1) / (256 * kLook);
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    void (*kern)(LookupParams) =
        c.table_f32 ? (c.out_f32 ? embedding_kernel<float, float> : embedding_kernel<float, uint16_t>)
                    : (c.out_f32 ? embedding_kernel<uint16_t, float> : embedding_kernel<uint16_t, uint16_t>);
    kern<<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "embedding");
    return MOE_OK;
}

int launch_embedding_plan(int64_t T, int64_t V, int d, const int32_t* ids, void* plan,
                          int32_t* status, cudaStream_t st) {
    PlanView v;
    plan_layout(T, V, d, static_cast<uint8_t*>(plan), &v);
    const int bytes = static_cast<int>((T < kWindow ? T : kWindow) + 31) / 32 * 4;
    embedding_plan_kernel<<<kCluster, kPlanThreads, bytes, st>>>(v, ids, T, V, status);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "embedding_plan");
    return MOE_OK;
}

int launch_embedding_backward(const moe_embedding_t& c, const void* plan, const void* dout,
                              void* dtable, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    GradParams p;
    plan_layout(c.T, c.V, c.d, static_cast<uint8_t*>(const_cast<void*>(plan)), &p.v);
    p.T = c.T;
    p.V = c.V;
    p.d = c.d;
    p.chunks = c.d / 8;
    p.spans = (p.chunks + 32 * kSpan - 1) / (32 * kSpan);
    p.accumulate = c.accumulate;
    p.scale = c.scale;
    p.dout = dout;
    p.dtable = dtable;
    int64_t need = c.T * p.spans;
    if (!c.accumulate && need < c.V) need = c.V;
    need = (need + 7) / 8;
    const int64_t most = static_cast<int64_t>(sms) * 8;
    const unsigned grid = static_cast<unsigned>(need < most ? need : most);
    void (*kern)(GradParams) =
        c.out_f32 ? (c.table_f32 ? embedding_bwd_kernel<float, float> : embedding_bwd_kernel<float, uint16_t>)
                  : (c.table_f32 ? embedding_bwd_kernel<uint16_t, float> : embedding_bwd_kernel<uint16_t, uint16_t>);
    kern<<<grid, 256, 0, st>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "embedding_bwd");
    if (c.T <= kPiece) return MOE_OK;   // no word has several pieces
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms) * 2, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = c.table_f32 ? cudaLaunchKernelEx(&cfg, embedding_join_kernel<float>, p)
                                      : cudaLaunchKernelEx(&cfg, embedding_join_kernel<uint16_t>, p);
    if (e != cudaSuccess) return MOE_ECUDA;
    trace_after(st, "embedding_join");
    return MOE_OK;
}

}  // namespace moe
