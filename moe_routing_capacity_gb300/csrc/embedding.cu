// embedding.cu -- lookup of table rows with scaling, and the gradient of the table by
// sorted tokens.
//
// The gradient of a word's row is the sum of its tokens' gradients in the tokens' order, so
// that it does not hang on the order in which anything runs.  A plan groups the tokens by
// word and cuts each word's tokens into pieces of at most kPiece; a warp sums a piece over
// 512 channels.  Words of one piece are written at once, the others' pieces go to scratch
// and are added up in their order by a second launch, so that a word with half of the
// tokens costs no more than many words (the plan of 16384 of one word: 19 us).
//   Every row of the gradient is written once, most of them zeros: 131072 x 6144 fp32 from
// 16384 tokens 483 us, 7.1 TB/s (a fill alone 412).  The zeros come from CTAs of their own
// that start one behind the other and write region by region; written by a warp of every
// CTA as bulk copies, all over the table at once, the same took 540, as stores 562.
// 50001 x 2048 from 8191 tokens with the plan: 56 us (floor 35), 12 of them the plan's four
// launches and 4.5 the joins'.  Lookup of 16384 rows of 6144 fp32 to bf16: 47.5 us.
#include "common.cuh"
#include "early.cuh"
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
    bool wide;   // out on a 32-byte boundary
};

// 8 channels as they are stored.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void spread(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void spread(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
// fp32 as one sector where the tensor starts on such a boundary (wide): L2 sees two halves
// of it otherwise.
__device__ __forceinline__ void store8(float* p, const float (&f)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                     "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
        return;
    }
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8], bool) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

constexpr int kLook = 4;   // chunks that a thread has under way

template <typename Tab, typename Out>
__global__ void __launch_bounds__(256) embedding_kernel(const LookupParams p) {
    wait_earlier();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 * kLook + threadIdx.x;
    Chunk<Tab> c[kLook];
    bool there[kLook];
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const int64_t i = i0 + j * 256;
        there[j] = false;
        if (i >= p.total) continue;
        const int64_t t = i / p.chunks;
        const int id = p.ids[t];
        there[j] = id >= 0 && id < p.V;
        if (there[j])
            c[j].load(static_cast<const Tab*>(p.table) + (id * static_cast<int64_t>(p.chunks) + (i - t * p.chunks)) * 8);
        else if (id != -1)
            report_error(p.status, MOE_EINVAL);
    }
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const int64_t i = i0 + j * 256;
        if (i >= p.total) continue;
        float f[8];
        if (there[j]) c[j].spread(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = there[j] ? f[e] * p.scale : 0.0f;
        store8(static_cast<Out*>(p.out) + i * 8, f, p.wide);
    }
}

// ------------------------------------------------------------------ plan

constexpr int kPiece = 32;       // tokens of a piece: one a lane
constexpr int kPlanThreads = 512;
constexpr int kWindow = 1 << 18; // tokens whose bits a CTA holds at once

struct PlanView {
    int32_t* head;    // [0] tokens placed, [1] pieces, [2] scratch rows, [3] words of several
                      // pieces, [4] a small batch's plan, which has no counts
    int32_t* count;   // [V]
    int32_t* start;   // [V] where a word's tokens begin in order
    int2* first;      // [V] its first piece and, where it has several, their first scratch row
    int32_t* rank;    // [T] a token's place among its word's as they came
    int32_t* mixed;   // [T] the tokens by word, as they came
    int32_t* order;   // [T] the tokens of words of several pieces, ascending
    int4* pieces;     // [T] {word, first place, tokens, scratch row or -1}
    int4* joins;      // [T / kPiece] {word, first scratch row, rows, first place}
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
    w.first = reinterpret_cast<int2*>(take(V * 8));
    w.rank = reinterpret_cast<int32_t*>(take(T * 4));
    w.mixed = reinterpret_cast<int32_t*>(take(T * 4));
    w.order = reinterpret_cast<int32_t*>(take(T * 4));
    w.pieces = reinterpret_cast<int4*>(take(T * 16));
    w.joins = reinterpret_cast<int4*>(take((T / kPiece + 1) * 16));
    w.part = reinterpret_cast<float*>(take((2 * (T / kPiece) + 1) * d * 4));
    if (v) *v = w;
    return o;
}

// Exclusive sum over the warp.
__device__ __forceinline__ int warp_before(int v) {
    const int lane = threadIdx.x & 31;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    return incl - v;
}

// What an earlier launch wrote is read past L1, which a launch that waits for it may have
// started with.
//
// The plan's four steps, a launch each: every one is a load or two and an atomic deep, and
// runs over the whole machine.  (One launch of a cluster of 8 CTAs with barriers between the
// steps took 17, 25, 73 and 390 us for 8191, 16384, 65536 and 262144 tokens.)

// Count: a token's rank among its word's as they come.  A warp's tokens of one word ask
// once for all of them (5 us less for the plan of 16384 tokens of one word).
__global__ void __launch_bounds__(kPlanThreads) embedding_count_kernel(const PlanView v, const int32_t* ids,
                                                                       int64_t T, int64_t V, int32_t* status) {
    wait_earlier();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int id = t < T ? ids[t] : -1;
    const bool in = id >= 0 && id < V;
    if (!in && id != -1) report_error(status, MOE_EINVAL);
    const int lane = threadIdx.x & 31;
    const unsigned same = __match_any_sync(0xffffffffu, in ? id : -1);
    const int leader = __ffs(same) - 1;
    int r = 0;
    if (in && lane == leader) r = atomicAdd(v.count + id, __popc(same));
    r = __shfl_sync(0xffffffffu, r, leader) + __popc(same & ((1u << lane) - 1u));
    if (t < T) v.rank[t] = in ? r : -1;
}

// A word's first token gives it its place and its pieces; a CTA asks for all its words.
__global__ void __launch_bounds__(kPlanThreads) embedding_pieces_kernel(const PlanView v, const int32_t* ids,
                                                                        int64_t T) {
    constexpr int W = kPlanThreads / 32;
    __shared__ int sums[3][W], first[3];
    wait_earlier();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const bool mine = t < T && __ldcg(v.rank + t) == 0;
    const int id = mine ? ids[t] : 0;
    const int n = mine ? __ldcg(v.count + id) : 0, np = (n + kPiece - 1) / kPiece, rows = np > 1 ? np : 0;
    int at = warp_before(n), pc = warp_before(np), row = warp_before(rows);
    if (lane == 31) {
        sums[0][wid] = at + n;
        sums[1][wid] = pc + np;
        sums[2][wid] = row + rows;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        int all = 0;
        for (int w = 0; w < W; ++w) {
            const int s = sums[threadIdx.x][w];
            sums[threadIdx.x][w] = all;
            all += s;
        }
        first[threadIdx.x] = all ? atomicAdd(v.head + threadIdx.x, all) : 0;
    }
    __syncthreads();
    at += sums[0][wid] + first[0];
    pc += sums[1][wid] + first[1];
    row += sums[2][wid] + first[2];
    if (!mine || !moe_check(at + n <= T && pc + np <= T, 1621)) return;
    v.start[id] = at;
    v.first[id] = make_int2(pc, row);
    if (np > 1) v.joins[atomicAdd(v.head + 3, 1)] = make_int4(id, row, np, at);
}

// The tokens to their words' places, as they came; every kPiece-th writes a piece.
__global__ void __launch_bounds__(kPlanThreads) embedding_place_kernel(const PlanView v, const int32_t* ids,
                                                                       int64_t T) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    wait_earlier();
    const int id = t < T ? ids[t] : -1;
    const int r = t < T ? __ldcg(v.rank + t) : -1;
    if (r < 0) return;
    const int at = __ldcg(v.start + id) + r;
    if (!moe_check(at < T, 1622)) return;
    v.mixed[at] = static_cast<int32_t>(t);
    if (r % kPiece) return;
    const int n = __ldcg(v.count + id), j = r / kPiece;
    const int2 f = __ldcg(v.first + id);
    if (!moe_check(f.x + j < T, 1629)) return;
    v.pieces[f.x + j] = make_int4(id, at, n - r < kPiece ? n - r : kPiece, n > kPiece ? f.y + j : -1);
}

// Words of several pieces in order (a piece's own order is the gradient's affair where it
// is the word's only one): a word's tokens as bits of a window of the batch, read out from
// its front.
__global__ void __launch_bounds__(kPlanThreads) embedding_order_kernel(const PlanView v, int64_t T) {
    extern __shared__ __align__(16) uint32_t bits[];
    __shared__ int sums[kPlanThreads / 32];
    wait_earlier();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int longs = __ldcg(v.head + 3);
    const int64_t window = T < kWindow ? T : kWindow;
    const int quads = static_cast<int>((window + 127) / 128);   // of words of bits
    const int each = (4 * quads + kPlanThreads - 1) / kPlanThreads;   // words a thread
    const int q0 = static_cast<int>(threadIdx.x) * each, q1 = q0 + each < 4 * quads ? q0 + each : 4 * quads;
    for (int l = blockIdx.x; l < longs; l += gridDim.x) {
        const int4 q = __ldcg(v.joins + l);
        const int n = __ldcg(v.count + q.x);
        int done = 0;
        for (int64_t w0 = 0; w0 < T; w0 += window) {
            for (int i = threadIdx.x; i < quads; i += kPlanThreads)
                reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
#pragma unroll 8
            for (int j = threadIdx.x; j < n; j += kPlanThreads) {
                const int64_t b = __ldcg(v.mixed + q.w + j) - w0;
                if (b >= 0 && b < window && moe_check(b < 128ll * quads, 1623))
                    atomicOr(bits + b / 32, 1u << (b & 31));
            }
            __syncthreads();
            int c = 0;
            for (int i = q0; i < q1; ++i) c += __popc(bits[i]);
            const int before = warp_before(c);
            if (lane == 31) sums[wid] = before + c;
            __syncthreads();
            int to = q.w + done + before;
#pragma unroll
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                if (w < wid) to += sums[w];
                done += sums[w];
            }
            const bool dense = 16ll * n >= window;   // a lane a bit of a neighbour's word, else each its own
            for (int k = 0; k < each; ++k) {
                const int i = q0 + k;
                uint32_t b = i < q1 ? bits[i] : 0;
                const int32_t t = static_cast<int32_t>(w0 + 32ll * i);
                if (!dense) {
                    for (; b; b &= b - 1, ++to)
                        if (moe_check(to < q.w + n, 1624)) v.order[to] = t + __ffs(b) - 1;
                    continue;
                }
                for (unsigned some = __ballot_sync(0xffffffffu, b != 0); some; some &= some - 1) {
                    const int who = __ffs(some) - 1;
                    const uint32_t word = __shfl_sync(0xffffffffu, b, who);
                    const int at = __shfl_sync(0xffffffffu, to, who) + __popc(word & ((1u << lane) - 1u));
                    const int32_t first = __shfl_sync(0xffffffffu, t, who);
                    if ((word >> lane & 1u) && moe_check(at < q.w + n, 1624)) v.order[at] = first + lane;
                }
                to += __popc(b);
            }
            __syncthreads();
        }
    }
}

constexpr int kSmall = 1024;   // tokens of a batch whose plan is one CTA's

// The plan of a small batch in one launch: the tokens sorted by word and token, a thread
// each, by a bitonic network whose near exchanges are a warp's.  (64, 500 and 1000
// tokens: 2.6, 4.9 and 8.4 us, by the steps above 6.8, 11.6 and 10.5.)
__global__ void __launch_bounds__(kSmall) embedding_small_kernel(const PlanView v, const int32_t* ids, int T,
                                                                 int64_t V, int32_t* status) {
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ unsigned long long keys[kSmall];
    __shared__ int begins[32], ends[32], sums[3][32];
    wait_earlier();
    const int i = threadIdx.x, lane = i & 31, wid = i >> 5, P = blockDim.x, warps = P / 32;
    const int id = i < T ? ids[i] : -1;
    const bool in = id >= 0 && id < V;
    if (!in && id != -1) report_error(status, MOE_EINVAL);
    unsigned long long key = in ? static_cast<unsigned long long>(id) << 32 | static_cast<unsigned>(i) : ~0ull;
    for (int size = 2; size <= P; size *= 2) {
        for (int d = size / 2; d > 0; d /= 2) {
            unsigned long long other;
            if (d >= 32) {
                __syncthreads();
                keys[i] = key;
                __syncthreads();
                other = keys[i ^ d];
            } else {
                other = __shfl_xor_sync(kAll, key, d);
            }
            const bool smaller = ((i & d) == 0) == ((i & size) == 0);   // is kept
            key = (key < other) == smaller ? key : other;
        }
    }
    __syncthreads();
    keys[i] = key;
    __syncthreads();
    const bool there = key != ~0ull;
    const int word = static_cast<int>(key >> 32);
    const bool start = there && (i == 0 || static_cast<int>(keys[i - 1] >> 32) != word);
    // a word's tokens stand from begin to end
    const unsigned starts = __ballot_sync(kAll, start), edges = __ballot_sync(kAll, start || !there);
    if (lane == 0) {
        begins[wid] = starts ? 32 * wid + 31 - __clz(starts) : -1;
        ends[wid] = edges ? 32 * wid + __ffs(edges) - 1 : P;
    }
    __syncthreads();
    const unsigned upto = (2u << lane) - 1u, mine = starts & upto, later = edges & ~upto;
    int begin = mine ? 32 * wid + 31 - __clz(mine) : -1, end = later ? 32 * wid + __ffs(later) - 1 : P;
    for (int w = wid - 1; begin < 0 && w >= 0; --w) begin = begins[w];
    for (int w = wid + 1; end == P && w < warps; ++w) end = ends[w];
    const int n = end - begin;
    const bool piece = there && (i - begin) % kPiece == 0, several = n > kPiece;
    const unsigned which[3] = {__ballot_sync(kAll, piece), __ballot_sync(kAll, piece && several),
                               __ballot_sync(kAll, start && several)};
    if (lane < 3) sums[lane][wid] = __popc(lane == 0 ? which[0] : lane == 1 ? which[1] : which[2]);
    __syncthreads();
    int at[3];   // pieces, scratch rows, words of several pieces before this one
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        at[k] = __popc(which[k] & ((1u << lane) - 1u));
        for (int w = 0; w < wid; ++w) at[k] += sums[k][w];
    }
    if (there) v.mixed[i] = v.order[i] = static_cast<int32_t>(key & 0xffffffffu);
    if (piece) v.pieces[at[0]] = make_int4(word, i, end - i < kPiece ? end - i : kPiece, several ? at[1] : -1);
    if (start && several) v.joins[at[2]] = make_int4(word, at[1], (n + kPiece - 1) / kPiece, begin);
    if (i == P - 1) {
        v.head[1] = at[0] + piece;
        v.head[2] = at[1] + (piece && several);
        v.head[3] = at[2] + (start && several);
        v.head[4] = 1;
    }
}

// ------------------------------------------------------------------ gradient

struct GradParams {
    PlanView v;
    int64_t T, V;
    int d, chunks, spans;   // chunks of 8 channels; spans of 512 channels a row
    int accumulate;
    int adders, run;        // CTAs that add up; rows of a CTA of zeros
    bool wide, part_wide;   // dtable, the scratch rows on a 32-byte boundary
    float scale;
    const void* dout;
    void* dtable;
};

constexpr int kSpan = 2;    // chunks a lane of a warp's 512 channels
template <typename In>
constexpr int kRows = sizeof(In) == 2 ? 4 : 2;   // rows that a warp has under way
template <typename In>
constexpr bool kAhead = sizeof(In) == 2;         // an only row is asked for an item ahead (fp32 would spill)

template <typename Tab>
__device__ __forceinline__ void finish(const GradParams& p, Tab* row, int c, float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] *= p.scale;
    if (p.accumulate) {
        Chunk<Tab> was;
        float old[8];
        was.load(row + 8 * c);
        was.spread(old);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += old[e];
    }
    store8(row + 8 * c, s, p.wide);
}

// The lane's token of a piece; the largest number behind the last.
__device__ __forceinline__ int piece_token(const GradParams& p, const int4& q) {
    const int lane = threadIdx.x & 31;
    return lane < q.z ? (q.w < 0 ? p.v.mixed : p.v.order)[q.y + lane] : 0x7fffffff;
}

// One piece's sum over 512 channels.
template <typename In, typename Tab>
__device__ __forceinline__ void add_piece(const GradParams& p, const int4& q, int t, int c0,
                                          const Chunk<In> (&only)[kSpan]) {
    const int lane = threadIdx.x & 31;
    int at = lane;   // the token's place among the piece's
    if (q.w < 0 && q.z > 1) {   // as they came
        at = 0;   // a lane without a token stands behind all: its t is the largest
        for (int j = 0; j < q.z; ++j) {
            const int other = __shfl_sync(0xffffffffu, t, j);
            at += other < t ? 1 : 0;
        }
    }
    float s[kSpan][8];
#pragma unroll
    for (int j = 0; j < kSpan; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[j][e] = 0.0f;
    constexpr int R = kRows<In>;
    if (kAhead<In> && q.z == 1) {
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
            if (c0 + 32 * j < p.chunks) only[j].spread(s[j]);
    } else
    for (int r0 = 0; r0 < q.z; r0 += R) {
        Chunk<In> f[R][kSpan];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int who = __ffs(__ballot_sync(0xffffffffu, at == r0 + k)) - 1;
            const int64_t row = __shfl_sync(0xffffffffu, t, who < 0 ? 0 : who);
            if (r0 + k >= q.z || !moe_check(row < p.T, 1627)) continue;
#pragma unroll
            for (int j = 0; j < kSpan; ++j)
                if (c0 + 32 * j < p.chunks)
                    f[k][j].load(static_cast<const In*>(p.dout) + row * p.d + 8 * (c0 + 32 * j));
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r0 + k >= q.z) break;
#pragma unroll
            for (int j = 0; j < kSpan; ++j) {
                float g[8];
                f[k][j].spread(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[j][e] += g[e];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const int c = c0 + 32 * j;
        if (c >= p.chunks) continue;
        if (q.w >= 0)
            store8(p.v.part + static_cast<int64_t>(q.w) * p.d + 8 * c, s[j], p.part_wide);
        else
            finish(p, static_cast<Tab*>(p.dtable) + static_cast<int64_t>(q.x) * p.d, c, s[j]);
    }
}

constexpr int kAdders = 3;                    // CTAs that add up, an SM
constexpr int64_t kZeros = 128 << 10;         // bytes of rows that a CTA of zeros looks after

// The first CTAs add up the pieces, a span a time, the next item's tokens already loaded,
// and the row where that is one.  Those behind write zeros to the words that do not occur,
// each to a run of rows, so that the machine writes one region after the other.
template <typename In, typename Tab>
__global__ void __launch_bounds__(256, kAdders) embedding_bwd_kernel(const GradParams p) {
    wait_earlier();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) >= p.adders) {
        __shared__ unsigned absent[kZeros / 16 / 32];
        const int64_t r0 = static_cast<int64_t>(blockIdx.x - p.adders) * p.run;
        const int rows = static_cast<int>(p.V - r0 < p.run ? p.V - r0 : p.run);
        const int each = p.d * static_cast<int>(sizeof(Tab)) / 16;   // 16-byte pieces of a row
        uint4* to = static_cast<uint4*>(p.dtable) + r0 * each;
        const bool small = p.v.head[4] != 0;
        for (int i = threadIdx.x; i < (rows + 31) / 32 * 32; i += 256) {
            const unsigned some = __ballot_sync(0xffffffffu, i < rows && (small || p.v.count[r0 + i] == 0));
            if (lane == 0) absent[i >> 5] = some;
        }
        __syncthreads();
        if (small) {
            for (int i = threadIdx.x; i < p.v.head[1]; i += 256) {
                const int64_t r = p.v.pieces[i].x - r0;
                if (r >= 0 && r < rows) atomicAnd(absent + (r >> 5), ~(1u << (r & 31)));
            }
            __syncthreads();
        }
        const int dr = 256 / each, dc = 256 % each;
        int r = static_cast<int>(threadIdx.x) / each, c = static_cast<int>(threadIdx.x) % each;
        while (r < rows) {
            if (absent[r >> 5] >> (r & 31) & 1) to[static_cast<int64_t>(r) * each + c] = make_uint4(0, 0, 0, 0);
            r += dr;
            c += dc;
            if (c >= each) {
                c -= each;
                ++r;
            }
        }
        return;
    }
    const int64_t warps = static_cast<int64_t>(p.adders) * 8;
    const int64_t items = static_cast<int64_t>(p.v.head[1]) * p.spans;
    int64_t it = static_cast<int64_t>(wid) * p.adders + blockIdx.x;
    if (it >= items) return;
    Chunk<In> row[kSpan], row2[kSpan];
    // the tokens of an item, and its row where that is one
    auto fetch = [&](int64_t item, int4& q, int& t, Chunk<In> (&f)[kSpan]) {
        q = p.v.pieces[item / p.spans];
        t = piece_token(p, q);
        if (kAhead<In> && q.z == 1) {
            const int64_t from = __shfl_sync(0xffffffffu, t, 0);
            const int c0 = static_cast<int>(item % p.spans) * 32 * kSpan + lane;
#pragma unroll
            for (int j = 0; j < kSpan; ++j)
                if (c0 + 32 * j < p.chunks && moe_check(from < p.T, 1627))
                    f[j].load(static_cast<const In*>(p.dout) + from * p.d + 8 * (c0 + 32 * j));
        }
    };
    int4 q, q2;
    int t, t2;
    fetch(it, q, t, row);
    while (true) {
        const int64_t then = it + warps;
        if (then < items) fetch(then, q2, t2, row2);
        if (moe_check(q.x >= 0 && q.x < p.V && q.y + q.z <= p.T && q.z <= kPiece, 1628))
            add_piece<In, Tab>(p, q, t, static_cast<int>(it % p.spans) * 32 * kSpan + lane, row);
        if (then >= items) return;
        it = then;
        q = q2;
        t = t2;
#pragma unroll
        for (int j = 0; j < kSpan; ++j) row[j] = row2[j];
    }
}

// Words of several pieces: 32 threads over 256 channels, 8 runs of pieces side by side.
template <typename Tab>
__global__ void __launch_bounds__(256) embedding_join_kernel(const GradParams p) {
    __shared__ float red[8][32][8];
    wait_earlier();   // the pieces' sums are complete
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int wide = (p.chunks + 31) / 32;
    const int64_t items = static_cast<int64_t>(p.v.head[3]) * wide;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t w = it / wide;
        const int c = static_cast<int>(it - w * wide) * 32 + lane;
        const int4 q = p.v.joins[w];
        float s[8] = {};
        if (c < p.chunks)
#pragma unroll 8
            for (int j = run; j < q.z; j += 8) {
                const float4* r = reinterpret_cast<const float4*>(p.v.part + static_cast<int64_t>(q.y + j) * p.d + 8 * c);
                const float4 a = __ldcg(r), b = __ldcg(r + 1);
                s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
                s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
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
    p.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    const int64_t grid = (p.total + 256 * kLook - 1) / (256 * kLook);
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    void (*kern)(LookupParams) =
        c.table_f32 ? (c.out_f32 ? embedding_kernel<float, float> : embedding_kernel<float, uint16_t>)
                    : (c.out_f32 ? embedding_kernel<uint16_t, float> : embedding_kernel<uint16_t, uint16_t>);
    if (const int rc = launch_early(kern, grid, 256, 0, st, p)) return rc;
    trace_after(st, "embedding");
    return MOE_OK;
}

int launch_embedding_plan(int64_t T, int64_t V, int d, const int32_t* ids, void* plan,
                          int32_t* status, cudaStream_t st) {
    PlanView v;
    plan_layout(T, V, d, static_cast<uint8_t*>(plan), &v);
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    if (T <= kSmall) {
        int threads = 32;
        while (threads < T) threads *= 2;
        if (const int rc = launch_early(embedding_small_kernel, 1, threads, 0, st, v, ids, T, V, status)) return rc;
        trace_after(st, "embedding_small");
        return MOE_OK;
    }
    const int64_t counters = reinterpret_cast<uint8_t*>(v.count + V) - reinterpret_cast<uint8_t*>(v.head);
    if (cudaMemsetAsync(v.head, 0, counters, st) != cudaSuccess) return MOE_ECUDA;
    const int64_t grid = (T + kPlanThreads - 1) / kPlanThreads;
    if (const int rc = launch_early(embedding_count_kernel, grid, kPlanThreads, 0, st, v, ids, T, V, status)) return rc;
    trace_after(st, "embedding_count");
    if (const int rc = launch_early(embedding_pieces_kernel, grid, kPlanThreads, 0, st, v, ids, T)) return rc;
    trace_after(st, "embedding_pieces");
    if (const int rc = launch_early(embedding_place_kernel, grid, kPlanThreads, 0, st, v, ids, T)) return rc;
    trace_after(st, "embedding_place");
    const int64_t most = T / (kPiece + 1), ctas = most < 4 * sms ? most : 4 * sms;
    const size_t bits = static_cast<size_t>(((T < kWindow ? T : kWindow) + 127) / 128 * 16);   // at most 32 KB
    if (const int rc = launch_early(embedding_order_kernel, ctas, kPlanThreads, bits, st, v, T)) return rc;
    trace_after(st, "embedding_order");
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
    p.wide = (reinterpret_cast<uintptr_t>(dtable) & 31) == 0;
    p.part_wide = (reinterpret_cast<uintptr_t>(p.v.part) & 31) == 0;
    int64_t need = c.T * p.spans;
    need = (need + 7) / 8;
    const int64_t most = static_cast<int64_t>(sms) * kAdders;
    p.adders = static_cast<int>(need < most ? need : most);
    const int64_t run = kZeros / (static_cast<int64_t>(c.d) * (c.table_f32 ? 4 : 2));
    p.run = static_cast<int>(run < 8 ? 8 : run);
    const int64_t grid = p.adders + (c.accumulate ? 0 : (c.V + p.run - 1) / p.run);
    void (*kern)(GradParams) =
        c.out_f32 ? (c.table_f32 ? embedding_bwd_kernel<float, float> : embedding_bwd_kernel<float, uint16_t>)
                  : (c.table_f32 ? embedding_bwd_kernel<uint16_t, float> : embedding_bwd_kernel<uint16_t, uint16_t>);
    if (const int rc = launch_early(kern, grid, 256, 0, st, p)) return rc;
    trace_after(st, "embedding_bwd");
    if (c.T <= kPiece) return MOE_OK;   // no word has several pieces
    if (const int rc = launch_early(c.table_f32 ? embedding_join_kernel<float> : embedding_join_kernel<uint16_t>,
                                    int64_t{2} * sms, 256, 0, st, p))
        return rc;
    trace_after(st, "embedding_join");
    return MOE_OK;
}

}  // namespace moe
