// attention.cuh -- what the attention kernels share: the plan's layout, TMEM
// loads and stores, MMAs with an A operand in TMEM, and packed fp32 pairs.
#pragma once

#include "common.cuh"

namespace moe {

// ------------------------------------------------------------------ the plan
// Work lists of one batch of packed sequences, in device memory:
//   header   int32[8]: number of entries of each list (q128, kv128, q256), and
//            whether the sequences were refused (the lists are empty then)
//   q128     query blocks of 128 rows, most key blocks first
//   kv128    key blocks of 128 rows, most query blocks first
//   q256     query blocks of 256 rows, most key blocks first
// An entry is {first token of the sequence, its length, block, 0}; block = -1:
// `length` tokens from the first one that belong to no sequence.
struct AttnPlanLayout {
    int64_t max128, max256;             // most entries of a list
    int64_t bins;                       // most blocks of one sequence, + 1
    int64_t q128, kv128, q256, cursor, total;   // byte offsets
};

constexpr int kPlanHeader = 32;
constexpr int kPlanRefused = 3;   // header word

inline AttnPlanLayout attn_plan_layout(int64_t T, int n_seqs) {
    AttnPlanLayout l;
    // whole and partial blocks of the sequences and of the two gaps
    l.max128 = T / 128 + n_seqs + 2;
    l.max256 = T / 256 + n_seqs + 2;
    l.bins = T / 128 + 2;
    l.q128 = kPlanHeader;
    l.kv128 = l.q128 + l.max128 * 16;
    l.q256 = l.kv128 + l.max128 * 16;
    l.cursor = l.q256 + l.max256 * 16;
    l.total = l.cursor + l.bins * 4;
    return l;
}

// A call on refused sequences writes nothing and says so in its own status.
__device__ __forceinline__ void report_refused(const int32_t* header, int32_t* status) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && header[kPlanRefused]) report_error(status, MOE_EINVAL);
}

// Checked builds: an entry of a list of blocks of `rows` rows is one of T tokens.
__device__ __forceinline__ bool plan_entry_ok(const int4& e, int64_t T, int rows) {
    return e.x >= 0 && e.y > 0 && static_cast<int64_t>(e.x) + e.y <= T &&
           (e.z < 0 ? e.z == -1 && e.y <= rows : static_cast<int64_t>(e.z) * rows < e.y);
}

// The items of this CTA, heaviest first: dealt out to the CTAs in turn, every
// other round from the other end, so that a CTA's early heavy item meets a
// lighter one in the next round.
struct AttnItems {
    int total, round = 0;
    __device__ explicit AttnItems(int n) : total(n) {}
    __device__ bool next(int& item) {
        const int g = gridDim.x;
        while (round * g < total) {
            item = round * g + static_cast<int>((round & 1) ? g - 1 - blockIdx.x : blockIdx.x);
            ++round;
            if (item < total) return true;
        }
        return false;
    }
    // of a list of `rows` rows a block and `units` items an entry
    __device__ bool next(int& item, const int4* tiles, int units, int64_t T, int rows, int site) {
        while (next(item))
            if (moe_check(plan_entry_ok(tiles[item / units], T, rows), site)) return true;
        return false;
    }
};

// ------------------------------------------------------------------ TMEM

// 32 consecutive columns, without waiting (tmem_wait_ld before their use).
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The MMA warp runs converged (its waits answer for the whole warp) so that
// addresses and descriptors live in uniform registers; one elected lane
// issues.  Issued from inside `if (lane == 0)`, every MMA first moved its
// operands to uniform registers, about 90 cycles each against the 64 that
// a 128 x 128 x 16 product runs.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}

// D[tmem] (+)= A[smem] B[smem]^T, by the elected lane.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t adesc,
                                       uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
        : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]: A's 128 rows are the TMEM lanes, each 32-bit
// column holds two consecutive K values (the lower half the first).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                       uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
        : "memory");
}

// Arrive once on `bar` when every MMA the elected lane has issued is done.
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(leader)
        : "memory");
}

// A tile of 128 tokens x D channels in shared memory is D / 64 boxes of 128
// rows of 64 channels (16 KB each, 128-byte swizzle, 8-row atoms of 1 KB).
// The same bytes serve as a K-major operand (M/N = tokens, K = channels) and
// as an MN-major one (M/N = channels, 64 of them a box; K = tokens).  The
// descriptors below are those of the tile's start; a step of 16 along K adds
// 32 bytes (within a box) or 2 KB.
constexpr uint32_t kBoxBytes = 16384;
constexpr uint64_t kDescBase = (static_cast<uint64_t>(1024 >> 4) << 32) |
                               (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);

// (The mask: in a cluster, a shared-memory address carries the CTA's rank.)
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return kDescBase | (static_cast<uint64_t>(1) << 16) | ((saddr & 0x3FFFFu) >> 4);
}

__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return kDescBase | (static_cast<uint64_t>(kBoxBytes >> 4) << 16) | ((saddr & 0x3FFFFu) >> 4);
}

// scores[tmem] = A B^T over D channels, both tiles K-major.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t leader, uint32_t d_tmem, uint64_t a,
                                           uint64_t b) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kBoxBytes + (kk % 4) * 32) >> 4;
        mma_ss(leader, d_tmem, a + off, b + off, idesc, kk > 0);
    }
}

// acc[tmem] (+)= A B over tokens 64 half .. 64 half + 63: A bf16, two tokens a
// column, B a tile read MN-major.
template <int D>
__device__ __forceinline__ void mma_tokens(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                           uint64_t b, int half, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, false, true);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const int k16 = 4 * half + kk;   // sixteen tokens
        mma_ts(leader, d_tmem, a_tmem + 8 * k16, b + ((k16 * 2048) >> 4), idesc,
               accumulate || kk > 0);
    }
}

// mbar_wait by a whole warp with one answer for all its lanes: the warp-wide
// TMEM operations that follow never run in part of a warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* status) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, status));
}

// The same for the MMA warp: a wait that is not over at once goes on out of
// line.  The warp shares its instruction cache with warps that run through
// thousands of instructions a block, so its own loop has to be short.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                     int32_t* status) {
    return mbar_wait(bar, parity, abort_flag, status);
}

__device__ __forceinline__ bool warp_wait_short(uint64_t* bar, uint32_t parity,
                                                volatile int* abort_flag, int32_t* status) {
    return __all_sync(0xFFFFFFFFu,
                      mbar_try_wait(bar, parity) || wait_on(bar, parity, abort_flag, status));
}

// acc[tmem] (+)= A B over 128 tokens: A bf16 in four pieces of 32 tokens (16
// columns each, 32 columns apart), B a tile read MN-major.
template <int D>
__device__ __forceinline__ void mma_tokens_quarters(uint32_t leader, uint32_t d_tmem,
                                                    uint32_t a_tmem, uint64_t b, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, false, true);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        mma_ts(leader, d_tmem, a_tmem + (kk / 2) * 32 + (kk % 2) * 8, b + ((kk * 2048) >> 4), idesc,
               accumulate || kk > 0);
}

// Brings the 128-byte line at `p` into L2.  (As bulk prefetches, one a row,
// 384 of them held their warps up for 6000 cycles.)
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// ------------------------------------------------------------------ arithmetic

// Bits i and up of 32, for any i.
__device__ __forceinline__ uint32_t bits_from(int i) {
    return i >= 32 ? 0u : ~0u << max(i, 0);
}

// 2^x (flushing denormal results): the hardware's own exponential, good to 2 units
// of fp32's last place, 2^-14 of the rounding of P to bf16 that follows it.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four lanes of a quad hold a row each, in four 16-byte pieces; afterwards a
// lane holds its own piece of each of the four rows, so that a quad's store
// covers 64 contiguous bytes of a row instead of 16 bytes of four rows.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & s) continue;
            uint4 &a = v[i], &b = v[i + s];
            const uint4 x = up ? a : b;
            uint4 y;
            y.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, s);
            y.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, s);
            y.z = __shfl_xor_sync(0xFFFFFFFFu, x.z, s);
            y.w = __shfl_xor_sync(0xFFFFFFFFu, x.w, s);
            if (up)
                a = y;
            else
                b = y;
        }
    }
}

// 32 columns [col, col + 32) of the warp's 32 rows to global memory as bf16:
// v is this thread's row in four pieces, base the address of the warp's first
// row, rows how many of them exist, D how many columns.
__device__ __forceinline__ void store_quad(uint4 (&v)[4], uint16_t* base, int64_t stride, int rows,
                                           int col, int D) {
    const int lane = threadIdx.x & 31;
    quad_transpose(v);
    const int c = col + 8 * (lane & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = (lane & ~3) + k;
        if (r < rows && c < D) *reinterpret_cast<uint4*>(base + r * stride + c) = v[k];
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float bf16_f32(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ uint16_t f32_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ------------------------------------------------------------------ values that are not finite
//
// The products run over whole blocks: a hidden pair's P and dS are 0, but 0
// times NaN or infinity is NaN.  Hidden pairs stand in the diagonal block (and
// behind a sequence's end, which dK and dV meet in every block of keys).  Where
// the operand that multiplies P or dS there (V, K, dO, Q) holds such a value,
// it becomes 0 in shared memory before the product, and the rows that do see
// it get it back at the end, from memory (*_visible): what a token does not
// see changes no bit of its results, and no row is worked out a second time.
//   The forward has a warp look at V on its way from the copy to the products
// (8192 tokens, 16/4 heads: 78 -> 80 us; by the softmax warps 80 to 84; a second pass,
// only where a result was not finite, 88 for the code it adds to the loops); dQ's
// forming warps look at K while they wait for the scores; dK and dV know from the
// queries' lse and D, which are not finite where Q or dO is not.

// Bits 15 and 31: the word's bf16 halves that are NaN or infinite.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ bool bf16_odd(uint32_t v) { return (v & 0x7F80u) == 0x7F80u; }

__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// Whether this thread's share (the tid-th of `threads`) of a landed tile holds a
// value that is not finite.
template <int D>
__device__ __forceinline__ bool odd_tile(uint32_t tile, int tid, int threads) {
    uint32_t odd = 0;
#pragma unroll 8
    for (uint32_t o = tid * 16; o < 256 * D; o += threads * 16) {
        const uint4 v = ld_shared16(tile + o);
        odd |= odd_halves(v.x) | odd_halves(v.y) | odd_halves(v.z) | odd_halves(v.w);
    }
    return odd != 0;
}

// Such values of the share become 0, for the products too.
template <int D>
__device__ __noinline__ void clean_tile(uint32_t tile, int tid, int threads) {
    const auto keep = [](uint32_t w) { return w & ~((odd_halves(w) >> 15) * 0xFFFFu); };
#pragma unroll 1
    for (uint32_t o = tid * 16; o < 256 * D; o += threads * 16) {
        const uint4 v = ld_shared16(tile + o);
        st_shared16(tile + o, make_uint4(keep(v.x), keep(v.y), keep(v.z), keep(v.w)));
    }
    fence_proxy_async_smem();
}

// Such values of a row of it, by a warp.
template <int D>
__device__ __forceinline__ void clean_row(uint32_t tile, int row) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
        const uint32_t at = tile + b * kBoxBytes + row * 128 + (threadIdx.x & 31) * 4;
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
        w &= ~((odd_halves(w) >> 15) * 0xFFFFu);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
    }
}

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace moe
