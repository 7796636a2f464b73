// grad_clip.cu -- global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Two passes over the data, bound by its bytes: the factor is known only once
// every gradient has been read.  The tensors' pieces form one list, of which a
// CTA takes every gridDim-th (neighbouring CTAs read neighbouring memory).
// Pass 1 sums squares: fp32 within a thread's share of a piece, pairs of fp32
// and 64 bits from there on, one partial a CTA, so the result does not depend
// on timing.  Pass 2 adds the partials in order (each CTA for itself) and
// scales.  The tensor records travel as kernel parameters: no copy to the
// device, and the call can be captured in a graph.
//   180M elements, fp32 and bf16 (708 MB, read twice, written once): 330 us,
// 6.45 TB/s over both passes.  700k elements: 7.1 us on the device, two
// launches.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kClipThreads = 512;
constexpr int kMaxCtas = 160;   // CTAs of a launch (one an SM), and partials of a batch
// Elements of a piece: 32 a thread, eight 16-byte loads of fp32 in flight.
// (Pieces of one load: 180M elements 818 us against 340, 700k 7.9 against 7.1,
// 100k 5.9 against 6.5.)
constexpr int kPiece = 32 * kClipThreads;

struct ClipTensor {
    const void* in;
    void* out;
    int64_t numel;
};

// N tensors a launch: first[i] = the list position of tensor i's first piece.
template <int N>
struct ClipBatch {
    ClipTensor t[N];
    int32_t first[N + 1];
    uint8_t kind[N];       // bit 0: bf16, bit 1: 16-byte aligned in and out
    int n;
};

template <int N>
__device__ __forceinline__ int tensor_of(const ClipBatch<N>& b, int piece) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first[mid] <= piece)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The tensor of `piece`, given an earlier piece's (or -1).
template <int N>
__device__ __forceinline__ int next_tensor(const ClipBatch<N>& b, int k, int piece) {
    if (k < 0) return tensor_of(b, piece);
    while (piece >= b.first[k + 1]) ++k;
    return k;
}

__device__ __forceinline__ float value(const void* p, int64_t i, bool bf) {
    if (bf)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    return static_cast<const float*>(p)[i];
}

// The share of a thread in a piece of n elements from `at`: f(x, count, i) for
// each 16 bytes (4 fp32 or 8 bf16 as x; i the element), or element by element
// where the tensor is not aligned and for the last elements of a tensor.
template <bool BF, class F>
__device__ __forceinline__ void piece_values(const void* in, int64_t at, int n, bool aligned, F f) {
    constexpr int V = BF ? 8 : 4;
    const int vecs = aligned ? n / V : 0;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(in) + at * (BF ? 2 : 4));
    const auto values = [](const uint4& r, float (&x)[V]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (BF) {
                x[2 * e] = bf16_lo(w[e]);
                x[(2 * e + 1) % V] = bf16_hi(w[e]);
            } else {
                x[e] = __uint_as_float(w[e]);
            }
        }
    };
    constexpr int LOADS = kPiece / kClipThreads / V;
    uint4 r[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int k = threadIdx.x + i * kClipThreads;
        if (k < vecs) r[i] = src[k];
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int k = threadIdx.x + i * kClipThreads;
        if (k < vecs) {
            float x[V];
            values(r[i], x);
            f(x, V, k * V);
        }
    }
    for (int i = vecs * V + threadIdx.x; i < n; i += kClipThreads) {
        float x[V];
        x[0] = value(in, at + i, BF);
        f(x, 1, i);
    }
}

// A thread's running sum: a pair of fp32 whose sum carries about 48 bits (a
// 64-bit addition costs 16 cycles a warp here), and 64 bits for what leaves
// fp32's range.
struct SquareSum {
    float hi = 0.f, lo = 0.f;
    double far = 0.0;
    __device__ void add(float v) {   // the exact error of hi + v goes to lo
        const float t = hi + v, b = t - hi;
        lo += (hi - (t - b)) + (v - b);
        hi = t;
    }
    __device__ double value() const { return far + (static_cast<double>(hi) + lo); }
};

// The same elements' squares in 64 bits, for a piece of which the first
// `whole` elements are read 16 bytes a thread.
template <bool BF>
__device__ __noinline__ double far_squares(const void* in, int64_t at, int n, int whole) {
    constexpr int V = BF ? 8 : 4;
    double sum = 0.0;
#pragma unroll 1
    for (int k = threadIdx.x * V; k < whole; k += kClipThreads * V)
#pragma unroll 1
        for (int e = 0; e < V; ++e) {
            const float x = value(in, at + k + e, BF);
            if (x != 0.f) sum += static_cast<double>(x) * x;
        }
#pragma unroll 1
    for (int i = whole + threadIdx.x; i < n; i += kClipThreads) {
        const float x = value(in, at + i, BF);
        sum += static_cast<double>(x) * x;
    }
    return sum;
}

// Squares of this thread's share: fp32 within the piece (64-bit additions cost
// 16 cycles a warp; 32 terms in fp32 lose at most 2^-19 of their sum, half of
// that in the norm); where their sum nears the ends of fp32's range, the same
// elements again in 64 bits.  Down to 1e-30 what squares below fp32's smallest
// normal number lose (32 times 7e-46) is far below the sum's own rounding.
// Zeros are ordinary (experts that met no token): their bits say so, without
// the second look, which takes 100M fp32 elements from 193 to 501 us.
template <bool BF>
__device__ __forceinline__ void piece_squares(const void* in, int64_t at, int n, bool aligned,
                                              SquareSum& total) {
    constexpr int V = BF ? 8 : 4;
    float s[V] = {};
    uint32_t bits = 0;
    piece_values<BF>(in, at, n, aligned, [&](const float (&x)[V], int count, int) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < count) {
                s[e] += x[e] * x[e];
                bits |= __float_as_uint(x[e]);
            }
    });
    if (!(bits << 1)) return;   // zeros of either sign
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) sum += s[e];
    if (sum > 1e-30f && sum < 1e30f) {
        total.add(sum);
        return;
    }
    total.far += far_squares<BF>(in, at, n, aligned ? n / V * V : 0);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 1)
    clip_squares_kernel(const __grid_constant__ ClipBatch<N> b, double* part) {
    __shared__ double red[kClipThreads];
    SquareSum total;
    const int pieces = b.first[b.n];
    int k = -1;
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        k = next_tensor(b, k, piece);
        const int64_t at = static_cast<int64_t>(piece - b.first[k]) * kPiece;
        const int64_t left = b.t[k].numel - at;
        const int n = left < kPiece ? static_cast<int>(left) : kPiece;
        if (!moe_check(k < b.n && at >= 0 && n > 0, 1231)) continue;
        if (b.kind[k] & 1)
            piece_squares<true>(b.t[k].in, at, n, b.kind[k] & 2, total);
        else
            piece_squares<false>(b.t[k].in, at, n, b.kind[k] & 2, total);
    }
    red[threadIdx.x] = total.value();
    __syncthreads();
    if (threadIdx.x < 32) {   // one warp's 64-bit additions instead of sixteen's
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kClipThreads / 32; ++i) sum += red[threadIdx.x + 32 * i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (threadIdx.x == 0) part[blockIdx.x] = sum;
    }
}

template <bool BF>
__device__ __forceinline__ void piece_scale(const void* in, void* out, int64_t at, int n,
                                            bool aligned, float c) {
    constexpr int V = BF ? 8 : 4;
    piece_values<BF>(in, at, n, aligned, [&](const float (&x)[V], int count, int i) {
        if (BF) {
            uint16_t* o = static_cast<uint16_t*>(out) + at + i;
            if (count == 1) {
                *o = __bfloat16_as_ushort(__float2bfloat16_rn(x[0] * c));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(x[2 * e % V] * c, x[(2 * e + 1) % V] * c);
                __stcs(reinterpret_cast<uint4*>(o), make_uint4(w[0], w[1], w[2], w[3]));
            }
        } else {
            float* o = static_cast<float*>(out) + at + i;
            if (count == 1)
                *o = x[0] * c;
            else
                __stcs(reinterpret_cast<float4*>(o),
                       make_float4(x[0] * c, x[1] * c, x[2] * c, x[3] * c));
        }
    });
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 1)
    clip_scale_kernel(const __grid_constant__ ClipBatch<N> b, const double* part, int parts,
                      float max_norm, float* norm_out) {
    __shared__ float scale;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are complete
    if (threadIdx.x < 32) {
        double total = 0.0;
        for (int i = threadIdx.x; i < parts; i += 32) total += part[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        if (threadIdx.x == 0) {
            // the root in fp32 unless the sum leaves its range
            const bool plain = total > 1e-30 && total < 1e38;
            const float norm = plain ? sqrtf(static_cast<float>(total))
                                     : static_cast<float>(sqrt(total));
            if (norm_out && blockIdx.x == 0) *norm_out = norm;
            // a norm that is not finite leaves the gradients to the caller
            const float ratio = max_norm / (norm + 1e-6f);
            scale = norm <= 3.402823466e38f && ratio < 1.0f ? ratio : 1.0f;
        }
    }
    __syncthreads();
    const float c = scale;
    const int pieces = b.first[b.n];
    int k = -1;
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        k = next_tensor(b, k, piece);
        const void* in = b.t[k].in;
        void* out = b.t[k].out;
        if (c == 1.0f && in == out) continue;
        const int64_t at = static_cast<int64_t>(piece - b.first[k]) * kPiece;
        const int64_t left = b.t[k].numel - at;
        const int n = left < kPiece ? static_cast<int>(left) : kPiece;
        if (!moe_check(k < b.n && at >= 0 && n > 0, 1232)) continue;
        if (b.kind[k] & 1)
            piece_scale<true>(in, out, at, n, b.kind[k] & 2, c);
        else
            piece_scale<false>(in, out, at, n, b.kind[k] & 2, c);
    }
}

template <int N>
int fill(ClipBatch<N>& b, const moe_grad_tensor_t* t, int64_t n) {
    int64_t at = 0;
    for (int64_t i = 0; i < n; ++i) {
        const uintptr_t both =
            reinterpret_cast<uintptr_t>(t[i].in) | reinterpret_cast<uintptr_t>(t[i].out);
        b.t[i].in = t[i].in;
        b.t[i].out = t[i].out;
        b.t[i].numel = t[i].numel;
        b.kind[i] = static_cast<uint8_t>((t[i].is_bf16 ? 1 : 0) | ((both & 15) == 0 ? 2 : 0));
        b.first[i] = static_cast<int32_t>(at);
        at += (t[i].numel + kPiece - 1) / kPiece;
        if (at >= (1ll << 31) - kMaxCtas) return MOE_EINVAL;
    }
    b.first[n] = static_cast<int32_t>(at);
    b.n = static_cast<int>(n);
    return MOE_OK;
}

int grid_for(int pieces, int sms) {
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    return pieces < most ? (pieces > 0 ? pieces : 1) : most;
}

// Tensors in batches of N: the squares of every batch, then the scaling.
template <int N>
int run(const moe_grad_tensor_t* t, int64_t n, float max_norm, float* norm, double* part,
        int sms, cudaStream_t st) {
    int parts = 0;
    ClipBatch<N> b;
    for (int64_t i = 0; i < n; i += N) {
        if (const int rc = fill(b, t + i, n - i < N ? n - i : N)) return rc;
        const int g = grid_for(b.first[b.n], sms);
        clip_squares_kernel<N><<<g, kClipThreads, 0, st>>>(b, part + parts);
        if (cudaPeekAtLastError() != cudaSuccess) return MOE_ECUDA;
        trace_after(st, "clip_squares");
        parts += g;
    }
    // the last batch first: it was read last (and needs no second fill)
    for (int64_t i = (n - 1) / N * N; i >= 0; i -= N) {
        if (i + N < n && fill(b, t + i, N)) return MOE_EINVAL;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid_for(b.first[b.n], sms), 1, 1);
        cfg.blockDim = dim3(kClipThreads, 1, 1);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, clip_scale_kernel<N>, b,
                               static_cast<const double*>(part), parts, max_norm,
                               i == 0 ? norm : nullptr) != cudaSuccess)
            return MOE_ECUDA;
        trace_after(st, "clip_scale");
    }
    return MOE_OK;
}

}  // namespace

int check_status_clip() { return moe_check_read_reset(); }

int64_t grad_clip_ws(int64_t n_tensors) {
    const int64_t batches = n_tensors <= 64 ? 1 : (n_tensors + 511) / 512;
    return batches * kMaxCtas * 8;
}

int launch_grad_clip(const moe_grad_tensor_t* tensors, int64_t n, float max_norm, float* norm,
                     void* ws, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    double* part = static_cast<double*>(ws);
    // Few records make a small launch (9 tensors: 7.2 us of the host against 8.3
    // with 512 records), many tensors few launches (300: 29 us against 43).
    return n <= 64 ? run<64>(tensors, n, max_norm, norm, part, sms, st)
                   : run<512>(tensors, n, max_norm, norm, part, sms, st);
}

}  // namespace moe
