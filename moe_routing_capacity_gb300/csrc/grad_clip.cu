// grad_clip.cu -- global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Two passes over the data, bound by its bytes.  The tensors' pieces of
// kChunk elements form one list; a CTA takes every gridDim-th piece.  Pass 1
// sums squares: fp32 within a thread's share of a piece, 64 bits from there
// on, one partial a CTA, so the result does not depend on timing.  Pass 2
// adds the partials in order (each CTA for itself) and scales, walking the
// list from its end: the pieces that pass 1 read last are still in L2.
// The tensor records travel as kernel parameters: no copy to the device, and
// the call can be captured in a graph.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kClipThreads = 512;
constexpr int kChunk = 16384;
constexpr int kMaxCtas = 2 * 160;   // CTAs of a launch, and partials of a batch

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

__device__ __forceinline__ float value(const void* p, int64_t i, bool bf) {
    if (bf)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    return static_cast<const float*>(p)[i];
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
    clip_squares_kernel(const __grid_constant__ ClipBatch<N> b, double* part) {
    __shared__ double red[kClipThreads / 32];
    double total = 0.0;
    const int pieces = b.first[b.n];
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        const int k = tensor_of(b, piece);
        const int64_t at = static_cast<int64_t>(piece - b.first[k]) * kChunk;
        const int64_t left = b.t[k].numel - at;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk;
        const bool bf = b.kind[k] & 1;
        const void* in = b.t[k].in;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (n == kChunk && (b.kind[k] & 2)) {
            if (bf) {
                const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in) + at);
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = v[threadIdx.x + i * kClipThreads];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[i] += bf16_lo(w[e]) * bf16_lo(w[e]);
                        s[i] += bf16_hi(w[e]) * bf16_hi(w[e]);
                    }
                }
            } else {
                const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(in) + at);
                float4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = v[threadIdx.x + i * kClipThreads];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] += x[i].x * x[i].x;
                    s[1] += x[i].y * x[i].y;
                    s[2] += x[i].z * x[i].z;
                    s[3] += x[i].w * x[i].w;
                }
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kClipThreads) {
                const float x = value(in, at + i, bf);
                s[0] += x * x;
            }
        }
        const float sum = (s[0] + s[1]) + (s[2] + s[3]);
        if (sum > 1e-20f && sum < 1e30f) {
            total += sum;
        } else {
            // squares near the ends of fp32's range (or all zero): the same
            // elements' squares again, in 64 bits
            const int per = (b.kind[k] & 2) && n == kChunk ? (bf ? 8 : 4) : 1;
            for (int i = threadIdx.x * per; i < n; i += kClipThreads * per)
                for (int e = 0; e < per; ++e) {
                    const float x = value(in, at + i + e, bf);
                    if (x != 0.f) total += static_cast<double>(x) * x;
                }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kClipThreads / 32; ++i) total += red[i];
        part[blockIdx.x] = total;
    }
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipBatch<N> b, const double* part, int parts,
                      float max_norm, float* norm_out) {
    __shared__ double red[kClipThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are complete
    double total = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) total += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    total = red[0];
    for (int i = 1; i < kClipThreads / 32; ++i) total += red[i];
    const double root = sqrt(total);
    const float norm = static_cast<float>(root);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    // a norm that is not finite leaves the gradients to the caller
    const bool finite = norm <= 3.402823466e38f;
    const double ratio = static_cast<double>(max_norm) / (root + 1e-6);
    const float c = finite && ratio < 1.0 ? static_cast<float>(ratio) : 1.0f;
    const int pieces = b.first[b.n];
    for (int piece = pieces - 1 - static_cast<int>(blockIdx.x); piece >= 0; piece -= gridDim.x) {
        const int k = tensor_of(b, piece);
        const void* in = b.t[k].in;
        void* out = b.t[k].out;
        if (c == 1.0f && in == out) continue;
        const int64_t at = static_cast<int64_t>(piece - b.first[k]) * kChunk;
        const int64_t left = b.t[k].numel - at;
        const int n = left < kChunk ? static_cast<int>(left) : kChunk;
        const bool bf = b.kind[k] & 1;
        if (n == kChunk && (b.kind[k] & 2)) {
            if (bf) {
                const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in) + at);
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = v[threadIdx.x + i * kClipThreads];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16x2(bf16_lo(w[e]) * c, bf16_hi(w[e]) * c);
                    o[threadIdx.x + i * kClipThreads] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(in) + at);
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
                float4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = v[threadIdx.x + i * kClipThreads];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[threadIdx.x + i * kClipThreads] =
                        make_float4(x[i].x * c, x[i].y * c, x[i].z * c, x[i].w * c);
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kClipThreads) {
                const float x = value(in, at + i, bf) * c;
                if (bf)
                    static_cast<uint16_t*>(out)[at + i] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(x));
                else
                    static_cast<float*>(out)[at + i] = x;
            }
        }
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
        at += (t[i].numel + kChunk - 1) / kChunk;
        if (at >= (1ll << 31) - kMaxCtas) return MOE_EINVAL;
    }
    b.first[n] = static_cast<int32_t>(at);
    b.n = static_cast<int>(n);
    return MOE_OK;
}

int grid_for(int pieces, int sms) {
    const int most = 2 * (sms < kMaxCtas / 2 ? sms : kMaxCtas / 2);
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
        if (cudaLaunchKernelEx(&cfg, clip_scale_kernel<N>, b, static_cast<const double*>(part),
                               parts, max_norm, i == 0 ? norm : nullptr) != cudaSuccess)
            return MOE_ECUDA;
        trace_after(st, "clip_scale");
    }
    return MOE_OK;
}

}  // namespace

int64_t grad_clip_ws(int64_t n_tensors) {
    const int64_t batches = n_tensors <= 64 ? 1 : (n_tensors + 511) / 512;
    return batches * kMaxCtas * 8;
}

int launch_grad_clip(const moe_grad_tensor_t* tensors, int64_t n, float max_norm, float* norm,
                     void* ws, cudaStream_t st) {
    int dev = 0, sms = 0;
    if (const int rc = current_device(&dev, &sms)) return rc;
    double* part = static_cast<double*>(ws);
    // few records make a small launch; many tensors few launches
    return n <= 64 ? run<64>(tensors, n, max_norm, norm, part, sms, st)
                   : run<512>(tensors, n, max_norm, norm, part, sms, st);
}

}  // namespace moe
