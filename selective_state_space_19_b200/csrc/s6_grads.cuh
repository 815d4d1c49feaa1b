// s6_grads.cuh -- the global norm of a training step's gradients, and their
// clipping by it, over many tensors in two launches (sm_100a).
//
//     n = sqrt(sum over all tensors and elements of g^2)
//     c = min(1, max_norm / (n + eps)),   g <- c g  where c < 1
//
// A list of tensors is cut into chunks of kGradChunkSmall or -Large elements of
// one tensor each; blocks walk the chunks with a fixed stride, so small and large tensors
// balance and the order of all additions is fixed.  Pointers and lengths travel
// in the kernel's parameters: nothing is copied to the device beforehand, and a
// captured graph holds its own table.
//
// Squares are added up in float32 over the 8 elements of one or two loads and
// in float64 from there.  Where such a group's sum has left the range in which
// float32 squares are exact to rounding (an overflow, or elements below 1e-15),
// the group is squared again in float64: the norm holds for every float32.
//
// The second kernel reads the first one's sums (at most kGradMaxBlocks for
// each 1024 tensors, float64) in every block, in the same order, and scales; it
// walks the chunks from the last to the first, as the last ones read are the
// likeliest to be in L2 still.  Nothing is written where c is 1.
#pragma once

#include "s6_vec.cuh"

namespace s6 {

constexpr int kGradChunkSmall = 4096, kGradChunkLarge = 16384;
constexpr int kGradThreads = 256;
constexpr int kGradMaxBlocks = 148 * 6;
constexpr int kGradTensors = 1024;  // of one launch; the table is 17 KB of parameters
constexpr int kGradFew = 96;        // a table for short lists

template <int M>
struct GradTable {
    void *ptr[M];       // bit 0 set: bfloat16
    long long n[M];     // elements
    int end[M];         // chunks of the tensors up to and with this one
    int tensors, chunks, chunk;  // chunk: elements of one
};

struct GradScaleArgs {
    const double *part;  // the sums, or null where the norm is given
    int parts;
    const float *norm_in;
    float *norm_out;  // written by block 0; may be null
    float max_norm, eps;
};

struct GradSpan {
    void *p;    // first element of the chunk
    int n;      // its elements
    bool bf16;
};

template <int M>
__device__ __forceinline__ GradSpan grad_span(const GradTable<M> &t, int chunk) {
    int lo = 0, hi = t.tensors - 1;  // the first tensor whose end is above chunk
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.end[mid] > chunk)
            hi = mid;
        else
            lo = mid + 1;
    }
    const long long at = static_cast<long long>(chunk - (lo ? t.end[lo - 1] : 0)) * t.chunk;
    const uintptr_t raw = reinterpret_cast<uintptr_t>(t.ptr[lo]);
    GradSpan s;
    s.bf16 = raw & 1u;
    s.p = reinterpret_cast<void *>((raw & ~static_cast<uintptr_t>(1)) + at * (s.bf16 ? 2 : 4));
    s.n = static_cast<int>(t.n[lo] - at < t.chunk ? t.n[lo] - at : t.chunk);
    return s;
}

// The sum of squares of 8 elements.  Between 2^-80 and 2^126 the squares that
// float32 flushed (below 2^-126) are less than 2^-43 of the sum; outside, and
// for NaN, the elements are taken in float64.  A group of zeros stays here.
__device__ __forceinline__ double square_sum8(const float (&f)[8]) {
    float s0 = f[0] * f[0], s1 = f[1] * f[1];
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s0 = fmaf(f[i], f[i], s0);
        s1 = fmaf(f[i + 1], f[i + 1], s1);
    }
    const float s = s0 + s1;
    if (s >= 0x1p-80f && s <= 0x1p126f)
        return static_cast<double>(s);
    double e = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), e);
    return e;
}

// The part of a chunk whose vectors of 16 bytes are aligned: [head, head + 8 groups) elements.
template <typename T>
__device__ __forceinline__ int grad_head(const T *p, int n) {
    const int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / static_cast<int>(sizeof(T));
    return head < n ? head : n;
}

template <typename T>
__device__ __forceinline__ void grad_load8(const T *p, float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        float a[4], b[4];
        const auto r0 = IoVec<T, 4>::load(p), r1 = IoVec<T, 4>::load(p + 4);
        IoVec<T, 4>::unpack(r0, a);
        IoVec<T, 4>::unpack(r1, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        IoVec<T, 8>::unpack(IoVec<T, 8>::load(p), f);
    }
}

template <typename T>
__device__ __forceinline__ void grad_store8(T *p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = f[i];
            b[i] = f[4 + i];
        }
        IoVec<T, 4>::store(p, IoVec<T, 4>::pack(a));
        IoVec<T, 4>::store(p + 4, IoVec<T, 4>::pack(b));
    } else {
        IoVec<T, 8>::store(p, IoVec<T, 8>::pack(f));
    }
}

template <typename T>
__device__ __forceinline__ double chunk_square_sum(const T *p, int n) {
    const int head = grad_head(p, n), groups = (n - head) >> 3, tail = head + 8 * groups;
    double s = 0.0;
#pragma unroll 4
    for (int k = threadIdx.x; k < groups; k += kGradThreads) {
        float f[8];
        grad_load8(p + head + 8 * k, f);
        s += square_sum8(f);
    }
    // fewer than 8 elements before the first vector and fewer than 8 behind the last
    const int rest = head + (n - tail);
    if (static_cast<int>(threadIdx.x) < rest) {
        const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : tail + threadIdx.x - head;
        const double v = static_cast<double>(io_traits<T>::to_f(p[i]));
        s = fma(v, v, s);
    }
    return s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(T *p, int n, float c) {
    const int head = grad_head(p, n), groups = (n - head) >> 3, tail = head + 8 * groups;
#pragma unroll 4
    for (int k = threadIdx.x; k < groups; k += kGradThreads) {
        float f[8];
        grad_load8(p + head + 8 * k, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] *= c;
        grad_store8(p + head + 8 * k, f);
    }
    const int rest = head + (n - tail);
    if (static_cast<int>(threadIdx.x) < rest) {
        const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : tail + threadIdx.x - head;
        p[i] = io_traits<T>::from_f(io_traits<T>::to_f(p[i]) * c);
    }
}

// The sum of v over the block, in every thread (two barriers).
__device__ __forceinline__ double grad_block_sum(double v, double *sh) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i)
        v += sh[i];
    return v;
}

template <int M>
__global__ void __launch_bounds__(kGradThreads, 6) s6_grad_square_kernel(const __grid_constant__ GradTable<M> t,
                                                                     double *part) {
    __shared__ double sh[kGradThreads / 32];
    cudaTriggerProgrammaticLaunchCompletion();
    double s = 0.0;
    for (int k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const GradSpan g = grad_span(t, k);
        s += g.bf16 ? chunk_square_sum(static_cast<const __nv_bfloat16 *>(g.p), g.n)
                    : chunk_square_sum(static_cast<const float *>(g.p), g.n);
    }
    s = grad_block_sum(s, sh);
    if (threadIdx.x == 0)
        part[blockIdx.x] = s;
}

template <int M>
__global__ void __launch_bounds__(kGradThreads, 6) s6_grad_scale_kernel(const __grid_constant__ GradTable<M> t,
                                                                    const GradScaleArgs a) {
    __shared__ double sh[kGradThreads / 32];
    cudaGridDependencySynchronize();
    float norm;
    if (a.part) {
        double s = 0.0;
        for (int k = threadIdx.x; k < a.parts; k += kGradThreads)
            s += a.part[k];
        norm = static_cast<float>(sqrt(grad_block_sum(s, sh)));
    } else {
        norm = *a.norm_in;
    }
    if (a.norm_out && blockIdx.x == 0 && threadIdx.x == 0)
        *a.norm_out = norm;
    // a NaN norm makes c NaN, and every gradient with it; an infinite one makes it 0
    const float c = a.max_norm / (norm + a.eps);
    if (c >= 1.0f)
        return;
    for (int k = t.chunks - 1 - static_cast<int>(blockIdx.x); k >= 0; k -= gridDim.x) {
        const GradSpan g = grad_span(t, k);
        if (g.bf16)
            chunk_scale(static_cast<__nv_bfloat16 *>(g.p), g.n, c);
        else
            chunk_scale(static_cast<float *>(g.p), g.n, c);
    }
}

}  // namespace s6
