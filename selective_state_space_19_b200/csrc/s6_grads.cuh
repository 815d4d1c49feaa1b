// s6_grads.cuh -- the global norm of a training step's gradients, and their
// clipping by it, over many tensors in two launches (sm_100a).
//
//     n = sqrt(sum over all tensors and elements of g^2)
//     c = min(1, max_norm / (n + eps)),   g <- c g  where c < 1
//
// A list of tensors is cut into chunks of as many bytes each (the last of a
// tensor may be shorter), and the blocks walk the chunks with a fixed stride, so
// small and large tensors balance and the order of all additions is fixed.  (A
// share of consecutive chunks for each block, which needs no search for the
// tensor, ran 3 % slower: the blocks' reads lie further apart.)  Pointers and
// lengths travel in the kernel's parameters: nothing is copied to the device
// beforehand, and a captured graph holds its own table.
//
// Squares are added up in float32 over 16 elements and in float64 from there.
// Where such a sum has left the range in which float32 squares are exact to
// rounding (an overflow, or elements below 1e-12), the elements are squared
// again in float64: the norm holds for every float32.
//
// The second kernel reads the first one's sums (at most kGradMaxBlocks for
// each 1024 tensors, float64) in every block, in the same order, and scales; it
// walks the chunks from the last to the first, as the last ones read are the
// likeliest to be in L2 still.  Nothing is written where c is 1 or n is 0.
//
// Bound by memory: the gradients are read twice and written once, the second
// read from L2 where they fit.  Measured on one B200 (copies run at 6,521 GB/s):
// 66 tensors of 46 MB 27 us; 132 tensors of 1 GB 486 us, where reading twice and
// writing takes 456.  One 16-byte vector a thread, a warp's next to one another:
// two neighbouring ones left each access with half-used sectors (31 us for the
// 66 tensors).  Four blocks an SM against six and eight: 486, 500, 497 us.
#pragma once

#include <cfloat>

#include "s6_vec.cuh"

namespace s6 {

constexpr int kGradChunkStep = 2048, kGradChunkMost = 16384;  // a chunk: a multiple of the one up to the other
constexpr int kGradThreads = 256;
constexpr int kGradMaxBlocks = 148 * 4;
constexpr int kGradTensors = 1024;  // of one launch; the table is 20 KB of parameters
constexpr int kGradFew = 96;        // a table for short lists

template <int M>
struct GradTable {
    void *ptr[M];       // bit 0 set: bfloat16
    long long n[M];     // elements
    int end[M];         // chunks of the tensors up to and with this one
    int tensors, chunks, chunk;  // chunk: float32 elements of one; of bfloat16, twice as many
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
    const uintptr_t raw = reinterpret_cast<uintptr_t>(t.ptr[lo]);
    GradSpan s;
    s.bf16 = raw & 1u;
    const int most = s.bf16 ? 2 * t.chunk : t.chunk;
    const long long at = static_cast<long long>(chunk - (lo ? t.end[lo - 1] : 0)) * most;
    s.p = reinterpret_cast<void *>((raw & ~static_cast<uintptr_t>(1)) + at * (s.bf16 ? 2 : 4));
    s.n = static_cast<int>(t.n[lo] - at < most ? t.n[lo] - at : most);
    return s;
}

// The sum of 16 squares, four to an accumulator (6 roundings at most).  Between
// 2^-80 and 2^126 the squares that float32 flushed (below 2^-126) are less than
// 2^-42 of the sum; outside, and for NaN, the elements are taken in float64.
__device__ __forceinline__ double square_sum(const float (&f)[16]) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = f[i] * f[i];
#pragma unroll
        for (int j = 4; j < 16; j += 4)
            q[i] = fmaf(f[i + j], f[i + j], q[i]);
    }
    const float s = (q[0] + q[1]) + (q[2] + q[3]);
    if (s >= 0x1p-80f && s <= 0x1p126f)
        return static_cast<double>(s);
    double e = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        e = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), e);
    return e;
}

// A chunk's aligned vectors of 16 bytes, [head, tail) elements, a warp's next to
// one another; fewer than a vector's elements lie before and behind them.
template <typename T>
struct GradChunk {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int B = 16 / V;  // vectors that a thread takes together, kGradThreads apart
    int head, vecs, tail, rest;
    __device__ __forceinline__ GradChunk(const T *p, int n) {
        const int h = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) /
                      static_cast<int>(sizeof(T));
        head = h < n ? h : n;
        vecs = (n - head) / V;
        tail = head + V * vecs;
        rest = n - V * vecs;
    }
    __device__ __forceinline__ int rest_at(int i) const { return i < head ? i : tail + i - head; }
};

template <typename T>
__device__ __forceinline__ double chunk_square_sum(const T *p, int n) {
    constexpr int V = GradChunk<T>::V, B = GradChunk<T>::B;
    using Vec = IoVec<T, V>;
    const GradChunk<T> c(p, n);
    double s = 0.0;
#pragma unroll 2
    for (int k = threadIdx.x; k < c.vecs; k += B * kGradThreads) {
        float f[16];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int at = k + b * kGradThreads;
            const typename Vec::raw r = at < c.vecs ? Vec::load(p + c.head + V * at) : Vec::zero();
            float t[V];
            Vec::unpack(r, t);
#pragma unroll
            for (int i = 0; i < V; ++i)
                f[b * V + i] = t[i];
        }
        s += square_sum(f);
    }
    if (static_cast<int>(threadIdx.x) < c.rest) {
        const double v = static_cast<double>(io_traits<T>::to_f(p[c.rest_at(threadIdx.x)]));
        s = fma(v, v, s);
    }
    return s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(T *p, int n, float scale, float post) {
    constexpr int V = GradChunk<T>::V;
    using Vec = IoVec<T, V>;
    const GradChunk<T> c(p, n);
#pragma unroll 4
    for (int k = threadIdx.x; k < c.vecs; k += kGradThreads) {
        T *at = p + c.head + V * k;
        float f[V];
        Vec::unpack(Vec::load(at), f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = f[i] * scale * post;
        Vec::store(at, Vec::pack(f));
    }
    if (static_cast<int>(threadIdx.x) < c.rest) {
        T *at = p + c.rest_at(threadIdx.x);
        *at = io_traits<T>::from_f(io_traits<T>::to_f(*at) * scale * post);
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
__global__ void __launch_bounds__(kGradThreads, 4) s6_grad_square_kernel(const __grid_constant__ GradTable<M> t,
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
__global__ void __launch_bounds__(kGradThreads, 4) s6_grad_scale_kernel(const __grid_constant__ GradTable<M> t,
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
    // a NaN norm makes c NaN, and every gradient with it; an infinite one makes it 0; gradients
    // that are all zero stay so, with a bound and an eps of 0 too (c is 0 / 0 then)
    float c = a.max_norm / (norm + a.eps), post = 1.0f;
    if (c >= 1.0f || norm == 0.0f)
        return;
    // a factor that float32 holds with fewer digits, or not at all, beside gradients large
    // enough for products that it does hold: 2^64 of it here and 2^-64 behind
    if (c < 0x1p-100f && norm <= FLT_MAX) {
        c = static_cast<float>(static_cast<double>(a.max_norm) /
                               (static_cast<double>(norm) + static_cast<double>(a.eps)) * 0x1p64);
        post = 0x1p-64f;
    }
    for (int k = t.chunks - 1 - static_cast<int>(blockIdx.x); k >= 0; k -= gridDim.x) {
        const GradSpan g = grad_span(t, k);
        if (g.bf16)
            chunk_scale(static_cast<__nv_bfloat16 *>(g.p), g.n, c, post);
        else
            chunk_scale(static_cast<float *>(g.p), g.n, c, post);
    }
}

}  // namespace s6
