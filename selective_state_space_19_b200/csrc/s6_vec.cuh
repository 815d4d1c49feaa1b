// s6_vec.cuh -- vectors of I/O elements moved as one load or store (sm_100a),
// and the fixed-order reductions the training-step kernels share.
#pragma once

#include "s6_common.cuh"

namespace s6 {

// BYTES of consecutive elements in registers, as one memory access moves them.
template <int BYTES>
struct raw_bytes;
template <>
struct raw_bytes<2> {
    using type = unsigned short;
};
template <>
struct raw_bytes<4> {
    using type = uint32_t;
};
template <>
struct raw_bytes<8> {
    using type = uint2;
};
template <>
struct raw_bytes<16> {
    using type = uint4;
};

template <typename T, int V>
struct IoVec {
    using raw = typename raw_bytes<sizeof(T) * V>::type;

    static __device__ __forceinline__ raw load(const T *p) { return *reinterpret_cast<const raw *>(p); }
    static __device__ __forceinline__ void store(T *p, raw r) { *reinterpret_cast<raw *>(p) = r; }
    static __device__ __forceinline__ raw zero() {
        raw r;
        if constexpr (sizeof(raw) == 16)
            r = make_uint4(0u, 0u, 0u, 0u);
        else if constexpr (sizeof(raw) == 8)
            r = make_uint2(0u, 0u);
        else
            r = 0;
        return r;
    }
    static __device__ __forceinline__ void unpack(const raw &r, float (&f)[V]) {
        union {
            raw r;
            T t[V];
        } u;
        u.r = r;
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = io_traits<T>::to_f(u.t[i]);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[V]) {
        union {
            raw r;
            T t[V];
        } u;
#pragma unroll
        for (int i = 0; i < V; ++i)
            u.t[i] = io_traits<T>::from_f(f[i]);
        return u.r;
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------- sums over blocks' partials
// The gradients of parameters are sums over rows that many blocks share.  Each
// block writes its sums, part[row][seg][c] (seg < segs, c < cols), and this
// kernel adds them up in a fixed order, so results repeat bit for bit (atomics
// would not).  Segment `seg` of column c goes to out0[c * segs0 + seg] for
// seg < segs0, and to out1[c] for seg = segs0; a null output is not wanted.
// A block owns 32 columns; warp w adds rows w, w + 16, ... and the 16 sums
// are added in order of w.  The partials of one call are a few MB at most and
// come from L2.
struct SumPartsArgs {
    const float *part;
    int rows, cols, segs, segs0;
    float *out0, *out1;
};

constexpr int kSumPartsWarps = 16;

__global__ void __launch_bounds__(32 * kSumPartsWarps) s6_sum_parts_kernel(const SumPartsArgs a) {
    __shared__ float sh[kSumPartsWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long n = static_cast<long long>(a.cols) * a.segs;
    const long long i = static_cast<long long>(blockIdx.x) * 32 + lane;
    cudaGridDependencySynchronize();
    float s = 0.0f;
    if (i < n) {
        const float *p = a.part + i;
        int r = warp;
        for (; r + 3 * kSumPartsWarps < a.rows; r += 4 * kSumPartsWarps) {
            const float v0 = p[r * n], v1 = p[(r + kSumPartsWarps) * n], v2 = p[(r + 2 * kSumPartsWarps) * n],
                        v3 = p[(r + 3 * kSumPartsWarps) * n];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; r < a.rows; r += kSumPartsWarps)
            s += p[r * n];
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < n) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumPartsWarps; ++w)
            t += sh[w][lane];
        const int seg = static_cast<int>(i / a.cols), c = static_cast<int>(i - static_cast<long long>(seg) * a.cols);
        if (seg < a.segs0) {
            if (a.out0)
                a.out0[static_cast<long long>(c) * a.segs0 + seg] = t;
        } else if (a.out1) {
            a.out1[c] = t;
        }
    }
}

}  // namespace s6
