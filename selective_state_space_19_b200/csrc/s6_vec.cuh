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

// ------------------------------------------------------- quads of a row
// Four elements of a row in one thread, as two float32 pairs.  V = 4: a vector,
// elements c .. c+3 (c and the row's length multiples of 4, rows aligned to
// vectors).  V = 1: the elements c, c + S, c + 2S, c + 3S.  Elements from n on
// are not touched and read as zero; `all`, a constant where it is used, says that
// there are none.
template <typename T, int V>
struct Quad {
    using Vec = IoVec<T, V>;
    typename Vec::raw r[4 / V];

    __device__ __forceinline__ void load(const T *p, bool all, int c, int S, int n) {
#pragma unroll
        for (int i = 0; i < 4 / V; ++i)
            r[i] = all || c + i * S < n ? Vec::load(p + c + i * S) : Vec::zero();
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4 / V; ++i)
            r[i] = Vec::zero();
    }
    __device__ __forceinline__ void pairs(f2_t (&q)[2]) const {
        if constexpr (sizeof(T) == 2 && V == 4) {
            // bfloat16 to float32: its bits are the top half
            q[0] = f2_pack(__uint_as_float(r[0].x << 16), __uint_as_float(r[0].x & 0xffff0000u));
            q[1] = f2_pack(__uint_as_float(r[0].y << 16), __uint_as_float(r[0].y & 0xffff0000u));
        } else if constexpr (V == 4) {
            q[0] = f2_pack(__uint_as_float(r[0].x), __uint_as_float(r[0].y));
            q[1] = f2_pack(__uint_as_float(r[0].z), __uint_as_float(r[0].w));
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                q[i] = f2_pack(__uint_as_float(static_cast<uint32_t>(r[2 * i]) << 16),
                               __uint_as_float(static_cast<uint32_t>(r[2 * i + 1]) << 16));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                q[i] = f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        }
    }
    static __device__ __forceinline__ void store(T *p, bool all, int c, int S, int n, const f2_t (&q)[2]) {
        float f[4];
        f2_unpack(q[0], f[0], f[1]);
        f2_unpack(q[1], f[2], f[3]);
        if constexpr (V == 4) {
            if (all || c < n)
                Vec::store(p + c, Vec::pack(f));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (all || c + i * S < n)
                    p[c + i * S] = io_traits<T>::from_f(f[i]);
        }
    }
};

// A value where the quad's elements are below n, 0 elsewhere.
template <int V>
__device__ __forceinline__ void quad_where(float v, bool all, int c, int S, int n, f2_t (&q)[2]) {
    if (all) {
        q[0] = q[1] = f2_pack(v, v);
    } else if constexpr (V == 4) {
        q[0] = q[1] = c < n ? f2_pack(v, v) : f2_pack(0.0f, 0.0f);
    } else {
        q[0] = f2_pack(c < n ? v : 0.0f, c + S < n ? v : 0.0f);
        q[1] = f2_pack(c + 2 * S < n ? v : 0.0f, c + 3 * S < n ? v : 0.0f);
    }
}

__device__ __forceinline__ f2_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(f2_t a, f2_t b) {
    float x, y;
    f2_unpack(f2_add(a, b), x, y);
    return x + y;
}

// ------------------------------------------------- rows into shared memory
// Shared bytes that rows of n bytes in all may take: they keep their place within 16 bytes.
__host__ __device__ constexpr int row_buffer_bytes(long long n) { return static_cast<int>((n + 15) / 16 * 16 + 16); }

// The place of an address within 16 bytes; that of element `at` of a tensor.
__device__ __forceinline__ int in16(const void *p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u); }
template <typename T>
__device__ __forceinline__ int in16(const T *p, long long at) {
    return static_cast<int>((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) +
                             static_cast<uint32_t>(at) * static_cast<uint32_t>(sizeof(T))) & 15u);
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// Starts the bulk copy of the stretch [a, a + n) of a tensor's memory [begin, end)
// into buf and adds its bytes to what `bar` expects (the caller arrives).  A bulk copy begins
// and ends on 16-byte boundaries of global memory: the stretch keeps its place
// within 16 bytes (a lands at buf + a % 16), and the up to 15 bytes around it
// that come along are its neighbours in the tensor.  Where the tensor itself
// begins or ends off a boundary, the copy stays inside it and the few elements
// between are moved singly, by this thread.
template <typename T>
__device__ __forceinline__ void bulk_fetch(unsigned char *buf, uintptr_t a, uint32_t n, uintptr_t begin,
                                           uintptr_t end, uint64_t *bar) {
    const uintptr_t base = a & ~static_cast<uintptr_t>(15), b = a + n;
    uintptr_t lo = base, hi = (b + 15) & ~static_cast<uintptr_t>(15);
    if (lo < begin || hi > end) {
        if (lo < begin)
            lo += 16;
        if (hi > end)
            hi -= 16;
        if (hi <= lo)
            lo = hi = b;  // all of it singly
        for (uintptr_t p = a; p < lo; p += sizeof(T))
            *reinterpret_cast<T *>(buf + (p - base)) = *reinterpret_cast<const T *>(p);
        for (uintptr_t p = hi > a ? hi : a; p < b; p += sizeof(T))
            *reinterpret_cast<T *>(buf + (p - base)) = *reinterpret_cast<const T *>(p);
        fence_proxy_async_smem();  // these stores before a later step's copy into the same bytes
        if (hi == lo)
            return;
    }
    const uint32_t bytes = static_cast<uint32_t>(hi - lo);
    mbar_expect_tx(bar, bytes);
    bulk_load(buf + (lo - base), reinterpret_cast<const void *>(lo), bytes, bar);
}

constexpr uint32_t kBulkPolls = 1u << 22;  // bound of a wait for a copy, far above any that arrives
constexpr unsigned int kErrTrainCopy = 16u;  // bit of the device error word: such a wait gave up

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Two sums over a warp in one walk: lanes 0-15 go on with the first, 16-31 with
// the second, and every lane receives both.
__device__ __forceinline__ void warp_sum2(float &a, float &b) {
    const bool low = (threadIdx.x & 16) == 0;
    float v = low ? a : b;
    v += __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// N sums (1, 2 or 4) over a block of WARPS warps (4, 8 or 16), in every thread
// and in a fixed order.  The walk over a warp halves the number of sums a lane
// carries with each of its first steps; the second walk, over the warps' slots,
// is made by every warp.  `any`: ORed over the block.  One barrier; `slots` must
// not be in use by readers of an earlier call (see the callers).
template <int N, int WARPS>
__device__ __forceinline__ bool block_sums(float (&v)[N], float (&slots)[4][16], bool any) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float t;
    if constexpr (N == 4) {
        const bool low = (lane & 16) == 0, lo8 = (lane & 8) == 0;
        float a = low ? v[0] : v[2], b = low ? v[1] : v[3];
        a += __shfl_xor_sync(0xffffffffu, low ? v[2] : v[0], 16);
        b += __shfl_xor_sync(0xffffffffu, low ? v[3] : v[1], 16);
        t = lo8 ? a : b;
        t += __shfl_xor_sync(0xffffffffu, lo8 ? b : a, 8);
    } else if constexpr (N == 2) {
        const bool low = (lane & 16) == 0;
        t = low ? v[0] : v[1];
        t += __shfl_xor_sync(0xffffffffu, low ? v[1] : v[0], 16);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
    } else {
        t = v[0];
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        t += __shfl_xor_sync(0xffffffffu, t, o);
    constexpr int span = 32 / N;  // lanes that carry one sum
    if (lane % span == 0)
        slots[lane / span][warp] = t;
    const bool bad = __syncthreads_or(any);
    // lane l of every warp takes slots l % span, l % span + span, ... of sum l / span
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; k += span)
        if (k + lane % span < WARPS)
            t += slots[lane / span][k + lane % span];
#pragma unroll
    for (int o = (span < WARPS ? span : WARPS) / 2; o > 0; o >>= 1)
        t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = __shfl_sync(0xffffffffu, t, k * span);
    return bad;
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
// would not): four rows in float32, and those in float64.  Segment `seg` of column c goes to out0[c * segs0 + seg] for
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
    __shared__ double sh[kSumPartsWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long n = static_cast<long long>(a.cols) * a.segs;
    const long long i = static_cast<long long>(blockIdx.x) * 32 + lane;
    cudaGridDependencySynchronize();
    double s = 0.0;
    if (i < n) {
        const float *p = a.part + i;
        int r = warp;
        for (; r + 3 * kSumPartsWarps < a.rows; r += 4 * kSumPartsWarps) {
            const float v0 = p[r * n], v1 = p[(r + kSumPartsWarps) * n], v2 = p[(r + 2 * kSumPartsWarps) * n],
                        v3 = p[(r + 3 * kSumPartsWarps) * n];
            s += static_cast<double>((v0 + v1) + (v2 + v3));
        }
        for (; r < a.rows; r += kSumPartsWarps)
            s += static_cast<double>(p[r * n]);
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < n) {
        double sum = 0.0;
#pragma unroll
        for (int w = 0; w < kSumPartsWarps; ++w)
            sum += sh[w][lane];
        const float t = static_cast<float>(sum);
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
