// s6_norm.cuh -- LayerNorm over the rows of a residual stream, forward (with the
// residual add in front of it) and backward, sm_100a.
//
// "mamba, live" (what is actually running): each block reads LayerNorm(x) and
// adds its output to x.  Biased variance, weight and bias.  Of a row of W
// elements:
//
//     s = x + r (r: the branch's output, or nothing)
//     m = sum(s) / W,   q = 1 / sqrt(sum((s - m)^2) / W + eps)
//     y = (s - m) q w + b
//
// A float32 sum times a rounded 1/W leaves m off by a few roundings of |m|: nothing
// where |m| is at most the deviations' root mean square, but a row of the constant
// 100 came out up to 5e-3 off by it, and rows at 1000 +- 0.01 up to 2e-2.  Where m is
// larger ("far"), the deviations d from that first m are summed up too, and what m
// was off by, c = sum(d) / W, is taken out:
//
//     sum((s - m)^2) / W = sum(d^2) / W - c^2,   y = (d - c) q w + b,   m = first m + c
//
// Far rows pay for a third reduction; in every row it cost 2 % on average and 5 to
// 20 % of narrow and bfloat16 ones.  (The backward's h goes by the m that was stored,
// a float32: of rows at 1000 +- 0.01 it is off by up to 3e-3.)
//
//     h = (s - m) q,    g = w dy
//     dx = ds + q (g - sum(g)/W - h sum(g h)/W)        ds: the gradient that
//     dw = sum over rows of dy h,  db = of dy          reaches s past the norm
//
// Both are bound by HBM: a row is read once, in the storage type, and
// everything is computed in float32 from there.  Three forms, by the width:
//
//  * up to kNormWarpWidth: a row is one warp's (up to 64 elements 16, 8, 4 or
//    2 lanes'), in its registers.  The warp walks rows with a fixed stride and
//    fetches the next one while it reduces the present one.
//  * up to kNormMaxWidth: rows come through shared memory, copied ahead of
//    their use without registers, and a block takes two of them at a time.
//  * above that: the _wide kernels, which read a row more than once.
//
// Measured on one B200 (copies run at 6,521 GB/s): 131072 rows of 384, a float32
// stream and a bfloat16 branch: forward with the add 99 us = 94 % of the copy
// rate, backward with the residual gradient 112 us = 96 %.  Wide rows: 8192x2560
// f32 32 us forward and 47 backward (81, 82 %), bfloat16 21 and 41 (63, 63 %:
// bound by issue, 18 and 30 instructions an element), 8191x2561 bfloat16 25 and 42
// (52, 62 %).  Where the block's capacity is not the row's (768 of 1024 columns):
// 32768x768 bfloat16 37 and 49 (42, 63 %), f32 39 and 55 (79, 85 %).  Narrow rows,
// a chain of load, reductions and store with little to overlap: 131072x64 f32 14 and
// 28 (72, 56 %), bfloat16 14 and 24 (36, 44 %).  The _wide forms: 4096x16384 f32 147
// and 224 (56, 55 %), bfloat16 123 and 167 (33, 49 %).
//
// Vectors of 4 elements where the rows begin on one, else single elements:
// rows of an odd width start anywhere, and the copies into shared memory keep
// their place within 16 bytes.
#pragma once

#include <type_traits>

#include "s6_vec.cuh"

namespace s6 {

constexpr int kNormWarpWidth = 512;  // widest row of one warp's registers: 16 elements a lane
constexpr int kNormBlockWarps = 4;   // warps (rows in flight) of a block of such rows
constexpr int kNormMaxWidth = 8192;  // widest row that passes through shared memory

// Warps of one-warp rows resident on an SM, by the elements that a lane holds:
// what the registers allow (the launch bounds hold the compiler to it).
__host__ __device__ constexpr int norm_warps_resident(int elems, bool bwd) {
    return bwd ? (elems <= 4 ? 24 : elems <= 8 ? 20 : elems <= 12 ? 16 : 12)
               : (elems <= 4 ? 32 : elems <= 8 ? 28 : elems <= 12 ? 20 : 16);
}

struct NormFwdArgs {
    long long rows;
    int width;
    float eps, inv_w;
    const void *x, *r;  // r may be null
    const float *w, *b; // may be null (ones, zeros)
    void *s, *y;        // s may be null; it may be x
    float *mean, *rstd; // may be null
};

struct NormBwdArgs {
    long long rows;
    int width;
    float inv_w;
    const void *x, *dy;
    const float *mean, *rstd, *w;  // w may be null
    const float *ds;               // may be null; may be dx
    float *dx;
    float *part;  // [blocks][2][width]: the block's dw and db; null = neither is wanted
};

// The sum of v over G neighbouring lanes, in each of them.  Rows of up to 64
// elements share a warp; its groups may part company at the last rows, so only
// the group's own lanes take part.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    const unsigned int mask = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (threadIdx.x & 31 & ~(G - 1));
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(mask, v, o);
    return v;
}

// A quad of parameters (all `def` where p is null); 0 from n on.
template <int V>
__device__ __forceinline__ void quad_params(const float *p, float def, int c, int S, int n, f2_t (&q)[2]) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = V == 4 ? c + i : c + i * S;
        f[i] = at < n ? (p ? p[at] : def) : 0.0f;
    }
    q[0] = f2_pack(f[0], f[1]);
    q[1] = f2_pack(f[2], f[3]);
}

// Whether a row's mean is large next to its deviations; sq: the mean of their squares.
__device__ __forceinline__ bool norm_far(float mean, float sq) { return mean * mean > sq; }

// The mean of the squares where the mean is taken `off` further on.  NaN stays NaN, and
// squares that overflowed stay infinite (for a rstd of 0).
__device__ __forceinline__ float norm_moved(float sq, float off) {
    const float var = fmaf(-off, off, sq);
    return var < 0.0f ? 0.0f : var;
}

constexpr int kNormWideThreads = 512;
constexpr int kNormWideBlocks = 4;  // of them on an SM

// The sum of v over a block of kNormWideThreads, through `red` (one slot a warp).
// Every thread adds the slots in the same order.
__device__ __forceinline__ float wide_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormWideThreads / 32; ++i)
        v += red[i];
    return v;
}

// A block's walk over a row of W elements: f(c, a, b) adds columns c .. c + V - 1 to two sums.
// A thread's float32 sums run over kNormWideRun vectors at most and are then added to
// a0 and b0 (of 2^24 columns it has 8,192 vectors).  U of them are in flight: four, or
// two of the backward's two vectors (four would spill).
constexpr int kNormWideRun = 64;

template <int V, int U, typename F>
__device__ __forceinline__ void wide_walk(int W, F f, float &a0, float &b0) {
    for (int c = threadIdx.x * V; c < W;) {
        const int span = kNormWideRun * kNormWideThreads * V, stop = W - c < span ? W : c + span;
        float a = 0.0f, b = 0.0f;
#pragma unroll U
        for (; c < stop; c += kNormWideThreads * V)
            f(c, a, b);
        a0 += a;
        b0 += b;
    }
}

template <typename X, typename Y, int V, int NQ, int G>
__global__ void __launch_bounds__(32 * kNormBlockWarps, norm_warps_resident(4 * NQ, false) / kNormBlockWarps)
    s6_layernorm_fwd_kernel(const NormFwdArgs a) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    constexpr int kRows = 32 / G * kNormBlockWarps;  // of a block
    const int lane = threadIdx.x % G, W = a.width;
    auto col = [&](int j) { return lane * V + 4 * G * j; };  // of quad j; only the last can pass the row's end
    f2_t wv[NQ][2], bv[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), G, W, wv[j]);
        quad_params<V>(a.b, 0.0f, col(j), G, W, bv[j]);
    }

    const long long step = static_cast<long long>(kRows) * gridDim.x;
    long long row = static_cast<long long>(kRows) * blockIdx.x + threadIdx.x / G;
    const X *x = static_cast<const X *>(a.x);
    const Y *r = static_cast<const Y *>(a.r);
    X *s = static_cast<X *>(a.s);
    Y *y = static_cast<Y *>(a.y);
    QX xr[NQ];
    QY rr[NQ];
    auto fetch = [&](long long at) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            xr[j].load(x + at * W, j + 1 < NQ, col(j), G, W);
            if (r)
                rr[j].load(r + at * W, j + 1 < NQ, col(j), G, W);
        }
    };
    if (row < a.rows)
        fetch(row);
    for (; row < a.rows; row += step) {
        f2_t v[NQ][2], t0 = f2_both(0.0f), t1 = t0;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            xr[j].pairs(v[j]);
            if (r) {
                f2_t t[2];
                rr[j].pairs(t);
                v[j][0] = f2_add(v[j][0], t[0]);
                v[j][1] = f2_add(v[j][1], t[1]);
                if (s)
                    QX::store(s + row * W, j + 1 < NQ, col(j), G, W, v[j]);
            }
            t0 = f2_add(t0, v[j][0]);
            t1 = f2_add(t1, v[j][1]);
        }
        if (row + step < a.rows)
            fetch(row + step);
        const float mean = group_sum<G>(f2_sum(t0, t1)) * a.inv_w;
        // squares of the deviations from the mean, not of the values
        t0 = t1 = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            f2_t m[2];
            quad_where<V>(-mean, j + 1 < NQ, col(j), G, W, m);
            v[j][0] = f2_add(v[j][0], m[0]);
            v[j][1] = f2_add(v[j][1], m[1]);
            t0 = f2_fma(v[j][0], v[j][0], t0);
            t1 = f2_fma(v[j][1], v[j][1], t1);
        }
        float sq = group_sum<G>(f2_sum(t0, t1)) * a.inv_w, off = 0.0f;
        if (norm_far(mean, sq)) {  // the same for all lanes of a row
            t0 = t1 = f2_both(0.0f);
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                t0 = f2_add(t0, v[j][0]);
                t1 = f2_add(t1, v[j][1]);
            }
            off = group_sum<G>(f2_sum(t0, t1)) * a.inv_w;
            sq = norm_moved(sq, off);
        }
        const float rstd = __frsqrt_rn(sq + a.eps);
        if (lane == 0) {
            if (a.mean)
                a.mean[row] = mean + off;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
        const f2_t q = f2_both(rstd), c = f2_both(-off * rstd);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const f2_t o[2] = {f2_fma(f2_fma(v[j][0], q, c), wv[j][0], bv[j][0]),
                               f2_fma(f2_fma(v[j][1], q, c), wv[j][1], bv[j][1])};
            QY::store(y + row * W, j + 1 < NQ, col(j), G, W, o);
        }
    }
}

// Rows above kNormMaxWidth: a block walks its row three times
// (sum, deviations and their squares, output); the second and third reads hit L2.  s is
// written on the last walk, since it may be x itself.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kNormWideThreads, kNormWideBlocks)
    s6_layernorm_fwd_wide_kernel(const NormFwdArgs a) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ float red[3][kNormWideThreads / 32];
    const int W = a.width;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const X *x = static_cast<const X *>(a.x) + row * W;
        const Y *r = a.r ? static_cast<const Y *>(a.r) + row * W : nullptr;
        auto value = [&](int c, float (&v)[V]) {
            VX::unpack(VX::load(x + c), v);
            if (r) {
                float t[V];
                VY::unpack(VY::load(r + c), t);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[i] += t[i];
            }
        };
        float sum = 0.0f, sq = 0.0f, off = 0.0f, none = 0.0f;
        wide_walk<V, 4>(W, [&](int c, float &sum, float &) {
            float v[V];
            value(c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum += v[i];
        }, sum, none);
        const float mean = wide_sum(sum, red[0]) * a.inv_w;
        wide_walk<V, 4>(W, [&](int c, float &sq, float &off) {
            float v[V];
            value(c, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sq = fmaf(v[i] - mean, v[i] - mean, sq);
                off += v[i] - mean;
            }
        }, sq, off);
        // bound by the walks: every row is treated as far
        sq = wide_sum(sq, red[1]) * a.inv_w;
        off = wide_sum(off, red[2]) * a.inv_w;
        const float rstd = __frsqrt_rn(norm_moved(sq, off) + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[row] = mean + off;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x * V; c < W; c += kNormWideThreads * V) {
            float v[V], o[V];
            value(c, v);
            if (r && a.s)
                VX::store(static_cast<X *>(a.s) + row * W + c, VX::pack(v));
#pragma unroll
            for (int i = 0; i < V; ++i)
                o[i] = fmaf(((v[i] - mean) - off) * rstd, a.w ? a.w[c + i] : 1.0f, a.b ? a.b[c + i] : 0.0f);
            VY::store(static_cast<Y *>(a.y) + row * W + c, VY::pack(o));
        }
    }
}

// ----------------------------------------------------------------- backward
// A lane owns the same columns of every row it meets, so dw and db stay in its
// registers until the last one; the block then writes one row of partial sums
// and s6_sum_parts_kernel adds those up in float64.  4,000 float32 additions of a
// gradient of 0.1 are off by 4e-5 of their sum, 256 by 2e-6, so in every form there
// are so many blocks that a thread adds up norm_run rows at most.  (Sums kept in
// shared memory between runs, with no more blocks than are resident, took 3 to 12 %
// more time, tall or not.)  Rows of up to 64 elements, of which there may be many,
// run over 2,048; the _wide kernels over 1,024, since 16000x12000 bfloat16 took 578 us
// in runs of 256 and 482 in the 327 that fill the SMs.
constexpr int norm_run(int width) { return width <= 64 ? 2048 : width <= kNormMaxWidth ? 256 : 1024; }

template <typename X, typename Y, int V, int NQ, int G>
__global__ void __launch_bounds__(32 * kNormBlockWarps, norm_warps_resident(4 * NQ, true) / kNormBlockWarps)
    s6_layernorm_bwd_kernel(const NormBwdArgs a) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    using QF = Quad<float, V>;
    constexpr int kRows = 32 / G * kNormBlockWarps;
    const int lane = threadIdx.x % G, W = a.width;
    auto col = [&](int j) { return lane * V + 4 * G * j; };
    f2_t wv[NQ][2], dw[NQ][2], db[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), G, W, wv[j]);
        dw[j][0] = dw[j][1] = db[j][0] = db[j][1] = f2_both(0.0f);
    }

    const long long step = static_cast<long long>(kRows) * gridDim.x;
    long long row = static_cast<long long>(kRows) * blockIdx.x + threadIdx.x / G;
    const X *x = static_cast<const X *>(a.x);
    const Y *dy = static_cast<const Y *>(a.dy);
    QX xr[NQ];
    QY gr[NQ];
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](long long at) {
        mean = a.mean[at];
        rstd = a.rstd[at];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            xr[j].load(x + at * W, j + 1 < NQ, col(j), G, W);
            gr[j].load(dy + at * W, j + 1 < NQ, col(j), G, W);
        }
    };
    if (row < a.rows)
        fetch(row);
    for (; row < a.rows; row += step) {
        f2_t h[NQ][2], g[NQ][2], s0 = f2_both(0.0f), s1 = s0;
        const f2_t q = f2_both(rstd);
        const float rq = rstd;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            f2_t m[2];
            xr[j].pairs(h[j]);
            gr[j].pairs(g[j]);
            // elements behind the row have g = 0 and h = 0 (not 0 - mean, which times rstd may
            // be infinite) and add nothing
            quad_where<V>(-mean, j + 1 < NQ, col(j), G, W, m);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                h[j][i] = f2_mul(f2_add(h[j][i], m[i]), q);
                dw[j][i] = f2_fma(g[j][i], h[j][i], dw[j][i]);
                db[j][i] = f2_add(db[j][i], g[j][i]);
                g[j][i] = f2_mul(g[j][i], wv[j][i]);
                s0 = f2_add(s0, g[j][i]);
                s1 = f2_fma(g[j][i], h[j][i], s1);
            }
        }
        if (row + step < a.rows)
            fetch(row + step);
        QF ds[NQ];
        if (a.ds) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                ds[j].load(a.ds + row * W, j + 1 < NQ, col(j), G, W);
        }
        float m0, m1, hi;
        f2_unpack(s0, m0, hi);
        m0 += hi;
        f2_unpack(s1, m1, hi);
        m1 += hi;
        if constexpr (G == 32) {
            warp_sum2(m0, m1);
        } else {
            m0 = group_sum<G>(m0);
            m1 = group_sum<G>(m1);
        }
        // q (g - m0 - h m1) as q (g - h m1) - q m0
        const f2_t c1 = f2_both(-m1 * a.inv_w), c0 = f2_both(-rq * (m0 * a.inv_w));
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            f2_t o[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                o[i] = f2_fma(f2_fma(h[j][i], c1, g[j][i]), q, c0);
            if (a.ds) {
                f2_t t[2];
                ds[j].pairs(t);
                o[0] = f2_add(o[0], t[0]);
                o[1] = f2_add(o[1], t[1]);
            }
            QF::store(a.dx + row * W, j + 1 < NQ, col(j), G, W, o);
        }
    }

    if (!a.part)
        return;
    // a warp's groups of lanes hold sums of the same columns, and so do the block's warps:
    // add them up in order
#pragma unroll
    for (int o = G; o < 32; o *= 2)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                dw[j][i] = f2_add(dw[j][i], __shfl_xor_sync(0xffffffffu, dw[j][i], o));
                db[j][i] = f2_add(db[j][i], __shfl_xor_sync(0xffffffffu, db[j][i], o));
            }
    __shared__ __align__(16) float sums[2][kNormWarpWidth];
    for (int k = 0; k < kNormBlockWarps; ++k) {
        if ((threadIdx.x >> 5) == k && (threadIdx.x & 31) < G) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                f2_t t[2];
                Quad<float, V> at;
                if (k) {
                    at.load(sums[0], true, col(j), G, 0);
                    at.pairs(t);
                    dw[j][0] = f2_add(t[0], dw[j][0]);
                    dw[j][1] = f2_add(t[1], dw[j][1]);
                    at.load(sums[1], true, col(j), G, 0);
                    at.pairs(t);
                    db[j][0] = f2_add(t[0], db[j][0]);
                    db[j][1] = f2_add(t[1], db[j][1]);
                }
                QF::store(sums[0], true, col(j), G, 0, dw[j]);
                QF::store(sums[1], true, col(j), G, 0, db[j]);
            }
        }
        __syncthreads();
    }
    float *part = a.part + static_cast<long long>(blockIdx.x) * 2 * W;
    for (int c = threadIdx.x; c < W; c += 32 * kNormBlockWarps) {
        part[c] = sums[0][c];
        part[W + c] = sums[1][c];
    }
}

// ------------------------------------------------ rows in shared memory
// A block of T threads takes R consecutive rows (one stretch of each tensor) at
// a step.  They come by bulk copies that thread 0 starts `stages` - 1 steps
// ahead; each thread takes NQ quads of columns of every row into registers once
// and keeps its columns' parameters (and, backward, their gradients' sums) in
// registers over all steps.  Two rows a step share the reductions' shuffles and
// barriers, which with one row, or with rows that pass through registers alone,
// cost more than the arithmetic (44 instructions an element at a width of 2560;
// rows summed by a warp each and read again for the output took 30).  Blocks
// have a multiple of 4 warps, one for each scheduler of the SM: with 5, the
// busiest scheduler had 1.3 times its share.
constexpr int kNormMaxStages = 4;

struct NormStream {
    int stages;
    int x_bytes, y_bytes, e_bytes;  // a step's buffers: x; r or dy; ds
    int stage() const { return x_bytes + y_bytes + e_bytes; }
};

// The ring of a block's steps.
struct NormRing {
    unsigned char *buf;
    uint64_t *full;
    int stages, stage_bytes;
    int st;          // stage of the present step
    uint32_t phase;  // its parity

    __device__ __forceinline__ unsigned char *at() const { return buf + st * stage_bytes; }
    __device__ __forceinline__ bool wait() const { return mbar_wait_bounded(&full[st], phase, kBulkPolls); }
    __device__ __forceinline__ void next() {
        if (++st == stages) {
            st = 0;
            phase ^= 1u;
        }
    }
    // After a wait that gave up: one thread waits, with the same bound, for the copies of
    // the present step and of the `left` steps behind it that have been started.
    __device__ __forceinline__ void drain(int left) {
        raise_device_error(kErrTrainCopy);
        wait();
        for (int k = 0; k < left; ++k) {
            next();
            wait();
        }
    }
};

struct NormFwdBlockArgs {
    NormFwdArgs n;
    NormStream s;
};

template <typename X, typename Y, int V, int NQ, int R, int T, int MINB>
__global__ void __launch_bounds__(T, MINB) s6_layernorm_fwd_block_kernel(const NormFwdBlockArgs args) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    constexpr int WARPS = T / 32;
    const NormFwdArgs &a = args.n;
    extern __shared__ __align__(16) unsigned char s6_norm_smem[];
    __shared__ uint64_t full[kNormMaxStages];
    __shared__ float slots[3][4][16];
    const int tid = threadIdx.x, W = a.width;
    const X *x = static_cast<const X *>(a.x);
    const Y *r = static_cast<const Y *>(a.r);
    auto col = [&](int j) { return tid * V + 4 * T * j; };  // only the last quad can pass the row's end
    // Three quads a thread are summed up behind their loads, which takes 80 registers (between
    // them 82 in one form: a block fewer on an SM, 8191x2561 f32 to bfloat16 37 us for 27); four
    // between their loads, 93 for 121 (16384x2047 bfloat16 33 us for 45).
    constexpr bool kSumsBehind = NQ == 3;
    const long long steps = (a.rows + R - 1) / R, total = a.rows * W;
    NormRing ring{s6_norm_smem, full, args.s.stages, args.s.x_bytes + args.s.y_bytes, 0, 0u};

    auto fetch = [&](int st, long long step) {  // thread 0
        const long long first = step * R * W;
        const uint32_t n = static_cast<uint32_t>((a.rows - step * R < R ? a.rows - step * R : R) * W);
        unsigned char *to = ring.buf + st * ring.stage_bytes;
        const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), r0 = reinterpret_cast<uintptr_t>(r);
        bulk_fetch<X>(to, x0 + first * sizeof(X), n * sizeof(X), x0, x0 + total * sizeof(X), &full[st]);
        if (r)
            bulk_fetch<Y>(to + args.s.x_bytes, r0 + first * sizeof(Y), n * sizeof(Y), r0,
                                   r0 + total * sizeof(Y), &full[st]);
        mbar_arrive(&full[st]);
    };
    if (tid == 0) {
        for (int st = 0; st < ring.stages; ++st)
            mbar_init(&full[st], 1);
        fence_mbarrier_init();
        for (int st = 0; st < ring.stages; ++st)
            if (blockIdx.x + static_cast<long long>(st) * gridDim.x < steps)
                fetch(st, blockIdx.x + static_cast<long long>(st) * gridDim.x);
    }
    f2_t wv[NQ][2], bv[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), T, W, wv[j]);
        quad_params<V>(a.b, 0.0f, col(j), T, W, bv[j]);
    }
    __syncthreads();

    for (long long step = blockIdx.x; step < steps; step += gridDim.x) {
        const long long row = step * R;
        const int here = a.rows - row < R ? static_cast<int>(a.rows - row) : R;
        const bool ok = ring.wait();
        const X *xs = reinterpret_cast<const X *>(ring.at() + in16(x, row * W));
        const Y *rs = reinterpret_cast<const Y *>(ring.at() + args.s.x_bytes + in16(r, row * W));
        f2_t v[R][NQ][2];
        float sum[R];
        // a row that is not there is read as zeros
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f2_t t0 = f2_both(0.0f), t1 = t0;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                v[k][j][0] = v[k][j][1] = f2_both(0.0f);
                if (k > 0 && k >= here)
                    continue;
                QX q;
                q.load(xs + k * W, j + 1 < NQ, col(j), T, W);
                q.pairs(v[k][j]);
                if (r) {
                    QY p;
                    f2_t t[2];
                    p.load(rs + k * W, j + 1 < NQ, col(j), T, W);
                    p.pairs(t);
                    v[k][j][0] = f2_add(v[k][j][0], t[0]);
                    v[k][j][1] = f2_add(v[k][j][1], t[1]);
                    if (a.s)
                        QX::store(static_cast<X *>(a.s) + (row + k) * W, j + 1 < NQ, col(j), T, W, v[k][j]);
                }
                if constexpr (!kSumsBehind) {
                    t0 = f2_add(t0, v[k][j][0]);
                    t1 = f2_add(t1, v[k][j][1]);
                }
            }
            if constexpr (kSumsBehind) {
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    t0 = f2_add(t0, v[k][j][0]);
                    t1 = f2_add(t1, v[k][j][1]);
                }
            }
            sum[k] = f2_sum(t0, t1);
        }
        if (block_sums<R, WARPS>(sum, slots[0], !ok)) {
            if (tid == 0) {
                const long long more = (steps - 1 - step) / gridDim.x;
                ring.drain(more < ring.stages - 1 ? static_cast<int>(more) : ring.stages - 1);
            }
            return;
        }
        // every thread has taken the step into registers: its stage is free
        if (tid == 0 && step + static_cast<long long>(ring.stages) * gridDim.x < steps)
            fetch(ring.st, step + static_cast<long long>(ring.stages) * gridDim.x);
        ring.next();
        float sq[R], off[R];  // sum: the means from here on
#pragma unroll
        for (int k = 0; k < R; ++k) {
            sum[k] *= a.inv_w;
            f2_t t0 = f2_both(0.0f), t1 = t0;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                f2_t m[2];
                quad_where<V>(-sum[k], j + 1 < NQ, col(j), T, W, m);
                v[k][j][0] = f2_add(v[k][j][0], m[0]);
                v[k][j][1] = f2_add(v[k][j][1], m[1]);
                t0 = f2_fma(v[k][j][0], v[k][j][0], t0);
                t1 = f2_fma(v[k][j][1], v[k][j][1], t1);
            }
            sq[k] = f2_sum(t0, t1);
        }
        block_sums<R, WARPS>(sq, slots[1], false);
        bool far = false;  // the same for all threads
#pragma unroll
        for (int k = 0; k < R; ++k) {
            sq[k] *= a.inv_w;
            off[k] = 0.0f;
            far = far || norm_far(sum[k], sq[k]);
            if (tid == 0 && a.mean && k < here)
                a.mean[row + k] = sum[k];
        }
        if (far) {
            float dev[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                f2_t t0 = f2_both(0.0f), t1 = t0;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    t0 = f2_add(t0, v[k][j][0]);
                    t1 = f2_add(t1, v[k][j][1]);
                }
                dev[k] = f2_sum(t0, t1);
            }
            block_sums<R, WARPS>(dev, slots[2], false);
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (norm_far(sum[k], sq[k])) {  // each row by itself, whatever shares its step
                    off[k] = dev[k] * a.inv_w;
                    sq[k] = norm_moved(sq[k], off[k]);
                    if (tid == 0 && a.mean && k < here)
                        a.mean[row + k] = sum[k] + off[k];
                }
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (k < here) {
                const float rstd = __frsqrt_rn(sq[k] + a.eps);
                if (tid == 0 && a.rstd)
                    a.rstd[row + k] = rstd;
                const f2_t q = f2_both(rstd), c = f2_both(-off[k] * rstd);
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const f2_t o[2] = {f2_fma(f2_fma(v[k][j][0], q, c), wv[j][0], bv[j][0]),
                                       f2_fma(f2_fma(v[k][j][1], q, c), wv[j][1], bv[j][1])};
                    QY::store(static_cast<Y *>(a.y) + (row + k) * W, j + 1 < NQ, col(j), T, W, o);
                }
            }
    }
}

struct NormBwdBlockArgs {
    NormBwdArgs n;
    NormStream s;
};

template <typename X, typename Y, int V, int NQ, int R, int T, int MINB>
__global__ void __launch_bounds__(T, MINB) s6_layernorm_bwd_block_kernel(const NormBwdBlockArgs args) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    using QF = Quad<float, V>;
    constexpr int WARPS = T / 32;
    const NormBwdArgs &a = args.n;
    extern __shared__ __align__(16) unsigned char s6_norm_smem[];
    __shared__ uint64_t full[kNormMaxStages];
    __shared__ float slots[2][4][16];
    const int tid = threadIdx.x, W = a.width;
    const X *x = static_cast<const X *>(a.x);
    const Y *dy = static_cast<const Y *>(a.dy);
    auto col = [&](int j) { return tid * V + 4 * T * j; };
    const long long steps = (a.rows + R - 1) / R, total = a.rows * W;
    NormRing ring{s6_norm_smem, full, args.s.stages, args.s.x_bytes + args.s.y_bytes + args.s.e_bytes, 0, 0u};

    auto fetch = [&](int st, long long step) {  // thread 0
        const long long first = step * R * W;
        const uint32_t n = static_cast<uint32_t>((a.rows - step * R < R ? a.rows - step * R : R) * W);
        unsigned char *to = ring.buf + st * ring.stage_bytes;
        const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), g0 = reinterpret_cast<uintptr_t>(dy),
                        e0 = reinterpret_cast<uintptr_t>(a.ds);
        bulk_fetch<X>(to, x0 + first * sizeof(X), n * sizeof(X), x0, x0 + total * sizeof(X), &full[st]);
        bulk_fetch<Y>(to + args.s.x_bytes, g0 + first * sizeof(Y), n * sizeof(Y), g0, g0 + total * sizeof(Y),
                               &full[st]);
        if (a.ds)
            bulk_fetch<float>(to + args.s.x_bytes + args.s.y_bytes, e0 + first * 4, n * 4, e0, e0 + total * 4,
                                       &full[st]);
        mbar_arrive(&full[st]);
    };
    if (tid == 0) {
        for (int st = 0; st < ring.stages; ++st)
            mbar_init(&full[st], 1);
        fence_mbarrier_init();
        for (int st = 0; st < ring.stages; ++st)
            if (blockIdx.x + static_cast<long long>(st) * gridDim.x < steps)
                fetch(st, blockIdx.x + static_cast<long long>(st) * gridDim.x);
    }
    f2_t wv[NQ][2], dw[NQ][2], db[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), T, W, wv[j]);
        dw[j][0] = dw[j][1] = db[j][0] = db[j][1] = f2_both(0.0f);
    }
    // a step's statistics are fetched one step ahead
    float mean[R], rstd[R];
    auto statistics = [&](long long step) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long row = step * R + k;
            mean[k] = row < a.rows ? a.mean[row] : 0.0f;
            rstd[k] = row < a.rows ? a.rstd[row] : 0.0f;
        }
    };
    if (blockIdx.x < steps)
        statistics(blockIdx.x);
    __syncthreads();

    int turn = 0;
    for (long long step = blockIdx.x; step < steps; step += gridDim.x, turn ^= 1) {
        const long long row = step * R;
        const int here = a.rows - row < R ? static_cast<int>(a.rows - row) : R;
        float q[R];
        f2_t h[R][NQ][2], g[R][NQ][2];
        float sums[2 * R];
        const bool ok = ring.wait();
        const X *xs = reinterpret_cast<const X *>(ring.at() + in16(x, row * W));
        const Y *gs = reinterpret_cast<const Y *>(ring.at() + args.s.x_bytes + in16(dy, row * W));
        const float *es = reinterpret_cast<const float *>(ring.at() + args.s.x_bytes + args.s.y_bytes +
                                                          in16(a.ds, row * W));
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const f2_t q2 = f2_both(rstd[k]);
            q[k] = rstd[k];
            f2_t s0 = f2_both(0.0f), s1 = s0;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                QX xq;
                QY gq;
                if (k == 0 || k < here) {
                    xq.load(xs + k * W, j + 1 < NQ, col(j), T, W);
                    gq.load(gs + k * W, j + 1 < NQ, col(j), T, W);
                } else {
                    xq.clear();
                    gq.clear();
                }
                f2_t m[2];
                xq.pairs(h[k][j]);
                gq.pairs(g[k][j]);
                // what is behind the row, or a row that is not there, has g = 0 and h = 0 (not
                // 0 - mean, which times rstd may be infinite) and adds nothing
                quad_where<V>(-mean[k], j + 1 < NQ, col(j), T, W, m);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[k][j][i] = f2_mul(f2_add(h[k][j][i], m[i]), q2);
                    dw[j][i] = f2_fma(g[k][j][i], h[k][j][i], dw[j][i]);
                    db[j][i] = f2_add(db[j][i], g[k][j][i]);
                    g[k][j][i] = f2_mul(g[k][j][i], wv[j][i]);
                    s0 = f2_add(s0, g[k][j][i]);
                    s1 = f2_fma(g[k][j][i], h[k][j][i], s1);
                }
            }
            float lo, hi;
            f2_unpack(s0, lo, hi);
            sums[2 * k] = lo + hi;
            f2_unpack(s1, lo, hi);
            sums[2 * k + 1] = lo + hi;
        }
        if (step + gridDim.x < steps)
            statistics(step + gridDim.x);
        // slots by turns: those of this step are written again two steps on, after the next
        // step's barrier, which every reader of them has passed
        if (block_sums<2 * R, WARPS>(sums, slots[turn], !ok)) {
            if (tid == 0) {
                const long long more = (steps - 1 - step) / gridDim.x;
                const int started = ring.stages - (step == blockIdx.x ? 1 : 2);
                ring.drain(more < started ? static_cast<int>(more) : started);
            }
            return;
        }
        // every thread is past the step before this one, ds too: its stage is free
        if (tid == 0 && step != blockIdx.x) {
            const long long ahead = step + static_cast<long long>(ring.stages - 1) * gridDim.x;
            if (ahead < steps)
                fetch(ring.st ? ring.st - 1 : ring.stages - 1, ahead);
        }
        ring.next();
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (k < here) {
                // q (g - m0 - h m1) as q (g - h m1) - q m0
                const f2_t q2 = f2_both(q[k]), c1 = f2_both(-sums[2 * k + 1] * a.inv_w),
                           c0 = f2_both(-q[k] * (sums[2 * k] * a.inv_w));
                float *dxp = a.dx + (row + k) * W;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    f2_t o[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        o[i] = f2_fma(f2_fma(h[k][j][i], c1, g[k][j][i]), q2, c0);
                    if (a.ds) {
                        QF eq;
                        f2_t t[2];
                        eq.load(es + k * W, j + 1 < NQ, col(j), T, W);
                        eq.pairs(t);
                        o[0] = f2_add(o[0], t[0]);
                        o[1] = f2_add(o[1], t[1]);
                    }
                    QF::store(dxp, j + 1 < NQ, col(j), T, W, o);
                }
            }
    }
    if (!a.part)
        return;
    float *part = a.part + static_cast<long long>(blockIdx.x) * 2 * W;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        // part's rows are W floats: single elements keep any alignment
        float f[4], g[4];
        f2_unpack(dw[j][0], f[0], f[1]);
        f2_unpack(dw[j][1], f[2], f[3]);
        f2_unpack(db[j][0], g[0], g[1]);
        f2_unpack(db[j][1], g[2], g[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = V == 4 ? col(j) + i : col(j) + i * T;
            if (c < W) {
                part[c] = f[i];
                part[W + c] = g[i];
            }
        }
    }
}

// Wide rows: the two sums of every row first (a block a row), ...
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kNormWideThreads, kNormWideBlocks)
    s6_layernorm_bwd_wide_sums_kernel(const NormBwdArgs a, float2 *sums) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ float red[2][kNormWideThreads / 32];
    const int W = a.width;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const X *x = static_cast<const X *>(a.x) + row * W;
        const Y *dy = static_cast<const Y *>(a.dy) + row * W;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s0 = 0.0f, s1 = 0.0f;
        wide_walk<V, V == 4 ? 2 : 4>(W, [&](int c, float &s0, float &s1) {
            float h[V], g[V];
            VX::unpack(VX::load(x + c), h);
            VY::unpack(VY::load(dy + c), g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = g[i] * (a.w ? a.w[c + i] : 1.0f);
                s0 += t;
                s1 = fmaf(t, (h[i] - mean) * rstd, s1);
            }
        }, s0, s1);
        s0 = wide_sum(s0, red[0]);
        s1 = wide_sum(s1, red[1]);
        if (threadIdx.x == 0)
            sums[row] = make_float2(s0 * a.inv_w, s1 * a.inv_w);
    }
}

// ... then dx, dw and db by columns: a thread owns V columns of a run of rows
// (gridDim.y runs), so dw and db again need one sum over the runs only.
constexpr int kNormColThreads = 128;

template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kNormColThreads) s6_layernorm_bwd_wide_cols_kernel(const NormBwdArgs a,
                                                                                   const float2 *sums) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    using VF = IoVec<float, V>;
    const int W = a.width;
    const int c = (blockIdx.x * kNormColThreads + threadIdx.x) * V;
    if (c >= W)
        return;
    const long long per = (a.rows + gridDim.y - 1) / gridDim.y;
    const long long first = per * blockIdx.y;
    const long long last = first + per < a.rows ? first + per : a.rows;
    float w[V], dw[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i] = a.w ? a.w[c + i] : 1.0f;
        dw[i] = db[i] = 0.0f;
    }
#pragma unroll 2
    for (long long row = first; row < last; ++row) {
        float h[V], g[V], o[V];
        VX::unpack(VX::load(static_cast<const X *>(a.x) + row * W + c), h);
        VY::unpack(VY::load(static_cast<const Y *>(a.dy) + row * W + c), g);
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 k = sums[row];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[i] = (h[i] - mean) * rstd;
            dw[i] = fmaf(g[i], h[i], dw[i]);
            db[i] += g[i];
            o[i] = rstd * (fmaf(g[i], w[i], -k.x) - h[i] * k.y);
        }
        if (a.ds) {
            float t[V];
            VF::unpack(VF::load(a.ds + row * W + c), t);
#pragma unroll
            for (int i = 0; i < V; ++i)
                o[i] += t[i];
        }
        VF::store(a.dx + row * W + c, VF::pack(o));
    }
    if (a.part) {
        float *part = a.part + static_cast<long long>(blockIdx.y) * 2 * W;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            part[c + i] = dw[i];
            part[W + c + i] = db[i];
        }
    }
}

}  // namespace s6
