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
//     h = (s - m) q,    g = w dy
//     dx = ds + q (g - sum(g)/W - h sum(g h)/W)        ds: the gradient that
//     dw = sum over rows of dy h,  db = of dy          reaches s past the norm
//
// Both are bound by HBM: a row is read once, in the storage type, and
// everything is computed in float32 from there.  Three forms, by the width:
//
//  * up to kNormWarpWidth: a row is one warp's, in its registers.  The warp
//    walks rows with a fixed stride and fetches the next one while it reduces
//    the present one.
//  * up to kNormMaxWidth: rows pass through shared memory, copied ahead of
//    their use without registers.  Forward, a row is one warp's still, so it
//    needs no barrier; backward, a block takes some rows at a time, a few
//    warps sum each row, and then each thread does its own columns of all of
//    them.  (Rows split over a block's registers, which this replaces, spent
//    44 instructions an element on reductions and addresses at a width of 2560.)
//  * above that: the _wide kernels, which read a row more than once.
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

constexpr int kNormWideThreads = 512;

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

template <typename X, typename Y, int V, int NQ>
__global__ void __launch_bounds__(32 * kNormBlockWarps, norm_warps_resident(4 * NQ, false) / kNormBlockWarps)
    s6_layernorm_fwd_kernel(const NormFwdArgs a) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    const int lane = threadIdx.x & 31, W = a.width;
    auto col = [&](int j) { return lane * V + 128 * j; };  // of quad j
    f2_t wv[NQ][2], bv[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), 32, W, wv[j]);
        quad_params<V>(a.b, 0.0f, col(j), 32, W, bv[j]);
    }

    const long long step = static_cast<long long>(kNormBlockWarps) * gridDim.x;
    long long row = static_cast<long long>(kNormBlockWarps) * blockIdx.x + (threadIdx.x >> 5);
    const X *x = static_cast<const X *>(a.x);
    const Y *r = static_cast<const Y *>(a.r);
    X *s = static_cast<X *>(a.s);
    Y *y = static_cast<Y *>(a.y);
    QX xr[NQ];
    QY rr[NQ];
    auto fetch = [&](long long at) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            xr[j].template load<false>(x + at * W, col(j), 32, W);
            if (r)
                rr[j].template load<false>(r + at * W, col(j), 32, W);
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
                    QX::template store<false>(s + row * W, col(j), 32, W, v[j]);
            }
            t0 = f2_add(t0, v[j][0]);
            t1 = f2_add(t1, v[j][1]);
        }
        if (row + step < a.rows)
            fetch(row + step);
        const float mean = warp_sum(f2_sum(t0, t1)) * a.inv_w;
        // squares of the deviations from the mean, not of the values: a mean that is
        // large next to the deviations costs no digits
        t0 = t1 = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            f2_t m[2];
            quad_where<V>(-mean, col(j), 32, W, m);
            v[j][0] = f2_add(v[j][0], m[0]);
            v[j][1] = f2_add(v[j][1], m[1]);
            t0 = f2_fma(v[j][0], v[j][0], t0);
            t1 = f2_fma(v[j][1], v[j][1], t1);
        }
        const float rstd = __frsqrt_rn(warp_sum(f2_sum(t0, t1)) * a.inv_w + a.eps);
        if (lane == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
        const f2_t q = f2_both(rstd);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const f2_t o[2] = {f2_fma(f2_mul(v[j][0], q), wv[j][0], bv[j][0]),
                               f2_fma(f2_mul(v[j][1], q), wv[j][1], bv[j][1])};
            QY::template store<false>(y + row * W, col(j), 32, W, o);
        }
    }
}

// Rows above kNormMaxWidth: a block walks its row three times
// (sum, squared deviations, output); the second and third reads hit L2.  s is
// written on the last walk, since it may be x itself.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kNormWideThreads) s6_layernorm_fwd_wide_kernel(const NormFwdArgs a) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ float red[2][kNormWideThreads / 32];
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
        float sum = 0.0f, sq = 0.0f;
        for (int c = threadIdx.x * V; c < W; c += kNormWideThreads * V) {
            float v[V];
            value(c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum += v[i];
        }
        const float mean = wide_sum(sum, red[0]) * a.inv_w;
        for (int c = threadIdx.x * V; c < W; c += kNormWideThreads * V) {
            float v[V];
            value(c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sq = fmaf(v[i] - mean, v[i] - mean, sq);
        }
        const float rstd = __frsqrt_rn(wide_sum(sq, red[1]) * a.inv_w + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[row] = mean;
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
                o[i] = fmaf((v[i] - mean) * rstd, a.w ? a.w[c + i] : 1.0f, a.b ? a.b[c + i] : 0.0f);
            VY::store(static_cast<Y *>(a.y) + row * W + c, VY::pack(o));
        }
    }
}

// ----------------------------------------------------------------- backward
// A lane owns the same columns of every row it meets, so dw and db stay in its
// registers until the last one; the block then writes one row of partial sums
// and s6_sum_parts_kernel adds those up.
template <typename X, typename Y, int V, int NQ>
__global__ void __launch_bounds__(32 * kNormBlockWarps, norm_warps_resident(4 * NQ, true) / kNormBlockWarps)
    s6_layernorm_bwd_kernel(const NormBwdArgs a) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    using QF = Quad<float, V>;
    const int lane = threadIdx.x & 31, W = a.width;
    auto col = [&](int j) { return lane * V + 128 * j; };
    f2_t wv[NQ][2], dw[NQ][2], db[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), 32, W, wv[j]);
        dw[j][0] = dw[j][1] = db[j][0] = db[j][1] = f2_both(0.0f);
    }

    const long long step = static_cast<long long>(kNormBlockWarps) * gridDim.x;
    long long row = static_cast<long long>(kNormBlockWarps) * blockIdx.x + (threadIdx.x >> 5);
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
            xr[j].template load<false>(x + at * W, col(j), 32, W);
            gr[j].template load<false>(dy + at * W, col(j), 32, W);
        }
    };
    if (row < a.rows)
        fetch(row);
    for (; row < a.rows; row += step) {
        f2_t h[NQ][2], g[NQ][2], s0 = f2_both(0.0f), s1 = s0;
        const f2_t m = f2_both(-mean), q = f2_both(rstd);
        const float rq = rstd;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            xr[j].pairs(h[j]);
            gr[j].pairs(g[j]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // elements behind the row have g = 0 and add nothing
                h[j][i] = f2_mul(f2_add(h[j][i], m), q);
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
                ds[j].template load<false>(a.ds + row * W, col(j), 32, W);
        }
        float m0, m1, hi;
        f2_unpack(s0, m0, hi);
        m0 += hi;
        f2_unpack(s1, m1, hi);
        m1 += hi;
        warp_sum2(m0, m1);
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
            QF::template store<false>(a.dx + row * W, col(j), 32, W, o);
        }
    }

    if (!a.part)
        return;
    // the block's warps hold sums of the same columns: add them up in order
    __shared__ __align__(16) float sums[2][kNormWarpWidth];
    for (int k = 0; k < kNormBlockWarps; ++k) {
        if ((threadIdx.x >> 5) == k) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                f2_t t[2];
                Quad<float, V> at;
                if (k) {
                    at.template load<true>(sums[0], col(j), 32, 0);
                    at.pairs(t);
                    dw[j][0] = f2_add(t[0], dw[j][0]);
                    dw[j][1] = f2_add(t[1], dw[j][1]);
                    at.template load<true>(sums[1], col(j), 32, 0);
                    at.pairs(t);
                    db[j][0] = f2_add(t[0], db[j][0]);
                    db[j][1] = f2_add(t[1], db[j][1]);
                }
                QF::template store<true>(sums[0], col(j), 32, 0, dw[j]);
                QF::template store<true>(sums[1], col(j), 32, 0, db[j]);
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
// Rows come by bulk copies, a few tiles ahead of their use (kNormStages).
// Forward, a row is a warp's own: lane 0 starts its copies and the warp waits
// for them alone.  w and b are kept beside the rows.  Three passes over the
// row's buffer (sum, squared deviations, output), each in the same order wherever
// the row begins, so a row's result does not depend on its place.
constexpr int kNormStages = 2;
constexpr int kNormRowWarps = 8;  // warps of a block, or as many as shared memory allows

struct NormRowsArgs {
    NormFwdArgs n;
    int x_bytes, r_bytes;  // row buffers
};

template <typename X, typename Y, int V>
__global__ void __launch_bounds__(32 * kNormRowWarps) s6_layernorm_fwd_rows_kernel(const NormRowsArgs args) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    using QF = Quad<float, V>;
    const NormFwdArgs &a = args.n;
    extern __shared__ __align__(16) unsigned char s6_norm_smem[];
    __shared__ uint64_t full[kNormRowWarps][kNormStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int W = a.width, c0 = lane * V;
    const int whole = W & ~127;  // columns of whole steps of the warp: a quad a lane
    float *w = reinterpret_cast<float *>(s6_norm_smem), *b = w + (W + 3) / 4 * 4;
    const int stage = args.x_bytes + args.r_bytes;
    unsigned char *rows = reinterpret_cast<unsigned char *>(b + (W + 3) / 4 * 4) + warp * kNormStages * stage;
    const X *x = static_cast<const X *>(a.x);
    const Y *r = static_cast<const Y *>(a.r);
    const long long total = a.rows * W;

    const long long step = static_cast<long long>(warps) * gridDim.x;
    long long row = static_cast<long long>(warps) * blockIdx.x + warp;
    auto fetch = [&](int st, long long at) {  // lane 0
        unsigned char *to = rows + st * stage;
        const BulkSpan sx = bulk_span(to, x, total, at * W, W);
        BulkSpan sr{nullptr, 0, 0};
        if (r)
            sr = bulk_span(to + args.x_bytes, r, total, at * W, W);
        mbar_arrive_expect_tx(&full[warp][st], sx.bytes + sr.bytes);
        bulk_start(to, sx, &full[warp][st]);
        bulk_start(to + args.x_bytes, sr, &full[warp][st]);
    };
    if (lane == 0) {
        for (int st = 0; st < kNormStages; ++st)
            mbar_init(&full[warp][st], 1);
        fence_mbarrier_init();
        for (int st = 0; st < kNormStages; ++st)
            if (row + st * step < a.rows)
                fetch(st, row + st * step);
    }
    for (int c = threadIdx.x; c < W; c += blockDim.x) {
        w[c] = a.w ? a.w[c] : 1.0f;
        b[c] = a.b ? a.b[c] : 0.0f;
    }
    __syncthreads();

    int st = 0;
    uint32_t phase = 0;
    for (; row < a.rows; row += step) {
        const bool ok = mbar_wait_bounded(&full[warp][st], phase, kBulkPolls);
        if (__any_sync(0xffffffffu, !ok)) {
            if (lane == 0) {
                raise_device_error(kErrTrainCopy);
                // the copies still in flight are waited for, with the same bound
                if (row + step < a.rows)
                    mbar_wait_bounded(&full[warp][st ^ 1], st ? phase ^ 1u : phase, kBulkPolls);
            }
            return;
        }
        const X *xs = reinterpret_cast<const X *>(rows + st * stage + in16(x, row * W));
        const Y *rs = r ? reinterpret_cast<const Y *>(rows + st * stage + args.x_bytes + in16(r, row * W)) : nullptr;
        auto value = [&](auto all, int c, f2_t (&v)[2]) {
            constexpr bool ALL = decltype(all)::value;
            QX q;
            q.template load<ALL>(xs, c, 32, W);
            q.pairs(v);
            if (r) {
                QY p;
                f2_t t[2];
                p.template load<ALL>(rs, c, 32, W);
                p.pairs(t);
                v[0] = f2_add(v[0], t[0]);
                v[1] = f2_add(v[1], t[1]);
            }
        };
        // fn(all, column) for the whole steps, then for the one that the row's end cuts
        auto walk = [&](auto fn) {
#pragma unroll 4
            for (int c = 0; c < whole; c += 128)
                fn(std::true_type{}, c0 + c);
            if (whole < W)
                fn(std::false_type{}, c0 + whole);
        };
        f2_t t0 = f2_both(0.0f), t1 = t0;
        walk([&](auto all, int c) {
            f2_t v[2];
            value(all, c, v);
            t0 = f2_add(t0, v[0]);
            t1 = f2_add(t1, v[1]);
        });
        const float mean = warp_sum(f2_sum(t0, t1)) * a.inv_w;
        const f2_t m = f2_both(-mean);
        t0 = t1 = f2_both(0.0f);
        walk([&](auto all, int c) {
            f2_t v[2], d[2] = {m, m};
            value(all, c, v);
            if constexpr (!decltype(all)::value)
                quad_where<V>(-mean, c, 32, W, d);
            v[0] = f2_add(v[0], d[0]);
            v[1] = f2_add(v[1], d[1]);
            t0 = f2_fma(v[0], v[0], t0);
            t1 = f2_fma(v[1], v[1], t1);
        });
        const float rstd = __frsqrt_rn(warp_sum(f2_sum(t0, t1)) * a.inv_w + a.eps);
        if (lane == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
        X *sp = a.s ? static_cast<X *>(a.s) + row * W : nullptr;
        Y *yp = static_cast<Y *>(a.y) + row * W;
        const f2_t q = f2_both(rstd);
        walk([&](auto all, int c) {
            constexpr bool ALL = decltype(all)::value;
            f2_t v[2], wv[2], bv[2];
            value(all, c, v);
            if (sp)
                QX::template store<ALL>(sp, c, 32, W, v);
            QF p;
            p.template load<ALL>(w, c, 32, W);
            p.pairs(wv);
            p.template load<ALL>(b, c, 32, W);
            p.pairs(bv);
            const f2_t o[2] = {f2_fma(f2_mul(f2_add(v[0], m), q), wv[0], bv[0]),
                               f2_fma(f2_mul(f2_add(v[1], m), q), wv[1], bv[1])};
            QY::template store<ALL>(yp, c, 32, W, o);
        });
        __syncwarp();  // every lane is done with the stage
        if (lane == 0 && row + kNormStages * step < a.rows)
            fetch(st, row + kNormStages * step);
        if (++st == kNormStages) {
            st = 0;
            phase ^= 1u;
        }
    }
}

// Backward: a block takes `tile` consecutive rows at a time, which are one
// stretch of each tensor; thread 0 starts their copies.  Each row's two sums are
// made by blockDim / 32 / tile warps, whose parts every thread then adds in
// order; a thread owns NQ quads of columns and keeps their dw and db in
// registers until the block's last tile.  Blocks have a multiple of 4 warps,
// one for each scheduler of the SM: with 5 (which a width of 2560 would fill
// exactly) the busiest one had 1.3 times its share.
struct NormTileArgs {
    NormBwdArgs n;
    int tile;
    int x_bytes, dy_bytes, ds_bytes;  // a tile's buffers
};

constexpr int kNormTileRows = 8;  // at most

template <typename X, typename Y, int V, int NQ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) s6_layernorm_bwd_tile_kernel(const NormTileArgs args) {
    using QX = Quad<X, V>;
    using QY = Quad<Y, V>;
    using QF = Quad<float, V>;
    const NormBwdArgs &a = args.n;
    extern __shared__ __align__(16) unsigned char s6_norm_smem[];
    __shared__ uint64_t full[kNormStages];
    __shared__ float stats[kNormStages][kNormTileRows][2];  // mean, rstd
    __shared__ float2 parts[kNormTileRows][MAXT / 32];      // each warp's two sums
    constexpr int T = MAXT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int W = a.width, R = args.tile;
    const int share = T / 32 / R;  // warps that sum a row
    float *w = reinterpret_cast<float *>(s6_norm_smem);
    const int stage = args.x_bytes + args.dy_bytes + args.ds_bytes;
    unsigned char *buf = reinterpret_cast<unsigned char *>(w + (W + 3) / 4 * 4);
    const X *x = static_cast<const X *>(a.x);
    const Y *dy = static_cast<const Y *>(a.dy);
    const long long total = a.rows * W;
    auto col = [&](int j) { return static_cast<int>(threadIdx.x) * V + 4 * T * j; };

    const long long tiles = (a.rows + R - 1) / R;
    auto rows_of = [&](long long tile) {
        return a.rows - tile * R < R ? static_cast<int>(a.rows - tile * R) : R;
    };
    auto fetch = [&](int st, long long tile) {
        if (tile < tiles) {
            const int n = rows_of(tile);
            if (threadIdx.x == 0) {
                unsigned char *to = buf + st * stage, *to_dy = to + args.x_bytes, *to_ds = to_dy + args.dy_bytes;
                const long long at = tile * R * W, len = static_cast<long long>(n) * W;
                const BulkSpan sx = bulk_span(to, x, total, at, len), sy = bulk_span(to_dy, dy, total, at, len);
                BulkSpan se{nullptr, 0, 0};
                if (a.ds)
                    se = bulk_span(to_ds, a.ds, total, at, len);
                mbar_arrive_expect_tx(&full[st], sx.bytes + sy.bytes + se.bytes);
                bulk_start(to, sx, &full[st]);
                bulk_start(to_dy, sy, &full[st]);
                bulk_start(to_ds, se, &full[st]);
            }
            const int k = threadIdx.x;
            if (k < n) {
                cp_async4(&stats[st][k][0], a.mean + tile * R + k);
                cp_async4(&stats[st][k][1], a.rstd + tile * R + k);
            }
        }
        cp_async_commit();
    };
    long long tile = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int st = 0; st < kNormStages; ++st)
            mbar_init(&full[st], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
#pragma unroll
    for (int st = 0; st < kNormStages; ++st)
        fetch(st, tile + static_cast<long long>(st) * gridDim.x);
    for (int c = threadIdx.x; c < W; c += T)
        w[c] = a.w ? a.w[c] : 1.0f;
    f2_t wv[NQ][2], dw[NQ][2], db[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        quad_params<V>(a.w, 1.0f, col(j), T, W, wv[j]);
        dw[j][0] = dw[j][1] = db[j][0] = db[j][1] = f2_both(0.0f);
    }

    int st = 0;
    uint32_t phase = 0;
    for (; tile < tiles; tile += gridDim.x) {
        const int here = rows_of(tile);
        cp_async_wait<kNormStages - 1>();
        const bool ok = mbar_wait_bounded(&full[st], phase, kBulkPolls);
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0) {
                raise_device_error(kErrTrainCopy);
                // the copies still in flight are waited for, with the same bound
                if (tile + gridDim.x < tiles)
                    mbar_wait_bounded(&full[st ^ 1], st ? phase ^ 1u : phase, kBulkPolls);
            }
            return;
        }
        const X *xs = reinterpret_cast<const X *>(buf + st * stage + in16(x, tile * R * W));
        const Y *gs = reinterpret_cast<const Y *>(buf + st * stage + args.x_bytes + in16(dy, tile * R * W));
        const float *es = reinterpret_cast<const float *>(buf + st * stage + args.x_bytes + args.dy_bytes +
                                                          in16(a.ds, tile * R * W));
        if (warp / share < here) {
            const int k = warp / share, part = warp - k * share;
            const X *xk = xs + k * W;
            const Y *gk = gs + k * W;
            const f2_t m = f2_both(-stats[st][k][0]), q = f2_both(stats[st][k][1]);
            f2_t s0 = f2_both(0.0f), s1 = s0;
            auto one = [&](auto all, int c) {
                constexpr bool ALL = decltype(all)::value;
                QX xq;
                QY gq;
                QF wq;
                f2_t h[2], g[2], wc[2];
                xq.template load<ALL>(xk, c, 32, W);
                gq.template load<ALL>(gk, c, 32, W);
                wq.template load<ALL>(w, c, 32, W);
                xq.pairs(h);
                gq.pairs(g);
                wq.pairs(wc);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    g[i] = f2_mul(g[i], wc[i]);
                    s0 = f2_add(s0, g[i]);
                    s1 = f2_fma(g[i], f2_mul(f2_add(h[i], m), q), s1);
                }
            };
            int c = part * 128;
#pragma unroll 4
            for (; c + 128 <= W; c += share * 128)
                one(std::true_type{}, c + lane * V);
            if (c < W)
                one(std::false_type{}, c + lane * V);
            float m0, m1, hi;
            f2_unpack(s0, m0, hi);
            m0 += hi;
            f2_unpack(s1, m1, hi);
            m1 += hi;
            warp_sum2(m0, m1);
            if (lane == 0)
                parts[k][part] = make_float2(m0, m1);
        }
        __syncthreads();
        float *dxp = a.dx + tile * R * W;
        for (int k = 0; k < here; ++k, dxp += W, xs += W, gs += W, es += W) {
            const float rstd = stats[st][k][1];
            const f2_t m = f2_both(-stats[st][k][0]), q = f2_both(rstd);
            float m0 = parts[k][0].x, m1 = parts[k][0].y;
            for (int p = 1; p < share; ++p) {
                m0 += parts[k][p].x;
                m1 += parts[k][p].y;
            }
            const f2_t c1 = f2_both(-m1 * a.inv_w), c0 = f2_both(-rstd * (m0 * a.inv_w));
            auto one = [&](auto all, int j) {
                constexpr bool ALL = decltype(all)::value;
                QX xq;
                QY gq;
                f2_t h[2], g[2], o[2];
                xq.template load<ALL>(xs, col(j), T, W);
                gq.template load<ALL>(gs, col(j), T, W);
                xq.pairs(h);
                gq.pairs(g);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[i] = f2_mul(f2_add(h[i], m), q);
                    dw[j][i] = f2_fma(g[i], h[i], dw[j][i]);
                    db[j][i] = f2_add(db[j][i], g[i]);
                    o[i] = f2_fma(f2_fma(h[i], c1, f2_mul(g[i], wv[j][i])), q, c0);
                }
                if (a.ds) {
                    QF eq;
                    f2_t t[2];
                    eq.template load<ALL>(es, col(j), T, W);
                    eq.pairs(t);
                    o[0] = f2_add(o[0], t[0]);
                    o[1] = f2_add(o[1], t[1]);
                }
                QF::template store<ALL>(dxp, col(j), T, W, o);
            };
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                if (4 * T * (j + 1) <= W)
                    one(std::true_type{}, j);
                else if (4 * T * j < W)
                    one(std::false_type{}, j);
            }
        }
        __syncthreads();  // every thread is done with the stage
        fetch(st, tile + static_cast<long long>(kNormStages) * gridDim.x);
        if (++st == kNormStages) {
            st = 0;
            phase ^= 1u;
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
__global__ void __launch_bounds__(kNormWideThreads) s6_layernorm_bwd_wide_sums_kernel(const NormBwdArgs a,
                                                                                    float2 *sums) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ float red[2][kNormWideThreads / 32];
    const int W = a.width;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const X *x = static_cast<const X *>(a.x) + row * W;
        const Y *dy = static_cast<const Y *>(a.dy) + row * W;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s0 = 0.0f, s1 = 0.0f;
        for (int c = threadIdx.x * V; c < W; c += kNormWideThreads * V) {
            float h[V], g[V];
            VX::unpack(VX::load(x + c), h);
            VY::unpack(VY::load(dy + c), g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = g[i] * (a.w ? a.w[c + i] : 1.0f);
                s0 += t;
                s1 = fmaf(t, (h[i] - mean) * rstd, s1);
            }
        }
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
