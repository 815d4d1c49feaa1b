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
// Both are bound by HBM: a row is read once into registers, in the storage
// type, and everything is computed in float32 from there.  A row belongs to
// one warp up to kNormWarpWidth elements and to one block above that; the warp
// or block walks rows with a fixed stride and fetches the next row while it
// reduces the present one.  Rows above kNormMaxWidth take the _wide kernels,
// which read a row more than once.
#pragma once

#include "s6_vec.cuh"

namespace s6 {

constexpr int kNormWarpWidth = 512;   // widest row of one warp: 16 elements a lane
constexpr int kNormBlockWarps = 4;    // warps (rows in flight) of a block of one-warp rows
constexpr int kNormMaxWidth = 8192;   // widest row held in registers
constexpr int kNormMaxWarps = 32;     // warps that share a row, at most

// Elements of a row that a thread holds where several warps share it.  The
// backward, which also holds sums for each of its columns, takes 16 above 4096
// (fewer, larger threads: a block's registers are bounded).
constexpr int norm_block_elems(int64_t width, bool bwd) { return bwd && width > 4096 ? 16 : 8; }
// Warps resident on an SM, by the elements that a thread holds: what the
// registers allow (the launch bounds below hold the compiler to it).
constexpr int norm_warps_resident(int elems, bool one_warp, bool bwd) {
    return one_warp ? (bwd ? (elems <= 4 ? 24 : elems <= 8 ? 20 : elems <= 12 ? 16 : 12)
                           : (elems <= 4 ? 32 : elems <= 8 ? 28 : elems <= 12 ? 20 : 16))
                    : (bwd ? (elems <= 8 ? 21 : 16) : 32);
}
constexpr int norm_max_threads(int elems, bool one_warp, bool bwd) {
    return one_warp ? 32 * kNormBlockWarps : 32 * norm_warps_resident(elems, false, bwd);
}
constexpr int norm_min_blocks(int elems, bool one_warp, bool bwd) {
    return one_warp ? norm_warps_resident(elems, true, bwd) / kNormBlockWarps : 1;
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

// The sum of v over the threads of a row: a warp's, or a block's through `red`
// (one slot a warp; the slots behind the block's own warps are zero).  Every
// thread adds the slots in the same order.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red, int nwarps) {
    v = warp_sum(v);
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < nwarps; i += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(red + i);
            v += (t.x + t.y) + (t.z + t.w);
        }
    }
    return v;
}

// Zeroes `n` slots; the first barrier of row_sum's caller comes after it.
__device__ __forceinline__ void clear_slots(float *red, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        red[i] = 0.0f;
    __syncthreads();
}

template <typename X, typename Y, int V, int NV, bool WARP>
__global__ void __launch_bounds__(norm_max_threads(NV *V, WARP, false), norm_min_blocks(NV *V, WARP, false))
    s6_layernorm_fwd_kernel(const NormFwdArgs a) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ __align__(16) float red[2][kNormMaxWarps];
    if constexpr (!WARP)
        clear_slots(red[0], 2 * kNormMaxWarps);
    const int nwarps = blockDim.x >> 5;
    const int G = WARP ? 32 : blockDim.x;                     // threads of a row
    const int li = WARP ? (threadIdx.x & 31) : threadIdx.x;  // this thread among them
    const int W = a.width;
    const X *x = static_cast<const X *>(a.x);
    const Y *r = static_cast<const Y *>(a.r);
    X *s = static_cast<X *>(a.s);
    Y *y = static_cast<Y *>(a.y);

    float wv[NV][V], bv[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (j * G + li) * V + i;
            wv[j][i] = a.w && c < W ? a.w[c] : 1.0f;
            bv[j][i] = a.b && c < W ? a.b[c] : 0.0f;
        }

    const long long per = WARP ? nwarps : 1;
    const long long step = per * gridDim.x;
    long long row = per * blockIdx.x + (WARP ? (threadIdx.x >> 5) : 0);
    typename VX::raw xr[NV];
    typename VY::raw rr[NV];
    const int c0 = li * V, dc = G * V;  // this thread's first column, and from one to the next
    auto fetch = [&](long long at) {
        const X *xp = x + at * W + c0;
        const Y *rp = r + at * W + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = c0 + j * dc < W;
            xr[j] = in ? VX::load(xp + j * dc) : VX::zero();
            if (r)
                rr[j] = in ? VY::load(rp + j * dc) : VY::zero();
        }
    };
    if (row < a.rows)
        fetch(row);
    for (; row < a.rows; row += step) {
        float v[NV][V], sum = 0.0f;
        X *sp = s + row * W + c0;
        Y *yp = y + row * W + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            VX::unpack(xr[j], v[j]);
            if (r) {
                float t[V];
                VY::unpack(rr[j], t);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[j][i] += t[i];
                if (s && c0 + j * dc < W)
                    VX::store(sp + j * dc, VX::pack(v[j]));
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum += v[j][i];
        }
        if (row + step < a.rows)
            fetch(row + step);
        const float mean = row_sum<WARP>(sum, red[0], nwarps) * a.inv_w;
        // squares of the deviations from the mean, not of the values: a mean that is
        // large next to the deviations costs no digits
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (c0 + j * dc < W) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[j][i] -= mean;
                    sq = fmaf(v[j][i], v[j][i], sq);
                }
            }
        const float rstd = __frsqrt_rn(row_sum<WARP>(sq, red[1], nwarps) * a.inv_w + a.eps);
        if (li == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (c0 + j * dc < W) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o[i] = fmaf(v[j][i] * rstd, wv[j][i], bv[j][i]);
                VY::store(yp + j * dc, VY::pack(o));
            }
        }
    }
}

// Rows that do not fit a block's registers: a block walks its row three times
// (sum, squared deviations, output); the second and third reads hit L2.  s is
// written on the last walk, since it may be x itself.
constexpr int kNormWideThreads = 512;

template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kNormWideThreads) s6_layernorm_fwd_wide_kernel(const NormFwdArgs a) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    __shared__ __align__(16) float red[2][kNormMaxWarps];
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
        const float mean = row_sum<false>(sum, red[0], kNormWideThreads / 32) * a.inv_w;
        for (int c = threadIdx.x * V; c < W; c += kNormWideThreads * V) {
            float v[V];
            value(c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sq = fmaf(v[i] - mean, v[i] - mean, sq);
        }
        const float rstd = __frsqrt_rn(row_sum<false>(sq, red[1], kNormWideThreads / 32) * a.inv_w + a.eps);
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
// A thread owns the same columns of every row it meets, so dw and db stay in
// its registers until the block's last row; the block then writes one row of
// partial sums and s6_sum_parts_kernel adds those up.
template <typename X, typename Y, int V, int NV, bool WARP>
__global__ void __launch_bounds__(norm_max_threads(NV *V, WARP, true), norm_min_blocks(NV *V, WARP, true))
    s6_layernorm_bwd_kernel(const NormBwdArgs a) {
    using VX = IoVec<X, V>;
    using VY = IoVec<Y, V>;
    using VF = IoVec<float, V>;
    __shared__ __align__(16) float red[2][2][kNormMaxWarps];
    if constexpr (!WARP)
        clear_slots(red[0][0], 4 * kNormMaxWarps);
    const int nwarps = blockDim.x >> 5;
    const int G = WARP ? 32 : blockDim.x;
    const int li = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int W = a.width;
    const X *x = static_cast<const X *>(a.x);
    const Y *dy = static_cast<const Y *>(a.dy);

    float wv[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (j * G + li) * V + i;
            wv[j][i] = a.w && c < W ? a.w[c] : 1.0f;
            dw[j][i] = 0.0f;
            db[j][i] = 0.0f;
        }

    const long long per = WARP ? nwarps : 1;
    const long long step = per * gridDim.x;
    long long row = per * blockIdx.x + (WARP ? (threadIdx.x >> 5) : 0);
    typename VX::raw xr[NV];
    typename VY::raw gr[NV];
    float mean = 0.0f, rstd = 0.0f;
    const int c0 = li * V, dc = G * V;
    auto fetch = [&](long long at) {
        mean = a.mean[at];
        rstd = a.rstd[at];
        const X *xp = x + at * W + c0;
        const Y *gp = dy + at * W + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = c0 + j * dc < W;
            xr[j] = in ? VX::load(xp + j * dc) : VX::zero();
            gr[j] = in ? VY::load(gp + j * dc) : VY::zero();
        }
    };
    if (row < a.rows)
        fetch(row);
    int turn = 0;
    for (; row < a.rows; row += step) {
        float h[NV][V], g[NV][V], s0 = 0.0f, s1 = 0.0f;
        const float q = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            VX::unpack(xr[j], h[j]);
            VY::unpack(gr[j], g[j]);
            if (c0 + j * dc < W) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[j][i] = (h[j][i] - mean) * q;
                    dw[j][i] = fmaf(g[j][i], h[j][i], dw[j][i]);
                    db[j][i] += g[j][i];
                    g[j][i] *= wv[j][i];
                    s0 += g[j][i];
                    s1 = fmaf(g[j][i], h[j][i], s1);
                }
            }
        }
        if (row + step < a.rows)
            fetch(row + step);
        const float *dsp = a.ds + row * W + c0;
        float *dxp = a.dx + row * W + c0;
        typename VF::raw dsr[NV];
        if (a.ds) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                dsr[j] = c0 + j * dc < W ? VF::load(dsp + j * dc) : VF::zero();
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        if constexpr (!WARP) {
            // two slots by turns: a slot is written again only after the barrier of the
            // row between, which every reader of it has passed
            float(*slot)[kNormMaxWarps] = red[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) {
                slot[0][threadIdx.x >> 5] = s0;
                slot[1][threadIdx.x >> 5] = s1;
            }
            __syncthreads();
            s0 = s1 = 0.0f;
            for (int i = 0; i < nwarps; i += 4) {
                const float4 t0 = *reinterpret_cast<const float4 *>(slot[0] + i);
                const float4 t1 = *reinterpret_cast<const float4 *>(slot[1] + i);
                s0 += (t0.x + t0.y) + (t0.z + t0.w);
                s1 += (t1.x + t1.y) + (t1.z + t1.w);
            }
        }
        const float m0 = s0 * a.inv_w, m1 = s1 * a.inv_w;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (c0 + j * dc < W) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o[i] = q * (g[j][i] - fmaf(h[j][i], m1, m0));
                if (a.ds) {
                    float t[V];
                    VF::unpack(dsr[j], t);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o[i] += t[i];
                }
                VF::store(dxp + j * dc, VF::pack(o));
            }
        }
    }

    if (!a.part)
        return;
    float *part = a.part + static_cast<long long>(blockIdx.x) * 2 * W;
    if constexpr (WARP) {
        // the block's warps hold sums of the same columns: add them up in order
        __shared__ float sums[2][kNormWarpWidth];
        for (int k = 0; k < nwarps; ++k) {
            if ((threadIdx.x >> 5) == k) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int c = (j * 32 + li) * V + i;
                        sums[0][c] = k ? sums[0][c] + dw[j][i] : dw[j][i];
                        sums[1][c] = k ? sums[1][c] + db[j][i] : db[j][i];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < W; c += blockDim.x) {
            part[c] = sums[0][c];
            part[W + c] = sums[1][c];
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (j * G + li) * V + i;
                if (c < W) {
                    part[c] = dw[j][i];
                    part[W + c] = db[j][i];
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
    __shared__ __align__(16) float red[2][kNormMaxWarps];
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
        s0 = row_sum<false>(s0, red[0], kNormWideThreads / 32);
        s1 = row_sum<false>(s1, red[1], kNormWideThreads / 32);
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
