// s6_conv_bwd.cuh -- gradients of the standalone causal depthwise conv + SiLU,
// sm_100a.
//
// "mamba, live" (what is actually running): xc = SiLU(depthwise_conv4(xin)).
// With v_t = conv_b + sum_k w_k x_{t-K+1+k} (x = 0 before token 0) and
// p = 1 / (1 + e^-v), for one channel of one sequence:
//
//     dv_t = dout_t p (1 + v_t (1 - p))
//     dx_t = sum_k w_k dv_{t+K-1-k}          (dv = 0 behind the last token)
//     dw_k = sum_t dv_t x_{t-K+1+k},  dconv_b = sum_t dv_t
//
// HBM-bound: x and dout read, dx written.  A thread owns V channels (one
// vector of every row; a warp covers 32 V consecutive channels) and walks a
// run of tokens forward, with the last K-1 inputs and the last K-1 dv in
// registers: the token that completes dv_t also completes dx_{t-K+1}.  A run
// of tokens [t0, t1) reads K-1 rows before it (inputs only) and K-1 behind it
// (for the dv that dx of its last tokens needs; these add nothing to dw).
// Rows of the next kConvBwdGroup tokens are in flight while the present ones
// are worked on, and the arithmetic runs on float32 pairs.  dw and dconv_b stay in registers over all runs of a warp,
// the block adds its warps up, and s6_sum_parts_kernel adds up the blocks in a
// fixed order.
#pragma once

#include <type_traits>

#include "s6_vec.cuh"

namespace s6 {

constexpr int kConvBwdWarps = 4;
constexpr int kConvBwdGroup = 4;   // tokens of the inner loop, each fetched one group ahead
constexpr int kConvBwdPerSM = 4;   // resident blocks (128 registers a thread)

struct ConvBwdArgs {
    int Bt, L, d;
    int run, runs;  // tokens of a run, runs of a sequence
    const void *x, *dout;
    const float *conv_w, *conv_b;  // conv_b may be null
    float *dx;
    float *part;  // [gridDim.y][K + 1][d]
};

// V channels as float32 pairs (a last odd one beside a zero).
template <typename T, int V>
__device__ __forceinline__ void conv_pairs(const typename IoVec<T, V>::raw &r, f2_t (&p)[(V + 1) / 2]) {
    float f[V];
    IoVec<T, V>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < V; i += 2)
        p[i / 2] = f2_pack(f[i], i + 1 < V ? f[i + 1 < V ? i + 1 : i] : 0.0f);
}

template <typename X, typename G, int V, int K>
__global__ void __launch_bounds__(32 * kConvBwdWarps, kConvBwdPerSM) s6_conv_silu_bwd_kernel(const ConvBwdArgs a) {
    using VX = IoVec<X, V>;
    using VG = IoVec<G, V>;
    using VF = IoVec<float, V>;
    constexpr int H = K - 1, U = kConvBwdGroup, P = (V + 1) / 2;
    static_assert(H < U, "the first group of a run holds the tokens that complete no dx of it");
    __shared__ float sums[K + 1][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * V;
    const bool live = c < a.d;  // d is a multiple of V
    const int d = a.d, L = a.L;

    f2_t w[K][P], cb[P], dw[K][P], db[P];
    const f2_t zero = f2_pack(0.0f, 0.0f), one = f2_pack(1.0f, 1.0f), minus = f2_pack(-1.0f, -1.0f);
    {
        auto param = [&](const float *p, int i, int stride, int at) {
            return live && p && i < V ? p[static_cast<long long>(c + i) * stride + at] : 0.0f;
        };
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                w[k][p] = f2_pack(param(a.conv_w, 2 * p, K, k), param(a.conv_w, 2 * p + 1, K, k));
                dw[k][p] = zero;
            }
            cb[p] = f2_pack(param(a.conv_b, 2 * p, 1, 0), param(a.conv_b, 2 * p + 1, 1, 0));
            db[p] = zero;
        }
    }

    const long long units = static_cast<long long>(a.Bt) * a.runs;
    const long long workers = static_cast<long long>(gridDim.y) * kConvBwdWarps;
    for (long long u = static_cast<long long>(blockIdx.y) * kConvBwdWarps + warp; live && u < units; u += workers) {
        const int b = static_cast<int>(u / a.runs);
        const int t0 = static_cast<int>(u - static_cast<long long>(b) * a.runs) * a.run;
        const int t1 = L - t0 < a.run ? L : t0 + a.run;
        const int end = t1 + H;                        // steps t0 .. end-1
        const int rows = end < L ? end : L;            // rows from here on are not read
        const long long first = (static_cast<long long>(b) * L + t0) * d + c;
        const X *xp = static_cast<const X *>(a.x) + first;     // row t of the loop, then of its fetches
        const G *gp = static_cast<const G *>(a.dout) + first;
        float *dxp = a.dx + first - static_cast<long long>(H) * d;  // row t - H

        f2_t xw[K][P];  // x_{t-K+1} .. x_t
        f2_t dv[K][P];  // dv_{t-K+1} .. dv_t
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < K; ++k)
                xw[k][p] = dv[k][p] = zero;
#pragma unroll
        for (int k = 0; k < H; ++k)  // x_{t0-K+1} .. x_{t0-1} into slots 1 .. K-1
            if (t0 - H + k >= 0)
                conv_pairs<X, V>(VX::load(xp - static_cast<long long>(H - k) * d), xw[k + 1]);
        typename VX::raw xr[U];
        typename VG::raw gr[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool in = t0 + j < rows;
            xr[j] = in ? VX::load(xp) : VX::zero();
            gr[j] = in ? VG::load(gp) : VG::zero();
            xp += d;
            gp += d;
        }
        // A group of U tokens.  EDGE: it may hold tokens before t0 + H, from t1 on or from L
        // on, or its fetches may; elsewhere no token is looked at.
        auto group = [&](auto edge, int t) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int tj = t + j;
                f2_t g[P];
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        xw[k][p] = xw[k + 1][p];
                        dv[k][p] = dv[k + 1][p];
                    }
                conv_pairs<X, V>(xr[j], xw[H]);
                conv_pairs<G, V>(gr[j], g);
                if (!EDGE || tj + U < rows) {
                    xr[j] = VX::load(xp);
                    gr[j] = VG::load(gp);
                }
                xp += d;
                gp += d;
                float o[2 * P];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    f2_t v = cb[p];
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        v = f2_fma(w[k][p], xw[k][p], v);
                    float e0, e1, q0, q1;
                    f2_unpack(f2_mul(v, f2_pack(-kLog2e, -kLog2e)), e0, e1);
                    f2_unpack(f2_add(f2_pack(ex2_approx(e0), ex2_approx(e1)), one), q0, q1);
                    const f2_t s = f2_pack(rcp_approx(q0), rcp_approx(q1));
                    const f2_t f = f2_mul(s, f2_fma(v, f2_fma(s, minus, one), one));
                    dv[H][p] = f2_mul(g[p], f);
                    if (EDGE && tj >= L)
                        dv[H][p] = zero;
                    if (!EDGE || tj < t1) {
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            dw[k][p] = f2_fma(dv[H][p], xw[k][p], dw[k][p]);
                        db[p] = f2_add(db[p], dv[H][p]);
                    }
                    f2_t r = f2_mul(w[0][p], dv[H][p]);
#pragma unroll
                    for (int k = 1; k < K; ++k)
                        r = f2_fma(w[k][p], dv[H - k][p], r);
                    f2_unpack(r, o[2 * p], o[2 * p + 1]);
                }
                if (!EDGE || (tj >= t0 + H && tj < end)) {
                    float st[V];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        st[i] = o[i];
                    VF::store(dxp, VF::pack(st));
                }
                dxp += d;
            }
        };
        for (int t = t0; t < end; t += U) {
            if (t > t0 && t + U <= t1 && t + 2 * U <= rows)
                group(std::false_type{}, t);
            else
                group(std::true_type{}, t);
        }
    }

    // the block's warps hold sums of the same channels: add them up in order
    for (int s = 0; s < kConvBwdWarps; ++s) {
        if (warp == s) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int k = 0; k <= K; ++k) {
                    float v[2];
                    f2_unpack(k < K ? dw[k < K ? k : 0][p] : db[p], v[0], v[1]);
#pragma unroll
                    for (int i = 0; i < 2 && 2 * p + i < V; ++i) {
                        float &at = sums[k][lane * V + 2 * p + i];
                        at = s ? at + v[i] : v[i];
                    }
                }
        }
        __syncthreads();
    }
    float *part = a.part + static_cast<long long>(blockIdx.y) * (K + 1) * d;
    for (int i = threadIdx.x; i < (K + 1) * 32 * V; i += 32 * kConvBwdWarps) {
        const int k = i / (32 * V), j = i - k * 32 * V, ch = blockIdx.x * 32 * V + j;
        if (ch < d)
            part[static_cast<long long>(k) * d + ch] = sums[k][j];
    }
}

}  // namespace s6
