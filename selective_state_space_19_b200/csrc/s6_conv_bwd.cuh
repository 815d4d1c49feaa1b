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
// HBM-bound: x and dout read, dx written.  A thread owns V channels, a float32
// pair (a single channel beside a zero where rows do not keep pairs aligned),
// and walks a run of tokens forward with the last K-1 inputs and the last K-1
// dv in registers: the token that completes dv_t also completes dx_{t-K+1}.  A
// run of tokens [t0, t1) reads K-1 rows before it (inputs only) and K-1 behind
// it (for the dv that dx of its last tokens needs; these add nothing to dw).
// Rows of the next kConvBwdGroup tokens are in flight while the present ones
// are worked on.  dw and dconv_b are float32 sums over a run (kConvBwdMaxRun
// tokens at most) and float64 sums over the runs of a block's warps, which
// s6_sum_parts_kernel then adds up over the blocks in a fixed order.
//
// Measured on one B200 (copies run at 6,521 GB/s): 16x8192x1536 f32 379 us = 98 %
// of the copy rate, with bfloat16 x 355 = 87 % (370 = 83 % where the inputs change
// from call to call), all bfloat16 335 = 74 % (bound by issue and the latency of 16
// warps an SM); 8x256x1536 f32 14 us = 40 % (its runs of 22 tokens take 25 steps and
// walk 32, three of their four groups guarded); 16x2048x1535 f32 143 us = 65 % (half
// of every pair is a zero).  Four
// channels and groups of 4 tokens (the registers allow no more) took 457, 352,
// 321 and 17 us; groups of 6 tokens 397, 384, 359 and 14.
#pragma once

#include <type_traits>

#include "s6_vec.cuh"

namespace s6 {

constexpr int kConvBwdWarps = 4;
constexpr int kConvBwdGroup = 8;   // tokens of the inner loop, each fetched one group ahead
constexpr int kConvBwdPerSM = 4;   // resident blocks (128 registers a thread)
constexpr int kConvBwdMaxRun = 1024;  // tokens that float32 sums run over, at most; off by 5e-7 of the result in runs of 683

struct ConvBwdArgs {
    int Bt, L, d;
    int run, runs;  // tokens of a run, runs of a sequence
    const void *x, *dout;
    const float *conv_w, *conv_b;  // conv_b may be null
    float *dx;
    float *part;  // [gridDim.y][K + 1][d]
};

// V channels as a float32 pair.
template <typename T, int V>
__device__ __forceinline__ f2_t conv_pair(const typename IoVec<T, V>::raw &r) {
    if constexpr (V == 1) {
        float f[1];
        IoVec<T, 1>::unpack(r, f);
        return f2_pack(f[0], 0.0f);
    } else if constexpr (sizeof(T) == 2) {
        return f2_pack(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    } else {
        return f2_pack(__uint_as_float(r.x), __uint_as_float(r.y));
    }
}

template <typename X, typename G, int V, int K>
__global__ void __launch_bounds__(32 * kConvBwdWarps, kConvBwdPerSM) s6_conv_silu_bwd_kernel(const ConvBwdArgs a) {
    using VX = IoVec<X, V>;
    using VG = IoVec<G, V>;
    using VF = IoVec<float, V>;
    constexpr int H = K - 1, U = kConvBwdGroup;
    static_assert(V <= 2, "a thread's channels are one pair");
    static_assert(H < U, "the first group of a run holds the tokens that complete no dx of it");
    __shared__ double sums[K + 1][V][32 * kConvBwdWarps];  // each thread's own, over its runs
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * V;
    const bool live = c < a.d;  // d is a multiple of V
    const int d = a.d, L = a.L;

    const f2_t zero = f2_pack(0.0f, 0.0f), one = f2_pack(1.0f, 1.0f), minus = f2_pack(-1.0f, -1.0f);
    auto param = [&](const float *p, int i, int stride, int at) {
        return live && p && i < V ? p[static_cast<long long>(c + i) * stride + at] : 0.0f;
    };
    f2_t w[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        w[k] = f2_pack(param(a.conv_w, 0, K, k), param(a.conv_w, 1, K, k));
    const f2_t cb = f2_pack(param(a.conv_b, 0, 1, 0), param(a.conv_b, 1, 1, 0));

#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
            sums[k][i][threadIdx.x] = 0.0;

    const long long units = static_cast<long long>(a.Bt) * a.runs;
    const long long workers = static_cast<long long>(gridDim.y) * kConvBwdWarps;
    for (long long u = static_cast<long long>(blockIdx.y) * kConvBwdWarps + warp; live && u < units; u += workers) {
        const int b = static_cast<int>(u / a.runs);
        const int t0 = static_cast<int>(u - static_cast<long long>(b) * a.runs) * a.run;
        const int t1 = L - t0 < a.run ? L : t0 + a.run;
        const int end = t1 + H;              // steps t0 .. end-1
        const int rows = end < L ? end : L;  // rows from here on are not read
        const long long first = (static_cast<long long>(b) * L + t0) * d + c;
        const X *xp = static_cast<const X *>(a.x) + first;  // the next row to be fetched
        const G *gp = static_cast<const G *>(a.dout) + first;
        float *dxp = a.dx + first - static_cast<long long>(H) * d;  // row t - H

        f2_t xw[K], dv[K];  // x_{t-K+1} .. x_t and dv_{t-K+1} .. dv_t
        f2_t dw[K], db = zero;
#pragma unroll
        for (int k = 0; k < K; ++k)
            xw[k] = dv[k] = dw[k] = zero;
#pragma unroll
        for (int k = 0; k < H; ++k)  // x_{t0-K+1} .. x_{t0-1} into slots 1 .. K-1
            if (t0 - H + k >= 0)
                xw[k + 1] = conv_pair<X, V>(VX::load(xp - static_cast<long long>(H - k) * d));
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
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    xw[k] = xw[k + 1];
                    dv[k] = dv[k + 1];
                }
                xw[H] = conv_pair<X, V>(xr[j]);
                const f2_t g = conv_pair<G, V>(gr[j]);
                if (!EDGE || tj + U < rows) {
                    xr[j] = VX::load(xp);
                    gr[j] = VG::load(gp);
                }
                xp += d;
                gp += d;
                f2_t v = cb;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    v = f2_fma(w[k], xw[k], v);
                float e0, e1, q0, q1;
                f2_unpack(f2_mul(v, f2_pack(-kLog2e, -kLog2e)), e0, e1);
                f2_unpack(f2_add(f2_pack(ex2_approx(e0), ex2_approx(e1)), one), q0, q1);
                const f2_t s = f2_pack(rcp_approx(q0), rcp_approx(q1));
                dv[H] = f2_mul(g, f2_mul(s, f2_fma(v, f2_fma(s, minus, one), one)));
                if (EDGE && tj >= L)
                    dv[H] = zero;
                if (!EDGE || tj < t1) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        dw[k] = f2_fma(dv[H], xw[k], dw[k]);
                    db = f2_add(db, dv[H]);
                }
                f2_t r = f2_mul(w[0], dv[H]);
#pragma unroll
                for (int k = 1; k < K; ++k)
                    r = f2_fma(w[k], dv[H - k], r);
                if (!EDGE || (tj >= t0 + H && tj < end)) {
                    float o[2], st[V];
                    f2_unpack(r, o[0], o[1]);
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
#pragma unroll
        for (int k = 0; k <= K; ++k) {
            float v[2];
            f2_unpack(k < K ? dw[k < K ? k : 0] : db, v[0], v[1]);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sums[k][i][threadIdx.x] += static_cast<double>(v[i]);
        }
    }

    // the block's warps hold sums of the same channels: add them up in order
    __syncthreads();
    float *part = a.part + static_cast<long long>(blockIdx.y) * (K + 1) * d;
    for (int e = threadIdx.x; e < (K + 1) * 32 * V; e += 32 * kConvBwdWarps) {
        const int k = e / (32 * V), j = e - k * 32 * V, ch = blockIdx.x * 32 * V + j;
        if (ch < d) {
            double s = 0.0;
#pragma unroll
            for (int q = 0; q < kConvBwdWarps; ++q)
                s += sums[k][j % V][32 * q + j / V];
            part[static_cast<long long>(k) * d + ch] = static_cast<float>(s);
        }
    }
}

}  // namespace s6
