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
// are worked on.  dw and dconv_b stay in registers over all runs of a warp,
// the block adds its warps up, and s6_sum_parts_kernel adds up the blocks in a
// fixed order.
#pragma once

#include "s6_vec.cuh"

namespace s6 {

constexpr int kConvBwdWarps = 4;
constexpr int kConvBwdGroup = 4;  // tokens fetched together

struct ConvBwdArgs {
    int Bt, L, d;
    int run, runs;  // tokens of a run, runs of a sequence
    const void *x, *dout;
    const float *conv_w, *conv_b;  // conv_b may be null
    float *dx;
    float *part;  // [gridDim.y][K + 1][d]
};

template <typename X, typename G, int V, int K>
__global__ void __launch_bounds__(32 * kConvBwdWarps) s6_conv_silu_bwd_kernel(const ConvBwdArgs a) {
    using VX = IoVec<X, V>;
    using VG = IoVec<G, V>;
    using VF = IoVec<float, V>;
    constexpr int H = K - 1, U = kConvBwdGroup;
    __shared__ float sums[K + 1][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * V;
    const bool live = c < a.d;  // d is a multiple of V
    const int d = a.d, L = a.L;

    float w[K][V], cb[V], dw[K][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            w[k][i] = live ? a.conv_w[static_cast<long long>(c + i) * K + k] : 0.0f;
            dw[k][i] = 0.0f;
        }
        cb[i] = live && a.conv_b ? a.conv_b[c + i] : 0.0f;
        db[i] = 0.0f;
    }

    const long long units = static_cast<long long>(a.Bt) * a.runs;
    const long long workers = static_cast<long long>(gridDim.y) * kConvBwdWarps;
    for (long long u = static_cast<long long>(blockIdx.y) * kConvBwdWarps + warp; live && u < units; u += workers) {
        const int b = static_cast<int>(u / a.runs);
        const int t0 = static_cast<int>(u - static_cast<long long>(b) * a.runs) * a.run;
        const int t1 = L - t0 < a.run ? L : t0 + a.run;
        const int end = t1 + H;                  // steps t0 .. end-1; rows from L on are not read
        const int rows_end = end < L ? end : L;
        const long long base = static_cast<long long>(b) * L * d + c;
        const X *x = static_cast<const X *>(a.x) + base;
        const G *g = static_cast<const G *>(a.dout) + base;
        float *dx = a.dx + base;

        float xw[K][V];  // x_{t-K+1} .. x_t
        float dv[K][V];  // dv_{t-K+1} .. dv_t
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                xw[k][i] = dv[k][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < H; ++k) {  // x_{t0-K+1} .. x_{t0-1} into slots 1 .. K-1
            const int t = t0 - H + k;
            if (t >= 0)
                VX::unpack(VX::load(x + static_cast<long long>(t) * d), xw[k + 1]);
        }
        typename VX::raw xr[U];
        typename VG::raw gr[U];
        auto fetch = [&](int t) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const bool in = t + j < rows_end;
                xr[j] = in ? VX::load(x + static_cast<long long>(t + j) * d) : VX::zero();
                gr[j] = in ? VG::load(g + static_cast<long long>(t + j) * d) : VG::zero();
            }
        };
        fetch(t0);
        for (int t = t0; t < end; t += U) {
            float xt[U][V], gt[U][V];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                VX::unpack(xr[j], xt[j]);
                VG::unpack(gr[j], gt[j]);
            }
            if (t + U < end)
                fetch(t + U);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int tj = t + j;
                if (tj < end) {
                    const bool mine = tj < t1, inside = tj < L;
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
#pragma unroll
                        for (int k = 0; k < H; ++k) {
                            xw[k][i] = xw[k + 1][i];
                            dv[k][i] = dv[k + 1][i];
                        }
                        xw[H][i] = xt[j][i];
                        float v = cb[i];
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            v = fmaf(w[k][i], xw[k][i], v);
                        const float p = rcp_approx(1.0f + ex2_approx(-v * kLog2e));
                        const float e = gt[j][i] * (p * fmaf(v, 1.0f - p, 1.0f));
                        dv[H][i] = inside ? e : 0.0f;
                        if (mine) {
#pragma unroll
                            for (int k = 0; k < K; ++k)
                                dw[k][i] = fmaf(dv[H][i], xw[k][i], dw[k][i]);
                            db[i] += dv[H][i];
                        }
                        o[i] = 0.0f;
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            o[i] = fmaf(w[k][i], dv[H - k][i], o[i]);
                    }
                    if (tj >= t0 + H)
                        VF::store(dx + static_cast<long long>(tj - H) * d, VF::pack(o));
                }
            }
        }
    }

    // the block's warps hold sums of the same channels: add them up in order
    for (int s = 0; s < kConvBwdWarps; ++s) {
        if (warp == s) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    sums[k][lane * V + i] = s ? sums[k][lane * V + i] + dw[k][i] : dw[k][i];
                sums[K][lane * V + i] = s ? sums[K][lane * V + i] + db[i] : db[i];
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
