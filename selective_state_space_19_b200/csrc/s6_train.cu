// s6_train.cu -- the training-step operators around the scan, declared in
// include/s6.h: LayerNorm forward and backward, the conv's backward, the norm
// and the clipping of gradients.  Argument checks, choice of kernel and launch;
// the arithmetic is in s6_norm.cuh, s6_conv_bwd.cuh and s6_grads.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "s6.h"
#include "s6_common.cuh"
#include "s6_conv_bwd.cuh"
#include "s6_grads.cuh"
#include "s6_host.cuh"
#include "s6_norm.cuh"
#include "s6_vec.cuh"

namespace {

using namespace s6::host;
using bf16 = __nv_bfloat16;

// The grids below are sized for the 148 SMs of a B200 and do not ask the device,
// so the workspace of a call depends on its sizes alone.  Blocks never wait for
// one another: on fewer SMs they only take longer.
constexpr int64_t kSMs = 148;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A kernel whose blocks may start while the one before it on the stream drains;
// it waits for that one's results itself (cudaGridDependencySynchronize).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

int sum_parts(const float *part, int64_t rows, int64_t cols, int segs, int segs0, float *out0, float *out1,
              cudaStream_t st) {
    s6::SumPartsArgs a;
    a.part = part;
    a.rows = static_cast<int>(rows);
    a.cols = static_cast<int>(cols);
    a.segs = segs;
    a.segs0 = segs0;
    a.out0 = out0;
    a.out1 = out1;
    return launch_status(launch_after(s6::s6_sum_parts_kernel, dim3(static_cast<unsigned>(ceil_div(cols * segs, 32))),
                                      32 * s6::kSumPartsWarps, st, a));
}

int check_workspace(const void *ws, int64_t bytes, int64_t need) {
    if (need > 0 && (!ws || bytes < need))
        return S6_ERR_INVALID_ARG;
    return ws && !aligned_to(ws, 8) ? S6_ERR_ALIGNMENT : S6_OK;
}

// The memory of an argument.  kEach: read element by element, so an output may be the
// very same memory (as large, so of elements as large).
enum Use { kRead, kEach, kWritten };
struct Mem {
    const void *p;
    int64_t rows, row_bytes;
    Use use;
    uint64_t bytes() const {  // at most 2^66 by the checked sizes
        uint64_t n;
        return __builtin_mul_overflow(static_cast<uint64_t>(rows), static_cast<uint64_t>(row_bytes), &n) ? ~uint64_t(0) : n;
    }
};

// Refuses outputs that share memory with one another or with an input; the outputs are
// listed first.
template <size_t N>
int check_apart(const Mem (&m)[N]) {
    uint64_t at[N], size[N];
    for (size_t i = 0; i < N; ++i) {
        at[i] = reinterpret_cast<uintptr_t>(m[i].p);
        size[i] = m[i].p ? m[i].bytes() : 0;
    }
    for (size_t i = 0; i < N && m[i].use == kWritten; ++i)  // these come first
        for (size_t j = i + 1; j < N; ++j) {
            const bool overlap = size[i] && size[j] && (at[i] <= at[j] ? at[j] - at[i] < size[i] : at[i] - at[j] < size[j]);
            if (overlap && !(m[j].use == kEach && at[i] == at[j] && size[i] == size[j]))
                return S6_ERR_INVALID_ARG;
        }
    return S6_OK;
}

// ---------------------------------------------------------------- LayerNorm
int check_norm_dims(const s6_norm_dims *dims) {
    if (!dims || dims->rows < 0 || dims->width < 1 || !std::isfinite(dims->eps) || dims->eps < 0.0f)
        return S6_ERR_INVALID_ARG;
    const bool types = (dims->x_dtype == S6_F32 && (dims->y_dtype == S6_F32 || dims->y_dtype == S6_BF16)) ||
                       (dims->x_dtype == S6_BF16 && dims->y_dtype == S6_BF16);
    if (!types || dims->width > (1 << 24) || dims->rows > (int64_t(1) << 40))
        return S6_ERR_UNSUPPORTED;
    return S6_OK;
}

// Rows of one warp or of some lanes: as many blocks as are resident, which walk the
// rows.
struct NormWarpPlan {
    int elems;  // elements of a row that a lane holds, at most
    int lanes;  // of a row: 32, or with 4 elements a lane the fewest that hold it, 2 at least
    int64_t blocks;
};

// `read`: bytes of a row that the forward reads where it also adds (0: it does not).
// Four streams of reads and writes are fastest with about 38 KB of reads in flight
// on an SM: 131072x384 f32 + f32 139 us with 20 warps (61 KB), 137 with 16, 132 with 12;
// f32 + bfloat16 106 with 20 (46 KB), 98 with 16, 109 with 12; bfloat16 71, 77, 85
// (31 KB with 20).  Without the add more warps are faster throughout.
constexpr int64_t kNormAddReads = 38 * 1024;

// Backward: rounds of the resident blocks, such that none of the `sums` rows of sums that
// one round keeps is over more than norm_run rows.
int64_t norm_rounds(int64_t rows, int64_t width, int64_t sums) {
    return ceil_div(rows, sums * s6::norm_run(static_cast<int>(width)));
}

NormWarpPlan norm_warp_plan(int64_t rows, int64_t width, bool bwd, int64_t read = 0) {
    NormWarpPlan p;
    p.elems = static_cast<int>(4 * ceil_div(width, 128));
    p.lanes = 32;
    while (p.lanes > 2 && 4 * (p.lanes / 2) >= width)
        p.lanes /= 2;
    const int64_t warp_rows = 32 / p.lanes;
    int64_t warps = s6::norm_warps_resident(p.elems, bwd);
    if (read)
        warps = std::min(warps, std::max<int64_t>(s6::kNormBlockWarps, kNormAddReads / (read * warp_rows)));
    p.blocks = std::min(ceil_div(rows, s6::kNormBlockWarps * warp_rows), kSMs * warps / s6::kNormBlockWarps);
    if (bwd)
        p.blocks *= norm_rounds(rows, width, p.blocks * s6::kNormBlockWarps * warp_rows);
    return p;
}

// Rows of a block: threads, quads of columns of a thread, rows of a step, blocks on
// an SM.
struct NormBlockPlan {
    int threads, quads, rows, per_sm;
    int64_t blocks;
};

constexpr int kSmemSM = 227 * 1024, kSmemBlock = 2 * 1024;  // of an SM; a block's other shared memory, at most
// by the registers: 128 a thread backward; forward 96 with four quads and 80 with fewer
// (float32 rows with four quads, two at a time, take 122: of 128 threads four blocks fit
// instead of five, 2 % of 16384x2048's time)
constexpr int norm_block_per_sm(int threads, int quads, bool bwd) {
    return bwd ? 512 / threads : threads == 512 ? 1 : (quads == 4 ? 640 : 768) / threads;
}
// The kernels' launch bound.  The forward comes out at what norm_block_per_sm counts
// on under the bound of 128 registers; held to that number it spills.
constexpr int norm_block_bound(int threads, int quads, bool bwd) {
    return !bwd && quads >= 3 ? 512 / threads : norm_block_per_sm(threads, quads, bwd);
}

// Quads of a thread up to which it holds two rows at once: beside its parameters'
// sums the backward spills with three (8192x2560 f32 54 us with two rows, 47 with
// one; 6000x5120 88 and 66).
constexpr int norm_two_rows_quads(bool bwd) { return bwd ? 2 : 4; }

// Two rows a step where two steps of them fit in shared memory beside at least
// three quarters of the blocks that the registers allow, else one.  `row_bytes`:
// what a row takes of all tensors.
NormBlockPlan norm_block_plan(int64_t rows, int64_t width, int64_t row_bytes, bool bwd) {
    NormBlockPlan p;
    p.threads = width <= 16 * 128 ? 128 : width <= 16 * 256 ? 256 : 512;
    p.quads = static_cast<int>(std::max<int64_t>(2, ceil_div(width, 4 * p.threads)));
    const int most = norm_block_per_sm(p.threads, p.quads, bwd);
    auto fits = [&](int64_t r) {  // blocks with two stages of r rows (16 bytes a tensor beside them)
        return static_cast<int>(kSmemSM / (2 * (r * row_bytes + 96) + kSmemBlock));
    };
    p.rows = p.quads <= norm_two_rows_quads(bwd) && 4 * std::min(most, fits(2)) >= 3 * most ? 2 : 1;
    p.per_sm = std::min(most, std::max(1, fits(p.rows)));
    p.blocks = std::min(ceil_div(rows, p.rows), kSMs * p.per_sm);
    if (bwd)
        p.blocks *= norm_rounds(rows, width, p.blocks);
    return p;
}

// As many stages as fit, 2 to kNormMaxStages; returns the shared memory.
int norm_stages(s6::NormStream &s, const NormBlockPlan &p) {
    const int fit = (kSmemSM / p.per_sm - kSmemBlock) / s.stage();
    s.stages = std::max(2, std::min(fit, s6::kNormMaxStages));
    return s.stages * s.stage();
}

// Runs of rows of the wide backward's second kernel: enough blocks to fill the
// SMs at its 128-thread blocks, whatever the vector width, times the rounds (up to the
// grid's 65,535, which 60 million rows have).
int64_t norm_wide_runs(int64_t rows, int64_t width) {
    const int64_t tiles = ceil_div(width, s6::kNormColThreads * 4);
    const int64_t runs = std::min<int64_t>(rows, std::max<int64_t>(1, kSMs * 8 / tiles));
    return std::min<int64_t>(runs * norm_rounds(rows, width, runs), 65535);
}

template <typename X, typename Y, int V, int NQ, int G>
void norm_launch(const s6::NormFwdArgs &a, unsigned grid, cudaStream_t st) {
    s6::s6_layernorm_fwd_kernel<X, Y, V, NQ, G><<<grid, 32 * s6::kNormBlockWarps, 0, st>>>(a);
}

template <typename X, typename Y, int V, int NQ, int G>
void norm_launch(const s6::NormBwdArgs &a, unsigned grid, cudaStream_t st) {
    s6::s6_layernorm_bwd_kernel<X, Y, V, NQ, G><<<grid, 32 * s6::kNormBlockWarps, 0, st>>>(a);
}

// The instantiation that holds p.elems elements a lane on p.lanes lanes.
template <typename X, typename Y, int V, typename Args>
int norm_warp_rows(const Args &a, const NormWarpPlan &p, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(p.blocks);
    if (p.lanes == 2)
        norm_launch<X, Y, V, 1, 2>(a, grid, st);
    else if (p.lanes == 4)
        norm_launch<X, Y, V, 1, 4>(a, grid, st);
    else if (p.lanes == 8)
        norm_launch<X, Y, V, 1, 8>(a, grid, st);
    else if (p.lanes == 16)
        norm_launch<X, Y, V, 1, 16>(a, grid, st);
    else if (p.elems <= 4)
        norm_launch<X, Y, V, 1, 32>(a, grid, st);
    else if (p.elems <= 8)
        norm_launch<X, Y, V, 2, 32>(a, grid, st);
    else if (p.elems <= 12)
        norm_launch<X, Y, V, 3, 32>(a, grid, st);
    else
        norm_launch<X, Y, V, 4, 32>(a, grid, st);
    return launch_status(cudaGetLastError());
}

template <typename X, typename Y, int V, int NQ, int R, int T>
auto norm_block_kernel(const s6::NormFwdBlockArgs &) {
    return s6::s6_layernorm_fwd_block_kernel<X, Y, V, NQ, R, T, norm_block_bound(T, NQ, false)>;
}
template <typename X, typename Y, int V, int NQ, int R, int T>
auto norm_block_kernel(const s6::NormBwdBlockArgs &) {
    return s6::s6_layernorm_bwd_block_kernel<X, Y, V, NQ, R, T, norm_block_bound(T, NQ, true)>;
}

// The default limit of 48 KB counts a block's static shared memory too.  Above it a
// kernel's own limit is raised, always to the same value: the limit belongs to the
// kernel on the device, and another thread's call may be between here and its launch.
template <typename X, typename Y, int V, int NQ, int R, int T, typename Args>
int norm_block_launch(const Args &a, const NormBlockPlan &p, int smem, cudaStream_t st) {
    auto kern = norm_block_kernel<X, Y, V, NQ, R, T>(a);
    if (smem > 48 * 1024 - kSmemBlock && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                              kSmemSM - kSmemBlock) != cudaSuccess)
        return S6_ERR_CUDA;
    kern<<<static_cast<unsigned>(p.blocks), T, static_cast<size_t>(smem), st>>>(a);
    return launch_status(cudaGetLastError());
}

template <typename X, typename Y, int V, int NQ, int T, typename Args>
int norm_block_r(const Args &a, const NormBlockPlan &p, int smem, cudaStream_t st) {
    if constexpr (NQ <= norm_two_rows_quads(std::is_same<Args, s6::NormBwdBlockArgs>::value))
        if (p.rows == 2)
            return norm_block_launch<X, Y, V, NQ, 2, T>(a, p, smem, st);
    return norm_block_launch<X, Y, V, NQ, 1, T>(a, p, smem, st);
}

// 2 to 4 quads of 128 threads, 3 or 4 of 256 or 512 (norm_block_plan).
template <typename X, typename Y, int V, typename Args>
int norm_block_rows(const Args &a, const NormBlockPlan &p, int smem, cudaStream_t st) {
    if (p.threads == 128)
        return p.quads == 2   ? norm_block_r<X, Y, V, 2, 128>(a, p, smem, st)
               : p.quads == 3 ? norm_block_r<X, Y, V, 3, 128>(a, p, smem, st)
                              : norm_block_r<X, Y, V, 4, 128>(a, p, smem, st);
    if (p.threads == 256)
        return p.quads == 3 ? norm_block_r<X, Y, V, 3, 256>(a, p, smem, st)
                            : norm_block_r<X, Y, V, 4, 256>(a, p, smem, st);
    return p.quads == 3 ? norm_block_r<X, Y, V, 3, 512>(a, p, smem, st)
                        : norm_block_r<X, Y, V, 4, 512>(a, p, smem, st);
}

template <typename X, typename Y, int V>
int norm_fwd_v(const s6::NormFwdArgs &a, cudaStream_t st) {
    if (a.width > s6::kNormMaxWidth) {
        const int64_t blocks = std::min<int64_t>(a.rows, kSMs * s6::kNormWideBlocks);
        s6::s6_layernorm_fwd_wide_kernel<X, Y, V>
            <<<static_cast<unsigned>(blocks), s6::kNormWideThreads, 0, st>>>(a);
        return launch_status(cudaGetLastError());
    }
    if (a.width <= s6::kNormWarpWidth)
        return norm_warp_rows<X, Y, V>(
            a, norm_warp_plan(a.rows, a.width, false, a.r ? a.width * int64_t(sizeof(X) + sizeof(Y)) : 0), st);
    const int64_t sx = sizeof(X), sr = a.r ? sizeof(Y) : 0;
    const NormBlockPlan p = norm_block_plan(a.rows, a.width, a.width * (sx + sr), false);
    const int64_t n = p.rows * static_cast<int64_t>(a.width);
    s6::NormFwdBlockArgs r;
    r.n = a;
    r.s.x_bytes = s6::row_buffer_bytes(n * sx);
    r.s.y_bytes = a.r ? s6::row_buffer_bytes(n * sr) : 0;
    r.s.e_bytes = 0;
    const int smem = norm_stages(r.s, p);
    return norm_block_rows<X, Y, V>(r, p, smem, st);
}

template <typename X, typename Y, int V>
int norm_bwd_v(const s6::NormBwdArgs &in, void *workspace, float *dw, float *db, cudaStream_t st) {
    s6::NormBwdArgs a = in;
    float *part = static_cast<float *>(workspace);
    const bool params = dw || db;
    int64_t parts = 0;
    if (a.width > s6::kNormMaxWidth) {
        float2 *sums = static_cast<float2 *>(workspace);
        part = static_cast<float *>(workspace) + 2 * a.rows;
        parts = norm_wide_runs(a.rows, a.width);
        a.part = params ? part : nullptr;
        const int64_t blocks = std::min<int64_t>(a.rows, kSMs * s6::kNormWideBlocks);
        s6::s6_layernorm_bwd_wide_sums_kernel<X, Y, V>
            <<<static_cast<unsigned>(blocks), s6::kNormWideThreads, 0, st>>>(a, sums);
        const dim3 grid(static_cast<unsigned>(ceil_div(a.width, s6::kNormColThreads * V)),
                        static_cast<unsigned>(parts));
        s6::s6_layernorm_bwd_wide_cols_kernel<X, Y, V><<<grid, s6::kNormColThreads, 0, st>>>(a, sums);
    } else {
        a.part = params ? part : nullptr;
        int rc;
        if (a.width <= s6::kNormWarpWidth) {
            const NormWarpPlan p = norm_warp_plan(a.rows, a.width, true);
            parts = p.blocks;
            rc = norm_warp_rows<X, Y, V>(a, p, st);
        } else {
            const int64_t sx = sizeof(X), sy = sizeof(Y), se = a.ds ? sizeof(float) : 0;
            const NormBlockPlan p = norm_block_plan(a.rows, a.width, a.width * (sx + sy + se), true);
            const int64_t n = p.rows * static_cast<int64_t>(a.width);
            s6::NormBwdBlockArgs t;
            t.n = a;
            t.s.x_bytes = s6::row_buffer_bytes(n * sx);
            t.s.y_bytes = s6::row_buffer_bytes(n * sy);
            t.s.e_bytes = a.ds ? s6::row_buffer_bytes(n * se) : 0;
            parts = p.blocks;
            rc = norm_block_rows<X, Y, V>(t, p, norm_stages(t.s, p), st);
        }
        if (rc != S6_OK)
            return rc;
    }
    const int rc = launch_status(cudaGetLastError());
    if (rc != S6_OK || !params)
        return rc;
    return sum_parts(part, parts, a.width, 2, 1, dw, db, st);
}

// Vectors of 4 elements where every row starts on one; single elements otherwise.
bool vec4(int64_t width, const void *const *io, const size_t *size, int n) {
    if (width % 4 != 0)
        return false;
    for (int i = 0; i < n; ++i)
        if (io[i] && !aligned_to(io[i], 4 * size[i]))
            return false;
    return true;
}

// -------------------------------------------------------------------- conv
struct ConvBwdPlan {
    int64_t tiles, blocks_y, run, runs;
};

constexpr int64_t kConvBwdBlocks = kSMs * s6::kConvBwdPerSM;
constexpr int64_t kConvBwdMinRun = 8;  // tokens; shorter runs read more rows twice than they save

int64_t conv_bwd_blocks_y(int64_t d, int64_t channels) {
    return std::max<int64_t>(1, kConvBwdBlocks / ceil_div(d, channels));
}

// Runs of a sequence: as many as it has warps, rounded down; where the sequences
// outnumber the warps, about four for each warp; and a multiple of that where they
// would be longer than kConvBwdMaxRun.  They are even where the sequences divide the
// warps (16x8192x1536: two runs for each).  Else warps are left over, or take a run
// fewer: 16 sequences of 5120 channels have 28 warps a tile of channels, of which 16
// work (16x100x5120 f32 29 us = 52 % of the copy rate), and above 1024 tokens 32 runs
// in two rounds (16x2048x5120 412 us = 75 %).
ConvBwdPlan conv_bwd_plan(int64_t Bt, int64_t L, int64_t d, int V) {
    ConvBwdPlan p;
    p.tiles = ceil_div(d, 32 * V);
    p.blocks_y = conv_bwd_blocks_y(d, 32 * V);
    const int64_t warps = p.blocks_y * s6::kConvBwdWarps;
    int64_t want = Bt < warps ? warps / Bt : ceil_div(4 * warps, Bt);  // runs of a sequence
    want *= ceil_div(ceil_div(L, want), static_cast<int64_t>(s6::kConvBwdMaxRun));
    p.run = std::max(ceil_div(L, want), std::min(L, kConvBwdMinRun));
    p.runs = ceil_div(L, p.run);
    p.blocks_y = std::min(p.blocks_y, ceil_div(Bt * p.runs, s6::kConvBwdWarps));
    return p;
}

template <typename X, typename G, int V, int K>
int conv_bwd_k(const s6::ConvBwdArgs &a, const ConvBwdPlan &p, float *dconv_w, float *dconv_b, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.blocks_y));
    s6::s6_conv_silu_bwd_kernel<X, G, V, K><<<grid, 32 * s6::kConvBwdWarps, 0, st>>>(a);
    const int rc = launch_status(cudaGetLastError());
    if (rc != S6_OK)
        return rc;
    return sum_parts(a.part, p.blocks_y, a.d, K + 1, K, dconv_w, dconv_b, st);
}

template <typename X, typename G, int V>
int conv_bwd_v(const s6::ConvBwdArgs &in, int64_t K, float *dconv_w, float *dconv_b, cudaStream_t st) {
    s6::ConvBwdArgs a = in;
    const ConvBwdPlan p = conv_bwd_plan(a.Bt, a.L, a.d, V);
    a.run = static_cast<int>(p.run);
    a.runs = static_cast<int>(p.runs);
    if (K == 2)
        return conv_bwd_k<X, G, V, 2>(a, p, dconv_w, dconv_b, st);
    if (K == 3)
        return conv_bwd_k<X, G, V, 3>(a, p, dconv_w, dconv_b, st);
    return conv_bwd_k<X, G, V, 4>(a, p, dconv_w, dconv_b, st);
}

template <typename X, typename G>
int conv_bwd_io(const s6::ConvBwdArgs &a, int64_t K, float *dconv_w, float *dconv_b, cudaStream_t st) {
    if (a.d % 2 == 0 && aligned_to(a.x, 2 * sizeof(X)) && aligned_to(a.dout, 2 * sizeof(G)) &&
        aligned_to(a.dx, 2 * sizeof(float)))
        return conv_bwd_v<X, G, 2>(a, K, dconv_w, dconv_b, st);
    return conv_bwd_v<X, G, 1>(a, K, dconv_w, dconv_b, st);
}

int check_conv_bwd_dims(const s6_dims *dims) {
    if (!dims || dims->batch < 0 || dims->seqlen < 0 || dims->d_inner < 1)
        return S6_ERR_INVALID_ARG;
    if ((dims->io_dtype != S6_F32 && dims->io_dtype != S6_BF16) || dims->conv_width < 2 || dims->conv_width > 4 ||
        dims->d_inner > (1 << 30) || dims->batch > (1 << 30) || dims->seqlen > (1 << 30))
        return S6_ERR_UNSUPPORTED;
    return S6_OK;
}

// --------------------------------------------------------------- gradients
constexpr int64_t kGradMaxNumel = int64_t(1) << 37;  // 2^26 of the smallest chunks

int64_t grad_words(int64_t numel, int32_t dtype) {  // float32 elements, or pairs of bfloat16 ones
    return dtype == S6_BF16 ? ceil_div(numel, 2) : numel;
}

// The size of a chunk (float32 elements; twice as many bfloat16 ones): such that
// every resident block gets as many as every other, one if they are short, with
// a chunk set aside for each tensor, whose last one may be a short one.
int grad_chunk(int64_t count, const int64_t *numel, const int32_t *dtypes) {
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i)
        total += grad_words(numel[i], dtypes[i]);
    const int64_t blocks = s6::kGradMaxBlocks, rounds = std::max<int64_t>(1, ceil_div(total, blocks * s6::kGradChunkMost));
    const int64_t chunks = std::max(blocks * rounds - count, blocks * rounds / 2);
    const int64_t chunk = ceil_div(ceil_div(total, chunks), s6::kGradChunkStep) * s6::kGradChunkStep;
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>(chunk, s6::kGradChunkStep), s6::kGradChunkMost));
}

// Checks a list; `write`: the tensors are written, so no two may share memory.
int check_grads(int64_t count, const void *const *grads, const int64_t *numel, const int32_t *dtypes, bool write) {
    if (count < 0 || (count > 0 && (!grads || !numel || !dtypes)))
        return S6_ERR_INVALID_ARG;
    if (count > (int64_t(1) << 24))
        return S6_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != S6_F32 && dtypes[i] != S6_BF16)
            return S6_ERR_UNSUPPORTED;
        if (numel[i] < 0 || (numel[i] > 0 && !grads[i]))
            return S6_ERR_INVALID_ARG;
        if (numel[i] > kGradMaxNumel)
            return S6_ERR_UNSUPPORTED;
        if (!aligned_to(grads[i], io_size(dtypes[i])))
            return S6_ERR_ALIGNMENT;
    }
    if (!write || count < 2)
        return S6_OK;
    struct Range {
        uintptr_t at, end;
    };
    Range *r = static_cast<Range *>(std::malloc(sizeof(Range) * static_cast<size_t>(count)));
    if (!r)
        return S6_ERR_HOST_MEMORY;
    size_t n = 0;
    for (int64_t i = 0; i < count; ++i)
        if (numel[i] > 0) {
            r[n].at = reinterpret_cast<uintptr_t>(grads[i]);
            r[n].end = r[n].at + static_cast<size_t>(numel[i]) * io_size(dtypes[i]);
            ++n;
        }
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.at < b.at; });
    bool apart = true;
    for (size_t i = 1; i < n; ++i)
        apart = apart && r[i].at >= r[i - 1].end;
    std::free(r);
    return apart ? S6_OK : S6_ERR_INVALID_ARG;
}

// Walks a list in tables of at most M tensors (and few enough chunks to count in
// an int) and calls fn(table) for each.
template <int M, typename Fn>
int for_tables(int64_t count, const void *const *grads, const int64_t *numel, const int32_t *dtypes, Fn fn) {
    s6::GradTable<M> t;
    t.tensors = t.chunks = 0;
    t.chunk = grad_chunk(count, numel, dtypes);
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] == 0)
            continue;
        const int chunks = static_cast<int>(ceil_div(grad_words(numel[i], dtypes[i]), t.chunk));  // at most 2^26 (check_grads)
        if (t.tensors == M || t.chunks + chunks > (1 << 30)) {
            const int rc = fn(t);
            if (rc != S6_OK)
                return rc;
            t.tensors = t.chunks = 0;
        }
        t.chunks += chunks;
        t.ptr[t.tensors] = reinterpret_cast<void *>(reinterpret_cast<uintptr_t>(grads[i]) |
                                                    (dtypes[i] == S6_BF16 ? 1u : 0u));
        t.n[t.tensors] = numel[i];
        t.end[t.tensors] = t.chunks;
        ++t.tensors;
    }
    return t.tensors ? fn(t) : S6_OK;
}

unsigned grad_grid(int chunks) { return static_cast<unsigned>(std::min(chunks, s6::kGradMaxBlocks)); }

template <int M>
int grads_run(int64_t count, const void *const *grads, const int64_t *numel, const int32_t *dtypes, bool squares,
              bool scale, s6::GradScaleArgs a, double *part, cudaStream_t st) {
    int rc = S6_OK;
    if (squares) {
        int parts = 0;
        rc = for_tables<M>(count, grads, numel, dtypes, [&](const s6::GradTable<M> &t) {
            const unsigned grid = grad_grid(t.chunks);
            s6::s6_grad_square_kernel<M><<<grid, s6::kGradThreads, 0, st>>>(t, part + parts);
            parts += static_cast<int>(grid);
            return launch_status(cudaGetLastError());
        });
        if (rc != S6_OK)
            return rc;
        a.part = part;
        a.parts = parts;
    }
    bool launched = false;
    if (scale)
        rc = for_tables<M>(count, grads, numel, dtypes, [&](const s6::GradTable<M> &t) {
            const cudaError_t e = launch_after(s6::s6_grad_scale_kernel<M>, dim3(grad_grid(t.chunks)),
                                               s6::kGradThreads, st, t, a);
            launched = true;
            a.norm_out = nullptr;  // the first launch writes it
            return launch_status(e);
        });
    if (rc == S6_OK && !launched && a.norm_out) {
        s6::GradTable<s6::kGradFew> none;
        none.tensors = none.chunks = 0;
        rc = launch_status(launch_after(s6::s6_grad_scale_kernel<s6::kGradFew>, dim3(1), s6::kGradThreads, st, none, a));
    }
    return rc;
}

int grads_common(int64_t count, const void *const *grads, const int64_t *numel, const int32_t *dtypes, bool squares,
                 bool scale, const float *norm_in, float *norm_out, float max_norm, float eps, void *workspace,
                 int64_t workspace_bytes, s6_stream_t stream) {
    int rc = check_grads(count, grads, numel, dtypes, scale);
    if (rc != S6_OK)
        return rc;
    if (squares ? !norm_out : !norm_in)
        return S6_ERR_INVALID_ARG;
    if (scale && (!std::isfinite(max_norm) || max_norm < 0.0f || !std::isfinite(eps) || eps < 0.0f))
        return S6_ERR_INVALID_ARG;
    if (!aligned_to(norm_in, 4) || !aligned_to(norm_out, 4))
        return S6_ERR_ALIGNMENT;
    // a norm inside a gradient would be scaled with it while other blocks read it
    const uintptr_t norm = reinterpret_cast<uintptr_t>(squares ? norm_out : norm_in);
    for (int64_t i = 0; scale && i < count; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(grads[i]);
        if (norm < at + static_cast<size_t>(numel[i]) * io_size(dtypes[i]) && at < norm + sizeof(float) && numel[i] > 0)
            return S6_ERR_INVALID_ARG;
    }
    if (squares) {
        rc = check_workspace(workspace, workspace_bytes, s6_grad_workspace(count, numel));
        if (rc != S6_OK)
            return rc;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (use_stream_device(st) != S6_OK)
        return S6_ERR_CUDA;
    s6::GradScaleArgs a;
    std::memset(&a, 0, sizeof(a));
    a.norm_in = norm_in;
    a.norm_out = norm_out;
    a.max_norm = max_norm;
    a.eps = eps;
    double *part = static_cast<double *>(workspace);
    return count <= s6::kGradFew
               ? grads_run<s6::kGradFew>(count, grads, numel, dtypes, squares, scale, a, part, st)
               : grads_run<s6::kGradTensors>(count, grads, numel, dtypes, squares, scale, a, part, st);
}

}  // namespace

// The error word of this translation unit's kernels (s6_device_status reads it
// beside that of s6_abi.cu).
cudaError_t s6_train_error_word(void **word) { return cudaGetSymbolAddress(word, s6::g_s6_device_error); }

extern "C" {

int s6_layernorm_fwd(const s6_norm_dims *dims, const void *x, const void *r, const float *w, const float *b, void *s,
                     void *y, float *mean, float *rstd, s6_stream_t stream) {
    DeviceRestore restore_device;
    const int rc = check_norm_dims(dims);
    if (rc != S6_OK || dims->rows == 0)
        return rc;
    if (!x || !y || (!r && s))
        return S6_ERR_INVALID_ARG;
    const size_t sx = io_size(dims->x_dtype), sy = io_size(dims->y_dtype);
    if (!aligned_to(x, sx) || !aligned_to(s, sx) || !aligned_to(r, sy) || !aligned_to(y, sy) || !aligned_to(w, 4) ||
        !aligned_to(b, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return S6_ERR_ALIGNMENT;
    const int64_t rows = dims->rows, W = dims->width, xb = W * static_cast<int64_t>(sx), yb = W * static_cast<int64_t>(sy);
    const Mem mem[] = {{s, rows, xb, kWritten}, {y, rows, yb, kWritten}, {mean, rows, 4, kWritten},
                       {rstd, rows, 4, kWritten}, {x, rows, xb, kEach}, {r, rows, yb, kEach}, {w, 1, 4 * W, kRead},
                       {b, 1, 4 * W, kRead}};
    if (check_apart(mem) != S6_OK)
        return S6_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (use_stream_device(st) != S6_OK)
        return S6_ERR_CUDA;
    s6::NormFwdArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = dims->rows;
    a.width = static_cast<int>(dims->width);
    a.eps = dims->eps;
    a.inv_w = static_cast<float>(1.0 / static_cast<double>(dims->width));
    a.x = x;
    a.r = r;
    a.w = w;
    a.b = b;
    a.s = s;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    const void *io[] = {x, s, r, y};
    const size_t size[] = {sx, sx, sy, sy};
    const bool v4 = vec4(dims->width, io, size, 4);
    if (dims->x_dtype == S6_BF16)
        return v4 ? norm_fwd_v<bf16, bf16, 4>(a, st) : norm_fwd_v<bf16, bf16, 1>(a, st);
    if (dims->y_dtype == S6_BF16)
        return v4 ? norm_fwd_v<float, bf16, 4>(a, st) : norm_fwd_v<float, bf16, 1>(a, st);
    return v4 ? norm_fwd_v<float, float, 4>(a, st) : norm_fwd_v<float, float, 1>(a, st);
}

int64_t s6_layernorm_bwd_workspace(const s6_norm_dims *dims) {
    const int rc = check_norm_dims(dims);
    if (rc != S6_OK || dims->rows == 0)
        return rc;
    const int64_t row = 2 * dims->width * static_cast<int64_t>(sizeof(float));
    if (dims->width > s6::kNormMaxWidth)
        return dims->rows * static_cast<int64_t>(sizeof(float2)) + norm_wide_runs(dims->rows, dims->width) * row;
    if (dims->width <= s6::kNormWarpWidth)
        return norm_warp_plan(dims->rows, dims->width, true).blocks * row;
    // with and without ds
    const int64_t io = dims->width * static_cast<int64_t>(io_size(dims->x_dtype) + io_size(dims->y_dtype));
    return row * std::max(norm_block_plan(dims->rows, dims->width, io, true).blocks,
                          norm_block_plan(dims->rows, dims->width, io + 4 * dims->width, true).blocks);
}

int s6_layernorm_bwd(const s6_norm_dims *dims, const void *x, const float *mean, const float *rstd, const float *w,
                     const void *dy, const float *ds, float *dx, float *dw, float *db, void *workspace,
                     int64_t workspace_bytes, s6_stream_t stream) {
    DeviceRestore restore_device;
    int rc = check_norm_dims(dims);
    if (rc != S6_OK)
        return rc;
    const size_t sx = io_size(dims->x_dtype), sy = io_size(dims->y_dtype);
    if (dims->rows > 0 && (!x || !mean || !rstd || !dy || !dx))
        return S6_ERR_INVALID_ARG;
    if (!aligned_to(x, sx) || !aligned_to(dy, sy) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(w, 4) || !aligned_to(ds, 4) || !aligned_to(dx, 4) || !aligned_to(dw, 4) || !aligned_to(db, 4))
        return S6_ERR_ALIGNMENT;
    const int64_t rows = dims->rows, W = dims->width, xb = W * static_cast<int64_t>(sx), yb = W * static_cast<int64_t>(sy);
    const int64_t need = s6_layernorm_bwd_workspace(dims);
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != S6_OK)
        return rc;
    const Mem mem[] = {{dx, rows, 4 * W, kWritten}, {dw, 1, 4 * W, kWritten}, {db, 1, 4 * W, kWritten},
                       {workspace, 1, need, kWritten}, {x, rows, xb, kEach}, {dy, rows, yb, kEach},
                       {ds, rows, 4 * W, kEach}, {mean, rows, 4, kRead}, {rstd, rows, 4, kRead}, {w, 1, 4 * W, kRead}};
    rc = check_apart(mem);
    if (rc != S6_OK)
        return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (use_stream_device(st) != S6_OK)
        return S6_ERR_CUDA;
    if (dims->rows == 0) {  // sums over no rows
        const size_t bytes = sizeof(float) * static_cast<size_t>(dims->width);
        if ((dw && cudaMemsetAsync(dw, 0, bytes, st) != cudaSuccess) ||
            (db && cudaMemsetAsync(db, 0, bytes, st) != cudaSuccess))
            return S6_ERR_CUDA;
        return S6_OK;
    }
    s6::NormBwdArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = dims->rows;
    a.width = static_cast<int>(dims->width);
    a.inv_w = static_cast<float>(1.0 / static_cast<double>(dims->width));
    a.x = x;
    a.dy = dy;
    a.mean = mean;
    a.rstd = rstd;
    a.w = w;
    a.ds = ds;
    a.dx = dx;
    const void *io[] = {x, dy, ds, dx};
    const size_t size[] = {sx, sy, 4, 4};
    const bool v4 = vec4(dims->width, io, size, 4);
    if (dims->x_dtype == S6_BF16)
        return v4 ? norm_bwd_v<bf16, bf16, 4>(a, workspace, dw, db, st)
                  : norm_bwd_v<bf16, bf16, 1>(a, workspace, dw, db, st);
    if (dims->y_dtype == S6_BF16)
        return v4 ? norm_bwd_v<float, bf16, 4>(a, workspace, dw, db, st)
                  : norm_bwd_v<float, bf16, 1>(a, workspace, dw, db, st);
    return v4 ? norm_bwd_v<float, float, 4>(a, workspace, dw, db, st)
              : norm_bwd_v<float, float, 1>(a, workspace, dw, db, st);
}

int64_t causal_conv1d_silu_bwd_workspace(const s6_dims *dims) {
    const int rc = check_conv_bwd_dims(dims);
    if (rc != S6_OK || dims->batch == 0 || dims->seqlen == 0)
        return rc;
    // the wider channel tile has the more blocks that share it
    return conv_bwd_blocks_y(dims->d_inner, 64) * (dims->conv_width + 1) * dims->d_inner *
           static_cast<int64_t>(sizeof(float));
}

int causal_conv1d_silu_bwd(const s6_dims *dims, const void *x, const float *conv_w, const float *conv_b,
                           const void *dout, int dout_dtype, float *dx, float *dconv_w, float *dconv_b,
                           void *workspace, int64_t workspace_bytes, s6_stream_t stream) {
    DeviceRestore restore_device;
    int rc = check_conv_bwd_dims(dims);
    if (rc != S6_OK)
        return rc;
    if (dout_dtype != S6_F32 && dout_dtype != dims->io_dtype)
        return S6_ERR_UNSUPPORTED;
    const int64_t Bt = dims->batch, L = dims->seqlen, d = dims->d_inner, K = dims->conv_width;
    const bool empty = Bt == 0 || L == 0;
    if (!conv_w || !dconv_w || (!empty && (!x || !dout || !dx)))
        return S6_ERR_INVALID_ARG;
    if (!aligned_to(x, io_size(dims->io_dtype)) || !aligned_to(dout, io_size(dout_dtype)) || !aligned_to(dx, 4) ||
        !aligned_to(conv_w, 4) || !aligned_to(conv_b, 4) || !aligned_to(dconv_w, 4) || !aligned_to(dconv_b, 4))
        return S6_ERR_ALIGNMENT;
    const int64_t need = causal_conv1d_silu_bwd_workspace(dims), tokens = Bt * L;
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != S6_OK)
        return rc;
    // x and dout are read around a token, too: dx may be neither
    const int64_t xb = d * static_cast<int64_t>(io_size(dims->io_dtype)), gb = d * static_cast<int64_t>(io_size(dout_dtype));
    const Mem mem[] = {{dx, tokens, 4 * d, kWritten}, {dconv_w, K, 4 * d, kWritten}, {dconv_b, 1, 4 * d, kWritten},
                       {workspace, 1, need, kWritten}, {x, tokens, xb, kRead}, {dout, tokens, gb, kRead},
                       {conv_w, K, 4 * d, kRead}, {conv_b, 1, 4 * d, kRead}};
    rc = check_apart(mem);
    if (rc != S6_OK)
        return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (use_stream_device(st) != S6_OK)
        return S6_ERR_CUDA;
    if (empty) {  // sums over no tokens
        if (cudaMemsetAsync(dconv_w, 0, sizeof(float) * static_cast<size_t>(d * K), st) != cudaSuccess ||
            (dconv_b && cudaMemsetAsync(dconv_b, 0, sizeof(float) * static_cast<size_t>(d), st) != cudaSuccess))
            return S6_ERR_CUDA;
        return S6_OK;
    }
    s6::ConvBwdArgs a;
    std::memset(&a, 0, sizeof(a));
    a.Bt = static_cast<int>(Bt);
    a.L = static_cast<int>(L);
    a.d = static_cast<int>(d);
    a.x = x;
    a.dout = dout;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.dx = dx;
    a.part = static_cast<float *>(workspace);
    if (dims->io_dtype == S6_F32)
        return conv_bwd_io<float, float>(a, K, dconv_w, dconv_b, st);
    return dout_dtype == S6_F32 ? conv_bwd_io<bf16, float>(a, K, dconv_w, dconv_b, st)
                                : conv_bwd_io<bf16, bf16>(a, K, dconv_w, dconv_b, st);
}

int64_t s6_grad_workspace(int64_t count, const int64_t *numel) {
    if (count < 0 || (count > 0 && !numel))
        return S6_ERR_INVALID_ARG;
    // one float64 for each block of each launch: a launch ends with a full table, or
    // with more than 2^29 chunks
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] < 0)
            return S6_ERR_INVALID_ARG;
        if (numel[i] > kGradMaxNumel)
            return S6_ERR_UNSUPPORTED;
        chunks += ceil_div(numel[i], s6::kGradChunkStep);
    }
    const int64_t launches = count / (count <= s6::kGradFew ? s6::kGradFew : s6::kGradTensors) + 1 + (chunks >> 29);
    return launches * s6::kGradMaxBlocks * static_cast<int64_t>(sizeof(double));
}

int s6_grad_norm(int64_t count, const void *const *grads, const int64_t *numel, const int32_t *dtypes, float *norm,
                 void *workspace, int64_t workspace_bytes, s6_stream_t stream) {
    DeviceRestore restore_device;
    return grads_common(count, grads, numel, dtypes, true, false, nullptr, norm, 0.0f, 0.0f, workspace,
                        workspace_bytes, stream);
}

int s6_grad_clip(int64_t count, void *const *grads, const int64_t *numel, const int32_t *dtypes, const float *norm,
                 float max_norm, float eps, s6_stream_t stream) {
    DeviceRestore restore_device;
    return grads_common(count, grads, numel, dtypes, false, true, norm, nullptr, max_norm, eps, nullptr, 0, stream);
}

int s6_clip_grad_norm(int64_t count, void *const *grads, const int64_t *numel, const int32_t *dtypes, float max_norm,
                      float eps, float *norm, void *workspace, int64_t workspace_bytes, s6_stream_t stream) {
    DeviceRestore restore_device;
    return grads_common(count, grads, numel, dtypes, true, true, nullptr, norm, max_norm, eps, workspace,
                        workspace_bytes, stream);
}

}  // extern "C"
