"""GPU tests of the training-step operators where they can go wrong at the edges of
their range: calls from several threads, every size of shared memory, rows far
from zero, tall inputs, long runs of tokens.  Bounds are derived from the float32
roundings (u = 2^-24 each), against float64 formulas."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

import train_reference as R
from s6_testutil import to_dev

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _in_a_new_process(code):
    """Runs code in a process of its own, whose kernels no other call has prepared."""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-2000:]


# ------------------------------------------------- shared memory of a launch
def test_layernorm_widths_around_the_default_shared_memory_limit():
    """A row's steps take every size of shared memory, those just below 48 KB too: as the
    first calls of a process, each form at widths on both sides of that size."""
    _in_a_new_process("""
import torch
import selective_state_space_19_b200 as S
bf = torch.bfloat16
for W in [*range(660, 690), *range(740, 775), *range(990, 1024), *range(2000, 2049, 4), *range(2990, 3073, 6)]:
    x = torch.randn(3, W, device="cuda")
    mean, rstd = x.mean(-1), x.var(-1, unbiased=False).add(1e-5).rsqrt()
    S.s6_layernorm_fwd(x, r=x.to(bf))
    S.s6_layernorm_fwd(x.to(bf))
    for a, dy in ((x, x), (x, x.to(bf)), (x.to(bf), x.to(bf))):
        S.s6_layernorm_bwd(dy, a, mean, rstd)
        S.s6_layernorm_bwd(dy, a, mean, rstd, ds=x)
torch.cuda.synchronize()
""")


def test_layernorm_from_two_threads_with_different_sizes():
    """Two widths of one kernel, and the residual gradient on one side only, launched from
    two threads at once."""
    import torch
    import selective_state_space_19_b200 as S
    got, errors = {}, []

    def calls(W, ds):
        try:
            stream = torch.cuda.Stream()
            x = torch.ones(4, W, device="cuda")
            mean, rstd = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
            torch.cuda.synchronize()
            for _ in range(3000):
                y = S.s6_layernorm_fwd(x, stream=stream, want_stats=False)[0]
                dx = S.s6_layernorm_bwd(x, x, mean, rstd, ds=x if ds else None, want_params=False, stream=stream)["dx"]
            stream.synchronize()
            got[W] = (y, dx)
        except Exception as e:  # noqa: BLE001 -- reported by the test's own thread
            errors.append(repr(e))
    threads = [threading.Thread(target=calls, args=a) for a in ((2052, False), (2560, True), (3000, False))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:3]
    for W, (y, dx) in got.items():
        # of ones: y is 0, a mean off by 2 u times rstd; dx is 1 - 1 - 1, each mean off by 2 u
        assert y.abs().max().item() <= 3 * R.U * 1e-5 ** -0.5, W
        assert (dx - (0.0 if W == 2560 else -1.0)).abs().max().item() <= 8 * R.U, W


# ------------------------------------------------------- rows far from zero
def _far_bounds(s, w, b, eps):
    """Forward of rows s (float64 of what the kernel adds up) and what it may be off by: the
    first mean by e1 = U (DEPTH + 2) mean|s|; then the deviations d, |d| <= |s - mean| + e1, by
    a rounding each, and their own mean, which is taken out, by U (DEPTH + 2) of mean|d|."""
    mean = s.mean(-1, keepdims=True)
    dev = s - mean
    var = (dev ** 2).mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    e1 = R.U * (R.DEPTH + 2) * np.abs(s).mean(-1, keepdims=True)
    d = np.abs(dev) + e1
    e_mean = R.U * (R.DEPTH + 3) * d.mean(-1, keepdims=True)
    e_d = 2 * R.U * d + e_mean
    e_var = R.U * (R.DEPTH + 6) * (d ** 2).mean(-1, keepdims=True) + (2 * np.abs(dev) * e_d + e_d ** 2).mean(-1, keepdims=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 3 * R.U)
    h = dev * rstd
    y = h * w + b
    e_y = np.abs(w) * (e_d * rstd + np.abs(dev) * e_rstd + 2 * R.U * np.abs(h)) + 2 * R.U * (np.abs(y) + np.abs(h * w))
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0] + R.U * np.abs(mean[:, 0]), e_rstd[:, 0])


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("W", [5, 40, 63, 64, 100, 130, 300, 384, 500, 771, 1000, 1535, 2561, 3001, 4100, 8191, 8192,
                               9000, 20000])
def test_layernorm_of_rows_far_from_zero(W, add):
    """Constant rows, and rows whose mean is up to 1e5 times their deviations, by turns with
    rows around zero: each within its bound, and the latter with the bits they have alone."""
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(W)
    centre = np.array([0.0, 100.0, 0.1, 1e4, 1000.0, 0.0, 1000.0, 1e-3, 0.0, 77.7, 123.4, 0.0])[:, None]
    dev = np.array([1.0, 0.0, 1.0, 0.0, 1.0, 1.0, 0.01, 1.0, 1.0, 0.0, 0.0, 1.0])[:, None]
    x = (centre + dev * rng.standard_normal((12, W))).astype(np.float32)
    r = (0.01 * dev * rng.standard_normal((12, W))).astype(np.float32)
    w, b = rng.standard_normal(W).astype(np.float32), rng.standard_normal(W).astype(np.float32)
    s = (x + r) if add else x  # the float32 sum
    (y, mean, rstd), (e_y, e_mean, e_rstd) = _far_bounds(s.astype(np.float64), w, b, 1e-5)
    assert e_y[[1, 3, 4, 6]].max() < 1e-3  # the bound itself keeps the digits
    xd, rd, wd, bd = (to_dev(a) for a in (x, r, w, b))
    got, _, m, q = S.s6_layernorm_fwd(xd, wd, bd, r=rd if add else None)
    R.within(got.cpu().numpy(), y, e_y, "y")
    R.within(m.cpu().numpy(), mean, e_mean, "mean")
    R.within(q.cpu().numpy(), rstd, e_rstd, "rstd")
    near = torch.tensor([0, 2, 5, 7, 8, 11], device="cuda")
    alone = S.s6_layernorm_fwd(xd[near].contiguous(), wd, bd, r=rd[near].contiguous() if add else None)
    assert torch.equal(alone[0], got[near]) and torch.equal(alone[2], m[near]) and torch.equal(alone[3], q[near])


@pytest.mark.parametrize("W", [40, 300, 1001, 2560, 9000])
def test_layernorm_of_bfloat16_rows_far_from_zero(W):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(W)
    x = torch.from_numpy((100.0 + np.array([[0.0], [0.5], [8.0]]) * rng.standard_normal((3, W))).astype(np.float32))
    for xt in (torch.bfloat16, torch.float32):
        s = x.bfloat16().to(xt)
        (y, mean, rstd), (e_y, e_mean, e_rstd) = _far_bounds(s.double().numpy(), 1.0, 0.0, 1e-5)
        got, _, m, q = S.s6_layernorm_fwd(s.cuda(), y_dtype=torch.bfloat16)
        R.within(got.double().cpu().numpy(), y, e_y + R.HALF["bf16"] * (np.abs(y) + e_y), "y")
        R.within(m.cpu().numpy(), mean, e_mean, "mean")
        R.within(q.cpu().numpy(), rstd, e_rstd, "rstd")


@pytest.mark.parametrize("W", [5, 31, 33, 64, 65, 130, 383, 385, 516, 771, 1001, 2561, 4097, 8191, 9001])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_layernorm_backward_of_rows_whose_mean_over_the_deviation_overflows(W, xt, yt):
    """Columns behind a row's end take no part, however large the row's mean times its rstd
    is (6e38 here, beside deviations of zero)."""
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(W)
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    x = torch.from_numpy(rng.standard_normal((5, W)).astype(np.float32)).to(types[xt])
    x[1], x[4] = 2.0 ** 120, -2.0 ** 120
    dy = torch.from_numpy(rng.standard_normal((5, W)).astype(np.float32)).to(types[yt])
    w = rng.standard_normal(W).astype(np.float32)
    mean, rstd = np.zeros(5, np.float32), np.ones(5, np.float32)
    mean[[1, 4]], rstd[[1, 4]] = [2.0 ** 120, -2.0 ** 120], 1e-5 ** -0.5
    ref, tol = R.ln_bwd(dy.double().numpy(), x.double().numpy(), mean.astype(np.float64), rstd.astype(np.float64), w)
    got = S.s6_layernorm_bwd(dy.cuda(), x.cuda(), to_dev(mean), to_dev(rstd), to_dev(w))
    for k in ("dx", "dw", "db"):
        R.within(got[k].cpu().numpy(), ref[k], tol[k], k)


# ----------------------------------------------------------------- gradients
def test_a_norm_beside_the_gradients_it_scales():
    """In one buffer, right before and behind a gradient; inside one it is refused."""
    import torch
    import selective_state_space_19_b200 as S
    buf = torch.full((1002,), 2.0, device="cuda")
    for at in (0, 1001):
        buf[1:1001] = 2.0
        norm = S.s6_clip_grad_norm([buf[1:1001]], 1.0, eps=0.0, norm=buf[at:at + 1])
        want = 2.0 * 1000 ** 0.5
        assert abs(norm.item() - want) <= R.NORM_REL * want
        assert (buf[1:1001] * want / 2.0 - 1.0).abs().max().item() <= 2 * R.SCALED_REL
    for at in (1, 500, 1000):
        with pytest.raises(S.S6Error):
            S.s6_clip_grad_norm([buf[1:1001]], 1.0, norm=buf[at:at + 1])
        with pytest.raises(S.S6Error):
            S.s6_grad_clip([buf[1:1001]], buf[at:at + 1], 1.0)
    assert S.s6_grad_norm([buf[1:1001]], norm=buf[5:6]) is not None  # read only: allowed


def test_a_flag_without_a_truth_value_raises_its_own_error():
    import torch
    import selective_state_space_19_b200 as S
    x, m, two = torch.randn(4, 64, device="cuda"), torch.zeros(4, device="cuda"), torch.ones(2, dtype=torch.bool)
    with pytest.raises(RuntimeError, match="ambiguous"):
        S.s6_layernorm_fwd(x, want_stats=two)
    with pytest.raises(RuntimeError, match="ambiguous"):
        S.s6_layernorm_bwd(x, x, m, m, want_params=two)
    assert S.s6_layernorm_fwd(x, want_stats=two[:1])[2] is not None


# ------------------------------------------------ many steps of a block's ring
def _off(a, dtype, by):
    """A contiguous tensor of a's values, `by` elements into its memory and with canaries
    around it, and a function that tells whether those are as they were."""
    import torch
    buf = torch.full((a.numel() + by + 40,), 7.0, dtype=dtype, device="cuda")
    t = buf[by:by + a.numel()].view(a.shape)
    t.copy_(a)
    return t, lambda: bool((buf[:by] == 7).all()) and bool((buf[by + a.numel():] == 7).all())


OFF = {"on": (8, 16, 24, 32), "off": (1, 3, 5, 7)}  # elements into the memory
RING = [(20001, 516), (9001, 1031), (6001, 2560), (4001, 4097), (3001, 8191), (9001, 384), (30001, 100), (90001, 30),
        (1500, 9001)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,W", RING)
@pytest.mark.parametrize("at", ["on", "off"])
def test_layernorm_of_many_rows_on_and_off_16_byte_boundaries(at, rows, W, xt, yt, add):
    """Blocks that take many steps (each stage of their shared memory several times), on
    tensors that begin on or off a 16-byte boundary, every row against float64."""
    import torch
    import selective_state_space_19_b200 as S
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(rows + W)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)
    x, x_whole = _off(normal(rows, W), types[xt], OFF[at][0])
    r, r_whole = _off(normal(rows, W), types[yt], OFF[at][1])
    y, y_whole = _off(torch.zeros(rows, W, device="cuda"), types[yt], OFF[at][2])
    s, s_whole = _off(torch.zeros(rows, W, device="cuda"), types[xt], OFF[at][3])
    w, b = normal(W), normal(W)
    out = S.s6_layernorm_fwd(x, w, b, r=r if add else None, s=s if add else None, y=y, y_dtype=types[yt])
    sums = (x.float() + r.float()) if add else x.float()
    half = R.HALF[yt]
    step = max(1, 8_000_000 // W)
    for at in range(0, rows, step):
        part = slice(at, at + step)
        (ry, rm, rq), (ey, em, eq) = _far_bounds_on_gpu(sums[part].double(), w.double(), b.double(), 1e-5)
        _within(y[part], ry, ey + half * (ry.abs() + ey), "y")
        _within(out[2][part], rm, em, "mean")
        _within(out[3][part], rq, eq, "rstd")
    assert not add or torch.equal(s, sums.to(types[xt]))
    assert x_whole() and r_whole() and y_whole() and s_whole()


def _far_bounds_on_gpu(s, w, b, eps):
    """_far_bounds in torch."""
    mean = s.mean(-1, keepdim=True)
    dev = s - mean
    var = dev.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    d = dev.abs() + R.U * (R.DEPTH + 2) * s.abs().mean(-1, keepdim=True)
    e_mean = R.U * (R.DEPTH + 3) * d.mean(-1, keepdim=True)
    e_d = 2 * R.U * d + e_mean
    e_var = R.U * (R.DEPTH + 6) * d.square().mean(-1, keepdim=True) + (2 * dev.abs() * e_d + e_d ** 2).mean(-1, keepdim=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 3 * R.U)
    h = dev * rstd
    y = h * w + b
    e_y = w.abs() * (e_d * rstd + dev.abs() * e_rstd + 2 * R.U * h.abs()) + 2 * R.U * (y.abs() + (h * w).abs())
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0] + R.U * mean[:, 0].abs(), e_rstd[:, 0])


def _within(got, ref, tol, what):
    share = ((got.double() - ref).abs() / (tol + 1e-37)).max().item()
    assert share <= 1.0, (what, share)  # NaN fails too


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,W", RING)
@pytest.mark.parametrize("at", ["on", "off"])
def test_layernorm_backward_of_many_rows_on_and_off_16_byte_boundaries(at, rows, W, xt, yt, add):
    import torch
    import selective_state_space_19_b200 as S
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(rows * 3 + W)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)
    x, x_whole = _off(normal(rows, W), types[xt], OFF[at][0])
    dy, dy_whole = _off(0.5 + normal(rows, W), types[yt], OFF[at][2])
    ds, ds_whole = _off(normal(rows, W), torch.float32, OFF[at][1])
    dx, dx_whole = _off(torch.zeros(rows, W, device="cuda"), torch.float32, OFF[at][0])
    w, mean, rstd = normal(W), 0.1 * normal(rows), 1.0 + 0.1 * normal(rows)
    got = S.s6_layernorm_bwd(dy, x, mean, rstd, w, ds=ds if add else None, dx=dx)
    sums = {k: torch.zeros(W, dtype=torch.float64, device="cuda") for k in ("dw", "db", "e_dw", "e_db")}
    step = max(1, 8_000_000 // W)
    for at in range(0, rows, step):
        part = slice(at, at + step)
        ref, tol, h, e_h = _bwd_bounds_on_gpu(dy[part].double(), x[part].double(), mean[part].double()[:, None],
                                              rstd[part].double()[:, None], w.double(), ds[part].double() if add else None)
        _within(dx[part], ref, tol, "dx")
        g = dy[part].double()
        sums["dw"] += (g * h).sum(0)
        sums["db"] += g.sum(0)
        sums["e_dw"] += R.U * R.DEPTH * (g * h).abs().sum(0) + (g.abs() * e_h).sum(0)
        sums["e_db"] += R.U * R.DEPTH * g.abs().sum(0)
    _within(got["dw"], sums["dw"], sums["e_dw"], "dw")
    _within(got["db"], sums["db"], sums["e_db"], "db")
    assert x_whole() and dy_whole() and ds_whole() and dx_whole()


def _bwd_bounds_on_gpu(dy, x, mean, rstd, w, ds):
    """train_reference.ln_bwd's dx in torch, and h with its bound."""
    h = (x - mean) * rstd
    g = dy * w
    c0, c1 = g.mean(-1, keepdim=True), (g * h).mean(-1, keepdim=True)
    dx = rstd * (g - c0 - h * c1)
    e_h = R.U * ((x - mean).abs() * rstd + 2 * h.abs())
    e_c0 = R.U * (R.DEPTH + 3) * g.abs().mean(-1, keepdim=True)
    e_c1 = R.U * (R.DEPTH + 3) * (g * h).abs().mean(-1, keepdim=True) + (g.abs() * e_h).mean(-1, keepdim=True)
    e_dx = rstd * (2 * R.U * g.abs() + e_c0 + h.abs() * e_c1 + c1.abs() * e_h
                   + 3 * R.U * (g.abs() + c0.abs() + (h * c1).abs())) + R.U * dx.abs()
    if ds is not None:
        dx = dx + ds
        e_dx = e_dx + R.U * dx.abs()
    return dx, e_dx, h, e_h


# ------------------------------------------------------ the conv's long runs
def _conv_against_float64(x, g, w, b, channels, depth, monkeypatch):
    """All three gradients of some channels (each is a problem of its own) against float64."""
    import selective_state_space_19_b200 as S
    monkeypatch.setattr(R, "DEPTH", depth)
    got = S.causal_conv1d_silu_bwd(x, w, g, conv_b=b)
    pick = [a.index_select(-1, channels).double().cpu().numpy() for a in (x, g)]
    ref, tol = R.conv_bwd(pick[0], w[channels].double().cpu().numpy(), b[channels].double().cpu().numpy(), pick[1])
    R.within(got["dx"].index_select(-1, channels).cpu().numpy(), ref["dx"], tol["dx"], "dx")
    for k in ("dconv_w", "dconv_b"):
        R.within(got[k][channels].cpu().numpy(), ref[k], tol[k], k)


CONV_TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


def _conv_inputs(shape, K, xt, gt):
    import torch
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(sum(shape) + K)
    x = (2.0 * torch.randn(shape, device="cuda", generator=gen)).to(types[xt])
    g = (0.3 + torch.randn(shape, device="cuda", generator=gen)).to(types[gt])
    w, b = (torch.randn(n, device="cuda", generator=gen) for n in ((shape[2], K), (shape[2],)))
    return x, g, w, b


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("xt,gt", CONV_TYPES)
@pytest.mark.parametrize("shape", [(16, 300, 1536), (16, 300, 1535), (3, 1021, 1090), (2, 333, 5119)])
def test_conv_backward_of_runs_of_many_groups(shape, xt, gt, K, monkeypatch):
    """Runs of 12 to 50 tokens and more: the groups of 8 that look at no token's place, between
    the first and the last ones, in pairs of channels and in single ones."""
    import torch
    x, g, w, b = _conv_inputs(shape, K, xt, gt)
    d = shape[2]
    channels = torch.tensor([*range(66), *range(d // 2, d // 2 + 66), *range(d - 66, d)], device="cuda")
    _conv_against_float64(x, g, w, b, channels, R.DEPTH, monkeypatch)


@pytest.mark.parametrize("K,xt,gt", [(4, "f32", "f32"), (3, "bf16", "f32"), (2, "bf16", "bf16")])
@pytest.mark.parametrize("shape", [(1, 30000, 5120), (16, 1500, 5120), (15, 2621, 2559)])
def test_conv_backward_of_runs_up_to_their_longest(shape, xt, gt, K, monkeypatch):
    """Sequences cut at 1024 tokens, warps that take several runs: sums of up to 1024 terms in
    float32 and of the runs in float64."""
    import torch
    x, g, w, b = _conv_inputs(shape, K, xt, gt)
    d = shape[2]
    channels = torch.tensor([*range(20), *range(d // 2, d // 2 + 20), *range(d - 20, d)], device="cuda")
    _conv_against_float64(x, g, w, b, channels, 1024 + R.DEPTH, monkeypatch)


# --------------------------------------------------------------- long sums
@pytest.mark.parametrize("rows,W,run", [(60_000_000, 30, 2048), (12_000_000, 100, 256), (4_700_000, 516, 256),
                                        (1_600_000, 2560, 256), (500_000, 9004, 1024)])
def test_layernorm_parameter_gradients_of_tall_inputs(rows, W, run):
    """Some thousands of rows for each thread, all with the gradient 0.1, whose float32 sum
    drifts: dw and db are within a depth of run + 64 additions of the exact rows * 0.1 (a run of
    rows, then the lanes' and warps' sums, and float64 over the blocks)."""
    import torch
    import selective_state_space_19_b200 as S
    free, _ = torch.cuda.mem_get_info()
    if free < 14 * rows * W:
        pytest.skip("needs %d GB of device memory" % (14 * rows * W >> 30))
    x = torch.zeros(rows, W, device="cuda")
    dy = torch.full((rows, W), 0.1, device="cuda")
    mean, rstd = torch.full((rows,), -1.0, device="cuda"), torch.ones(rows, device="cuda")  # h = 1
    got = S.s6_layernorm_bwd(dy, x, mean, rstd)
    want = rows * float(np.float32(0.1))
    for k in ("dw", "db"):
        assert (got[k].double() - want).abs().max().item() <= (run + 64) * R.U * want, k


@pytest.mark.parametrize("W", [1 << 20, (1 << 22) + 1, 1 << 24])
def test_layernorm_of_the_widest_rows(W):
    """Rows of up to 2^24 columns: sums of a thread's up to 8,192 vectors."""
    import torch
    import selective_state_space_19_b200 as S
    gen = torch.Generator(device="cuda").manual_seed(W)
    x = 3.0 + torch.randn(2, W, device="cuda", generator=gen)
    dy = 0.1 + 0.01 * torch.randn(2, W, device="cuda", generator=gen)
    xs, gs = x.double(), dy.double()
    mean = xs.mean(-1, keepdim=True)
    rstd = ((xs - mean).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    h = (xs - mean) * rstd
    y, _, m, q = S.s6_layernorm_fwd(x)
    depth = 4 * 64 + 128 + 32  # a run's elements; the runs; the block's 5 + 16
    # the mean is corrected by the deviations' own, so it is off by a few roundings of itself
    assert ((m.double() - mean[:, 0]).abs() / (2 * R.U * mean[:, 0].abs() + depth * R.U)).max().item() <= 1.0
    assert ((q.double() - rstd[:, 0]).abs() / rstd[:, 0]).max().item() <= depth * R.U
    assert ((y.double() - h).abs() - 2 * depth * R.U * (1.0 + h.abs())).max().item() <= 0.0
    mf, qf = mean[:, 0].float(), rstd[:, 0].float()
    got = S.s6_layernorm_bwd(dy, x, mf, qf)
    (ref, tol, _, _) = _bwd_bounds_on_gpu(gs, xs, mf.double()[:, None], qf.double()[:, None],
                                          torch.ones(W, dtype=torch.float64, device="cuda"), None)
    tol = tol * (depth + 3) / (R.DEPTH + 3)  # its means' sums are deeper
    _within(got["dx"], ref, tol, "dx")


# ------------------------------------------------------------ shared memory
@pytest.mark.parametrize("W", [40, 384, 1001, 2560, 9001])
def test_outputs_in_the_place_of_their_inputs(W):
    """y in x or r, dx in x, dy or ds: the same bits as apart; overlaps that are not element on
    element are refused."""
    import torch
    import selective_state_space_19_b200 as S
    x, r, ds = (torch.randn(700, W, device="cuda") for _ in range(3))
    y, s, mean, rstd = S.s6_layernorm_fwd(x, r=r)
    for into in (0, 1):
        a = [x.clone(), r.clone()]
        assert torch.equal(S.s6_layernorm_fwd(a[0], r=a[1], y=a[into])[0], y) and torch.equal(a[into], y)
    a = [x.clone(), r.clone()]
    y2, s2, _, _ = S.s6_layernorm_fwd(a[0], r=a[1], s=a[0], y=a[1])
    assert torch.equal(y2, y) and torch.equal(s2, s)
    dx = S.s6_layernorm_bwd(r, s, mean, rstd, ds=ds)["dx"]
    for into in range(3):
        a = [r.clone(), s.clone(), ds.clone()]
        assert torch.equal(S.s6_layernorm_bwd(a[0], a[1], mean, rstd, ds=a[2], dx=a[into])["dx"], dx)
    buf = torch.zeros(701 * W, device="cuda")
    lo, hi = buf[:700 * W].view(700, W), buf[W:].view(700, W)
    for call in (lambda: S.s6_layernorm_fwd(lo, y=hi), lambda: S.s6_layernorm_fwd(x, r=r, s=lo, y=lo),
                 lambda: S.s6_layernorm_fwd(x, r=hi, s=lo), lambda: S.s6_layernorm_fwd(x, w=buf[5:5 + W], y=lo),
                 lambda: S.s6_layernorm_bwd(x, lo, mean, rstd, dx=hi),
                 lambda: S.s6_layernorm_bwd(x, s, buf[:700], rstd, dx=lo)):
        with pytest.raises(S.S6Error):
            call()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("size,max_norm,eps", [(1e30, 1e-14, 1e-6), (1e36, 1e-9, 0.0), (1e9, 1e-30, 1e-6), (3e36, 1.0, 0.0),
                                               (1e30, 1e-10, 3e38), (1e38, 1e-3, 3.3e38), (1.0, 1e-37, 0.0), (1.0, 0.5, 0.0)])
def test_clipping_by_factors_below_float32s_range(size, max_norm, eps, t):
    """min(1, max_norm / (norm + eps)) where the factor, or norm + eps, leaves float32's range and
    the scaled gradients do not."""
    import torch
    import selective_state_space_19_b200 as S
    g = (size * torch.linspace(-1.0, 1.0, 5).double()).float().to(torch.bfloat16 if t == "bf16" else torch.float32)
    a = g.double().numpy()
    n = R.grad_norm([a])
    want = a * (float(np.float32(max_norm)) / (n + float(np.float32(eps))))
    dev = g.cuda()
    norm = S.s6_clip_grad_norm([dev], max_norm, eps=eps)
    assert abs(norm.item() - n) <= R.NORM_REL * n
    half = R.HALF[t] if t == "bf16" else 0.0
    # one rounding more (the second factor), and the smallest step of the storage type
    step = 2.0 ** -133 if t == "bf16" else 2.0 ** -149
    R.within(dev.double().cpu().numpy(), want, (R.SCALED_REL + R.U + half) * (1 + half) * np.abs(want) + step, "clipped")
