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
