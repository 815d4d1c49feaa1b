"""GPU tests of the training-step operators against float64 formulas, within bounds
derived from the float32 arithmetic (train_reference.py): LayerNorm forward and
backward, the conv's backward, the gradients' norm and clipping, and a block's
training step that runs them together with the scan."""
import math

import numpy as np
import pytest

import s6_inputs as SI
import train_reference as R
from s6_testutil import as_f64, from_dev, note, to_dev

pytestmark = pytest.mark.gpu

CANARY = 7.0


def _draw(rng, shape, t, scale=1.0):
    """A float64 array of values that the storage type holds, and the device tensor."""
    a = SI.to_storage((scale * rng.standard_normal(shape)).astype(np.float32), t)
    return as_f64(a), to_dev(a)


def _dtype(t):
    import torch
    return torch.bfloat16 if t == "bf16" else torch.float32


def _guarded(shape, dtype, off=0):
    """A contiguous tensor inside a larger buffer of canaries, `off` elements behind its start."""
    import torch
    n = math.prod(shape)
    buf = torch.full((n + off + 32,), CANARY, dtype=dtype, device="cuda")
    return buf[off:off + n].view(shape), buf, (off, off + n)


def _untouched(buf, span):
    return bool((buf[:span[0]] == CANARY).all()) and bool((buf[span[1]:] == CANARY).all())


def _f64(t):
    return as_f64(from_dev(t))


# -------------------------------------------------------------- LayerNorm
TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")]
# one row and one column, a part of a warp, every count of vectors a thread holds, the border to several warps,
# odd widths on each side of it, and the widest rows with their wide form
SHAPES = [(1, 1), (3, 2), (5, 8), (67, 7), (131, 9), (45, 16), (33, 31), (70, 33), (9, 64), (13, 65), (30001, 12), (1, 384), (300, 384), (9, 130), (37, 500), (2, 512), (4, 513), (3, 516),
          (21, 1001), (33, 1536), (2500, 64), (5, 2560), (3, 2561), (2, 8192), (2, 8191), (2, 8196), (3, 8193),
          (1, 20000), (7001, 516), (2500, 1031), (1300, 2568)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("rows,W", SHAPES)
def test_layernorm_forward(rows, W, xt, yt, add):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(rows * 7 + W)
    x, xd = _draw(rng, (rows, W), xt)
    r, rd = _draw(rng, (rows, W), yt)
    w, wd = _draw(rng, (W,), "f32")
    b, bd = _draw(rng, (W,), "f32")
    ref, tol = R.ln_fwd(x, w, b, 1e-5, r if add else None)
    y, ybuf, yspan = _guarded((rows, W), _dtype(yt))
    s, sbuf, sspan = _guarded((rows, W), _dtype(xt))
    out = S.s6_layernorm_fwd(xd, wd, bd, r=rd if add else None, s=s if add else None, y=y, y_dtype=_dtype(yt))
    torch.cuda.synchronize()
    assert out[0] is y and out[1] is (s if add else xd)
    note("layernorm fwd y (share of its bound)",
         R.within(_f64(y), ref["y"], tol["y"] + R.HALF[yt] * (np.abs(ref["y"]) + tol["y"]), "y"))
    R.within(out[2].cpu().numpy(), ref["mean"], tol["mean"] + R.U * np.abs(ref["mean"]), "mean")
    R.within(out[3].cpu().numpy(), ref["rstd"], tol["rstd"], "rstd")
    assert _untouched(ybuf, yspan) and _untouched(sbuf, sspan)
    if add:  # one float32 sum, then the rounding to the stream's type
        R.within(_f64(s), ref["s"], (R.U + R.HALF[xt] * (1 + R.U)) * np.abs(ref["s"]), "s")
        # the sum may go into x itself
        x2 = xd.clone()
        y2, s2, _, _ = S.s6_layernorm_fwd(x2, wd, bd, r=rd, s=x2, y_dtype=_dtype(yt), want_stats=False)
        assert s2 is x2 and torch.equal(x2, s) and torch.equal(y2, y)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("rows,W", SHAPES)
def test_layernorm_backward(rows, W, xt, yt, add):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(rows * 11 + W)
    x, xd = _draw(rng, (rows, W), xt)
    dy, dyd = _draw(rng, (rows, W), yt)
    ds, dsd = _draw(rng, (rows, W), "f32")
    w, wd = _draw(rng, (W,), "f32")
    fwd, _ = R.ln_fwd(x, w, 0.0, 1e-5)
    mean, rstd = fwd["mean"].astype(np.float32), fwd["rstd"].astype(np.float32)
    ref, tol = R.ln_bwd(dy, x, mean.astype(np.float64), rstd.astype(np.float64), w, ds if add else None)
    dx, buf, span = _guarded((rows, W), torch.float32)
    got = S.s6_layernorm_bwd(dyd, xd, to_dev(mean), to_dev(rstd), wd, ds=dsd if add else None, dx=dx)
    torch.cuda.synchronize()
    for k in ("dx", "dw", "db"):
        note(f"layernorm bwd {k} (share of its bound)", R.within(got[k].cpu().numpy(), ref[k], tol[k], k))
    assert got["dx"] is dx and _untouched(buf, span)
    # the same bits again; without the parameters' gradients; and into ds itself
    again = S.s6_layernorm_bwd(dyd, xd, to_dev(mean), to_dev(rstd), wd, ds=dsd if add else None)
    assert all(torch.equal(again[k], got[k]) for k in got)
    only = S.s6_layernorm_bwd(dyd, xd, to_dev(mean), to_dev(rstd), wd, ds=dsd if add else None, want_params=False)
    assert torch.equal(only["dx"], dx) and only["dw"] is None and only["db"] is None
    if add:
        S.s6_layernorm_bwd(dyd, xd, to_dev(mean), to_dev(rstd), wd, ds=dsd, dx=dsd)
        assert torch.equal(dsd, dx)


@pytest.mark.parametrize("W", [384, 1536])
def test_layernorm_rows_off_the_vector_alignment(W):
    """Tensors that begin one element into their memory take single elements, with the
    same values within the bounds; without w and b, which are then ones and zeros."""
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(W)
    rows = 5
    for xt, yt in TYPES:
        x, xd0 = _draw(rng, (rows, W), xt)
        xd, _, _ = _guarded((rows, W), _dtype(xt), off=1)
        xd.copy_(xd0)
        y, ybuf, yspan = _guarded((rows, W), _dtype(yt), off=3)
        ref, tol = R.ln_fwd(x, np.ones(W), np.zeros(W), 1e-5)
        _, _, mean, rstd = S.s6_layernorm_fwd(xd, y=y)
        R.within(_f64(y), ref["y"], tol["y"] + R.HALF[yt] * (np.abs(ref["y"]) + tol["y"]), "y")
        assert _untouched(ybuf, yspan)
        dy, dyd = _draw(rng, (rows, W), yt)
        ref, tol = R.ln_bwd(dy, x, _f64(mean), _f64(rstd), np.ones(W))
        got = S.s6_layernorm_bwd(dyd, xd, mean, rstd)
        for k in ("dx", "dw", "db"):
            R.within(got[k].cpu().numpy(), ref[k], tol[k], k)


def test_layernorm_mean_far_above_the_deviations():
    """Rows at 1000 with deviations of 1: the squares of the values would lose them."""
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(1)
    for W in (384, 1000, 3000, 9000):
        x = (1000.0 + rng.standard_normal((4, W))).astype(np.float32)
        ref, tol = R.ln_fwd(x.astype(np.float64), np.ones(W), np.zeros(W), 1e-5)
        y, _, mean, rstd = S.s6_layernorm_fwd(to_dev(x))
        R.within(_f64(y), ref["y"], tol["y"] + R.U * np.abs(ref["y"]), "y")
        R.within(_f64(rstd), ref["rstd"], tol["rstd"], "rstd")
        assert tol["y"].max() < 0.05


def test_layernorm_rows_keep_to_themselves():
    """A constant row gives b, and rows with infinities or NaN give NaN there only."""
    import torch
    import selective_state_space_19_b200 as S
    for W in (5, 384, 1001, 1536, 9000):
        x = torch.randn(6, W, device="cuda")
        b = torch.randn(W, device="cuda")
        x[1], x[2, W // 2], x[4, 0] = 3.0, float("inf"), float("nan")
        y, _, mean, rstd = S.s6_layernorm_fwd(x, b=b)
        assert torch.equal(y[1], b) or torch.allclose(y[1], b, atol=1.2e-4)  # 3 W / W: two roundings, over sqrt(eps)
        bad = torch.tensor([2, 4], device="cuda")
        good = torch.tensor([0, 1, 3, 5], device="cuda")
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[good]).all()
        clean = S.s6_layernorm_fwd(x[good].contiguous(), b=b)
        assert torch.equal(clean[0], y[good]) and torch.equal(clean[2], mean[good])
        dy = torch.randn(6, W, device="cuda")
        got = S.s6_layernorm_bwd(dy, x, mean, rstd)
        assert torch.isfinite(got["dx"][good]).all() and torch.isfinite(got["db"]).all()


def test_layernorm_no_rows_and_leading_dimensions():
    import torch
    import selective_state_space_19_b200 as S
    x = torch.empty(0, 64, device="cuda")
    y, s, mean, rstd = S.s6_layernorm_fwd(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    g = S.s6_layernorm_bwd(y, x, mean, rstd)
    assert not g["dw"].any() and not g["db"].any() and g["dx"].shape == (0, 64)
    x = torch.randn(2, 3, 4, 40, device="cuda")
    y, s, mean, rstd = S.s6_layernorm_fwd(x)
    assert y.shape == x.shape and mean.shape == (2, 3, 4)
    flat = S.s6_layernorm_fwd(x.view(24, 40))
    assert torch.equal(flat[0].view_as(y), y)
    g = S.s6_layernorm_bwd(y, x, mean, rstd)
    assert torch.equal(g["dx"].view(24, 40), S.s6_layernorm_bwd(flat[0], flat[1], flat[2], flat[3])["dx"])


def test_layernorm_refusals():
    import torch
    import selective_state_space_19_b200 as S
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        S.s6_layernorm_fwd(x.t())
    with pytest.raises(TypeError):
        S.s6_layernorm_fwd(x.half())
    with pytest.raises(TypeError):
        S.s6_layernorm_fwd(x.bfloat16(), y_dtype=torch.float32)
    with pytest.raises(ValueError, match="needs r"):
        S.s6_layernorm_fwd(x, s=x)
    with pytest.raises(ValueError, match="shape"):
        S.s6_layernorm_fwd(x, w=torch.ones(63, device="cuda"))
    with pytest.raises(S.S6Error):
        S.s6_layernorm_fwd(x, eps=-1.0)
    with pytest.raises(S.S6Error):
        S.s6_layernorm_fwd(x[:, :0].contiguous())
    m = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        S.s6_layernorm_bwd(x, x, m[:3], m)
    with pytest.raises(TypeError):
        S.s6_layernorm_bwd(x, x.bfloat16(), m, m)


# ------------------------------------------------------------------- conv
CONV_TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
CONV_SHAPES = [(1, 1, 1), (2, 2, 4), (1, 3, 5), (3, 7, 130), (2, 16, 64), (1, 17, 128), (2, 100, 136), (3, 65, 6),
               (1, 1000, 8), (2, 515, 33), (40, 3, 12), (1200, 2, 8)]


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("xt,gt", CONV_TYPES)
@pytest.mark.parametrize("Bt,L,d", CONV_SHAPES)
def test_conv_backward(Bt, L, d, xt, gt, K):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(L * 3 + d + K)
    x, xd = _draw(rng, (Bt, L, d), xt, 2.0)
    g, gd = _draw(rng, (Bt, L, d), gt)
    w, wd = _draw(rng, (d, K), "f32")
    b, bd = _draw(rng, (d,), "f32")
    for bias in (True, False):
        ref, tol = R.conv_bwd(x, w, b if bias else None, g)
        got = S.causal_conv1d_silu_bwd(xd, wd, gd, conv_b=bd if bias else None)
        torch.cuda.synchronize()
        for k in ("dx", "dconv_w") + (("dconv_b",) if bias else ()):
            note(f"conv bwd {k} (share of its bound)", R.within(got[k].cpu().numpy(), ref[k], tol[k], k))
        assert bias or got["dconv_b"] is None
    again = S.causal_conv1d_silu_bwd(xd, wd, gd)
    assert all(again[k] is None or torch.equal(again[k], got[k]) for k in got)


def test_conv_backward_off_the_vector_alignment():
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(5)
    shape = (2, 37, 64)
    for off in (1, 2):
        for xt, gt in CONV_TYPES:
            x, x0 = _draw(rng, shape, xt)
            g, gd = _draw(rng, shape, gt)
            w, wd = _draw(rng, (64, 4), "f32")
            xd, _, _ = _guarded(shape, _dtype(xt), off=off)
            xd.copy_(x0)
            ref, tol = R.conv_bwd(x, w, None, g)
            got = S.causal_conv1d_silu_bwd(xd, wd, gd)
            for k in ("dx", "dconv_w"):
                R.within(got[k].cpu().numpy(), ref[k], tol[k], k)


def test_conv_backward_is_the_forwards_difference():
    """Along a direction, the gradients agree with a central difference of the float64 forward."""
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(8)
    x, xd = _draw(rng, (2, 50, 24), "f32")
    g, gd = _draw(rng, (2, 50, 24), "f32")
    w, wd = _draw(rng, (24, 4), "f32")
    b, bd = _draw(rng, (24,), "f32")
    got = S.causal_conv1d_silu_bwd(xd, wd, gd, conv_b=bd)
    ex, ew, eb = rng.standard_normal(x.shape), rng.standard_normal(w.shape), rng.standard_normal(b.shape)
    h = 1e-6
    up, down = (float((g * R.conv_fwd(x + q * ex, w + q * ew, b + q * eb)).sum()) for q in (h, -h))
    slope = sum(float((got[k].cpu().numpy().astype(np.float64) * e).sum())
                for k, e in (("dx", ex), ("dconv_w", ew), ("dconv_b", eb)))
    ref, tol = R.conv_bwd(x, w, b, g)
    allowed = sum(float((tol[k] * np.abs(e)).sum()) for k, e in (("dx", ex), ("dconv_w", ew), ("dconv_b", eb)))
    # the difference itself: h^2 / 6 of a third derivative, and the forward's float64 rounding over h
    assert abs(slope - (up - down) / (2 * h)) <= allowed + 1e-5


@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv_backward_reaches_k_tokens_only(K):
    """An infinite input changes the gradients of the tokens whose windows hold it, no others."""
    import torch
    import selective_state_space_19_b200 as S
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(2, 40, 8, device="cuda", generator=gen)
    g = torch.randn(2, 40, 8, device="cuda", generator=gen)
    w = torch.randn(8, K, device="cuda", generator=gen)
    clean = S.causal_conv1d_silu_bwd(x, w, g)["dx"]
    x[1, 20, 3] = float("inf")
    got = S.causal_conv1d_silu_bwd(x, w, g)["dx"]
    same = torch.ones_like(x, dtype=torch.bool)
    same[1, 20 - K + 1:20 + K, 3] = False
    assert torch.equal(got[same], clean[same])
    # large inputs on both sides: the factor tends to 1 and to 0, with no NaN between
    x = torch.full((1, 30, 8), 1e30, device="cuda")
    w = torch.ones(8, K, device="cuda")
    w[::2] = -1.0
    got = S.causal_conv1d_silu_bwd(x, w, torch.ones_like(x))["dx"]
    assert torch.isfinite(got).all()
    assert torch.equal(got[0, :, ::2], torch.zeros_like(got[0, :, ::2]))
    assert torch.equal(got[0, :30 - K + 1, 1::2], torch.full_like(got[0, :30 - K + 1, 1::2], float(K)))


def test_conv_backward_empty_and_refusals():
    import torch
    import selective_state_space_19_b200 as S
    w = torch.randn(8, 4, device="cuda")
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        got = S.causal_conv1d_silu_bwd(x, w, x, conv_b=w[:, 0].contiguous())
        assert got["dx"].shape == shape and not got["dconv_w"].any() and not got["dconv_b"].any()
    x = torch.randn(2, 5, 8, device="cuda")
    with pytest.raises(S.S6Error):
        S.causal_conv1d_silu_bwd(x, torch.randn(8, 5, device="cuda"), x)
    with pytest.raises(TypeError):
        S.causal_conv1d_silu_bwd(x, w, x.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        S.causal_conv1d_silu_bwd(x, w, x[:, :4].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        S.causal_conv1d_silu_bwd(x, w, x.transpose(1, 2).contiguous().transpose(1, 2))


# -------------------------------------------------------------- gradients
def _gradient_list(rng, sizes, types, scale=1.0):
    pairs = [_draw(rng, (n,), t, scale) for n, t in zip(sizes, types)]
    return [p[0] for p in pairs], [p[1] for p in pairs]


@pytest.mark.parametrize("sizes", [[1], [7], [8192], [8193, 1, 5], [0, 3, 0], [100, 8191, 16384, 16385, 40000, 9],
                                   [3] * 97, [17] * 1025, [1000000]])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_gradient_norm_and_clipping(sizes, kind):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(len(sizes) + sizes[0])
    types = [kind if kind != "mixed" else ("f32", "bf16")[i % 3 == 1] for i in range(len(sizes))]
    ref, dev = _gradient_list(rng, sizes, types, 0.1)
    n = R.grad_norm(ref)
    norm = S.s6_grad_norm(dev)
    torch.cuda.synchronize()
    assert norm.shape == () and abs(norm.item() - n) <= R.NORM_REL * n
    assert torch.equal(norm, S.s6_grad_norm(dev))
    # above the bound: scaled
    c = 0.3 * n / (n + 1e-6)
    got = [g.clone() for g in dev]
    assert torch.equal(S.s6_clip_grad_norm(got, 0.3 * n), norm)
    for g, a, t in zip(got, ref, types):
        half = R.HALF[t] if t == "bf16" else 0.0
        R.within(_f64(g), a * c, (R.SCALED_REL + half * (1 + R.SCALED_REL)) * np.abs(a * c), "clipped")
    # by a given norm: the same
    by = [g.clone() for g in dev]
    S.s6_grad_clip(by, norm, 0.3 * n)
    assert all(torch.equal(p, q) for p, q in zip(by, got))
    # below the bound: as they were
    S.s6_clip_grad_norm(by, 0.5 * n)
    assert all(torch.equal(p, q) for p, q in zip(by, got))


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_gradients_at_every_alignment_leave_their_neighbours(t):
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(3)
    for off in range(9):
        for n in (1, 5, 8, 15, 16, 31, 8200):
            a, a0 = _draw(rng, (n,), t)
            g, buf, span = _guarded((n,), _dtype(t), off=off)
            g.copy_(a0)
            want = R.grad_norm([a])
            norm = S.s6_clip_grad_norm([g], 0.5 * want)
            assert abs(norm.item() - want) <= R.NORM_REL * want, (off, n)
            c = 0.5 * want / (want + 1e-6)
            half = R.HALF[t] if t == "bf16" else 0.0
            R.within(_f64(g), a * c, (R.SCALED_REL + half * (1 + R.SCALED_REL)) * np.abs(a * c), "clipped")
            assert _untouched(buf, span), (off, n)
    torch.cuda.synchronize()


def test_gradient_norm_over_the_whole_range_of_float32():
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(4)
    for scale in (1e-38, 1e-30, 1e-21, 1e-13, 1.0, 1e18, 1e30, 1e35):
        for n in (3, 8, 5000):
            a = (scale * rng.standard_normal(n)).astype(np.float32)
            want = R.grad_norm([a])
            got = S.s6_grad_norm([to_dev(a)]).item()
            assert abs(got - want) <= R.NORM_REL * want + 2.0 ** -150, (scale, n, got, want)
    # small elements beside large ones, and zeros alone
    a = np.concatenate([np.full(4096, 1e-25), np.full(4096, 1e-24), [3e-22]]).astype(np.float32)
    assert abs(S.s6_grad_norm([to_dev(a)]).item() - R.grad_norm([a])) <= R.NORM_REL * R.grad_norm([a])
    z = torch.zeros(1000, device="cuda")
    assert S.s6_clip_grad_norm([z], 1.0).item() == 0.0 and not z.any()
    # a bound of 0 clears every gradient
    g = torch.randn(1000, device="cuda")
    S.s6_clip_grad_norm([g], 0.0)
    assert not g.any()


def test_gradients_that_are_not_finite():
    import torch
    import selective_state_space_19_b200 as S
    for t in (torch.float32, torch.bfloat16):
        a, b = torch.ones(3000, device="cuda", dtype=t), torch.ones(100, device="cuda")
        a[2000] = float("inf")
        norm = S.s6_clip_grad_norm([a, b], 1.0)
        assert norm.item() == float("inf") and not b.any() and torch.isnan(a[2000]) and not a[:2000].any()
        a, b = torch.ones(3000, device="cuda", dtype=t), torch.ones(100, device="cuda")
        a[7] = float("nan")
        norm = S.s6_clip_grad_norm([a, b], 1e9)
        assert torch.isnan(norm) and torch.isnan(a).all() and torch.isnan(b).all()
    huge = torch.full((10000,), 3e38, device="cuda")  # a norm above the largest float32
    assert S.s6_grad_norm([huge]).item() == float("inf")


def test_gradient_lists_of_every_kind():
    import torch
    import selective_state_space_19_b200 as S
    assert S.s6_grad_norm([]).item() == 0.0
    assert S.s6_clip_grad_norm([None], 1.0).item() == 0.0
    assert S.s6_grad_norm([torch.empty(0, device="cuda")]).item() == 0.0
    g = {"du": torch.full((2, 8), 3.0, device="cuda"), "dz": None, "dB": torch.full((16,), 4.0, device="cuda")}
    out = torch.zeros(1, device="cuda")
    assert S.s6_grad_norm(g, norm=out) is out and out.item() == 20.0
    assert S.s6_grad_norm(g["du"]).item() == 12.0
    S.s6_grad_clip(g.values(), out, 10.0, eps=0.0)
    assert torch.equal(g["du"], torch.full((2, 8), 1.5, device="cuda"))
    assert S.s6_grad_norm([out, out]).item() == pytest.approx(20.0 * 2 ** 0.5)  # read only: twice is allowed
    with pytest.raises(S.S6Error):
        S.s6_clip_grad_norm([out, out], 1.0)
    with pytest.raises(S.S6Error):
        S.s6_clip_grad_norm([g["du"]], float("inf"))
    with pytest.raises(ValueError, match="contiguous"):
        S.s6_grad_norm([g["du"].t()])
    with pytest.raises(TypeError):
        S.s6_grad_norm([g["du"].half()])
    with pytest.raises(ValueError, match="1 element"):
        S.s6_grad_norm(g, norm=torch.zeros(2, device="cuda"))


# ----------------------------------------------- streams, graphs, two at once
def _calls(S, seed, rows=300, W=384):
    """One call of each operator on its own inputs: a function and its inputs."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)
    x, r, w, b, dy = normal(rows, W), normal(rows, W), normal(W), normal(W), normal(rows, W)
    xc, g, cw, cb = normal(3, 100, 64), normal(3, 100, 64), normal(64, 4), normal(64)
    grads = [normal(5000), normal(77)]

    def run(stream=None):
        y, s, mean, rstd = S.s6_layernorm_fwd(x, w, b, r=r, stream=stream)
        ln = S.s6_layernorm_bwd(dy, s, mean, rstd, w, ds=r, stream=stream)
        cv = S.causal_conv1d_silu_bwd(xc, cw, g, conv_b=cb, stream=stream)
        norm = S.s6_clip_grad_norm(grads, 1.0, stream=stream)
        return [y, s, mean, rstd, *ln.values(), *cv.values(), norm]
    return run, [x, r, dy, xc, g], grads


def test_on_two_streams_at_once():
    import torch
    import selective_state_space_19_b200 as S
    sets = [_calls(S, k, rows=2000 + 100 * k) for k in range(2)]
    keep = [[g.clone() for g in s[2]] for s in sets]
    want = [run() for run, _, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, _, grads), old in zip(sets, keep):
            for g, o in zip(grads, old):
                g.copy_(o)
        torch.cuda.synchronize()
        got = [run(stream=s) for (run, _, _), s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_and_replayed_in_two_graphs():
    """Two graphs of the same operators, replayed by turns and at the same time, on inputs
    that change between the replays."""
    import torch
    import selective_state_space_19_b200 as S
    sets = [_calls(S, 10 + k) for k in range(2)]
    graphs, outs = [], []
    for run, _, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # no call before the capture is needed
            outs.append(run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(3):
        for _, inputs, grads in sets:
            for t in inputs + grads:
                t.normal_()
        keep = [[g.clone() for g in s[2]] for s in sets]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        clipped = [[g.clone() for g in s[2]] for s in sets]
        for (run, _, grads), old, a, c in zip(sets, keep, got, clipped):
            for g, o in zip(grads, old):
                g.copy_(o)
            want = run()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(a, want)), turn
            assert all(torch.equal(p, q) for p, q in zip(c, grads)), turn


@pytest.mark.parametrize("W", [40, 1000, 1536, 8192, 9001])
def test_every_form_of_the_layernorm_captured(W):
    """Rows of some lanes, of a block through shared memory and of several walks, in one
    graph and on a second stream, without an earlier call."""
    import torch
    import selective_state_space_19_b200 as S
    run, inputs, grads = _calls(S, W, rows=700, W=W)
    keep = [g.clone() for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    side = torch.cuda.Stream()
    for turn in range(2):
        for t in inputs:
            t.normal_()
        results = []
        for how in ("replay", "call", "stream"):
            for g, o in zip(grads, keep):
                g.copy_(o)
            torch.cuda.synchronize()
            if how == "replay":
                graph.replay()
                torch.cuda.synchronize()
                results.append([t.clone() for t in out])
            else:
                results.append(run(stream=side if how == "stream" else None))
                torch.cuda.synchronize()
        assert all(torch.equal(p, q) for r in results[1:] for p, q in zip(r, results[0]))


def test_gradients_of_zero_stay_zero_whatever_the_bound():
    import torch
    import selective_state_space_19_b200 as S
    z = torch.zeros(300, device="cuda")
    for max_norm, eps in ((0.0, 0.0), (0.0, 1e-6), (1.0, 0.0)):
        assert S.s6_clip_grad_norm([z], max_norm, eps=eps).item() == 0.0
        assert torch.equal(z, torch.zeros_like(z))


def test_layernorm_result_does_not_depend_on_the_rows_around_it():
    """A row gives the same bits alone, in a batch and at another place in it."""
    import torch
    import selective_state_space_19_b200 as S
    for W in (33, 384, 1001, 2560, 8191):
        for t in (torch.float32, torch.bfloat16):
            x = torch.randn(37, W, device="cuda").to(t)
            dy = torch.randn(37, W, device="cuda").to(t)
            y, _, mean, rstd = S.s6_layernorm_fwd(x)
            dx = S.s6_layernorm_bwd(dy, x, mean, rstd)["dx"]
            for first in (0, 1, 8, 36):
                part = x[first:].clone()
                y2, _, m2, r2 = S.s6_layernorm_fwd(part)
                dx2 = S.s6_layernorm_bwd(dy[first:].clone(), part, m2, r2)["dx"]
                assert torch.equal(y2, y[first:]) and torch.equal(m2, mean[first:]) and torch.equal(dx2, dx[first:])


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their last rows, tokens and elements equal those of a
    small call on the same values."""
    import torch
    import selective_state_space_19_b200 as S
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    bf = torch.bfloat16
    for rows, W in ((5_700_000, 384), (840_000, 2561), (240_000, 9001)):  # a form of the kernels each
        x, dy = torch.empty(rows, W, device="cuda", dtype=bf), torch.empty(rows, W, device="cuda", dtype=bf)
        assert x.numel() > 1 << 31
        x.normal_()
        dy.normal_()
        y, _, mean, rstd = S.s6_layernorm_fwd(x)
        y2, _, m2, r2 = S.s6_layernorm_fwd(x[-50:].clone())
        assert torch.equal(y[-50:], y2) and torch.equal(mean[-50:], m2) and torch.equal(rstd[-50:], r2)
        del y
        dx = S.s6_layernorm_bwd(dy, x, mean, rstd)["dx"]
        assert torch.equal(dx[-50:], S.s6_layernorm_bwd(dy[-50:].clone(), x[-50:].clone(), m2, r2)["dx"])
        del x, dy, dx
    x = torch.randn(3, 650_000, 1102, device="cuda", dtype=bf)
    w = torch.randn(1102, 4, device="cuda")
    assert x.numel() > 1 << 31
    dx = S.causal_conv1d_silu_bwd(x, w, x)["dx"]
    tail = x[2:, -64:].clone()
    assert torch.equal(dx[2:, -60:], S.causal_conv1d_silu_bwd(tail, w, tail)["dx"][:, -60:])
    del dx, tail
    flat = x.view(-1)
    flat.fill_(0.0)
    flat[-1], flat[5], flat[(1 << 31) + 3] = 3.0, 4.0, 12.0
    assert S.s6_clip_grad_norm([flat], 6.5, eps=0.0).item() == 13.0
    assert flat[-1].item() == 1.5 and flat[5].item() == 2.0 and flat[(1 << 31) + 3].item() == 6.0


def test_the_c_call_without_the_optional_outputs():
    """The C ABI's own freedom: a sum that is not stored, statistics that are not wanted."""
    import ctypes
    import torch
    import selective_state_space_19_b200 as S
    for W in (40, 1536, 9000):
        x, r = torch.randn(9, W, device="cuda"), torch.randn(9, W, device="cuda")
        want = S.s6_layernorm_fwd(x, r=r)[0]
        keep = x.clone()
        y = torch.empty_like(x)
        dims = S.NormDims(9, W, S.S6_F32, S.S6_F32, 1e-5)
        st = S.lib().s6_layernorm_fwd(ctypes.byref(dims), x.data_ptr(), r.data_ptr(), None, None, None, y.data_ptr(),
                                      None, None, torch.cuda.current_stream().cuda_stream)
        assert st == S.S6_OK and torch.equal(y, want) and torch.equal(x, keep)


def test_no_bounded_wait_gave_up():
    import selective_state_space_19_b200 as S
    assert S.s6_device_status() == 0


def test_stream_of_another_device_is_refused():
    import torch
    import selective_state_space_19_b200 as S

    class Elsewhere:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on"):
        S.s6_layernorm_fwd(torch.zeros(2, 8, device="cuda:0"), stream=Elsewhere())


# ------------------------------------------------- a block's training step
def _block_reference(p, x, dout):
    """The block in torch float64 with autograd: out = s + out_proj(scan(...)); the
    gradients of sum(dout * out)."""
    import torch
    q = {k: torch.from_numpy(v).double().requires_grad_() for k, v in p.items()}
    xs = torch.from_numpy(x).double().requires_grad_()
    Bt, L, dm = x.shape
    mean = xs.mean(-1, keepdim=True)
    hn = (xs - mean) / torch.sqrt(((xs - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * q["ln_w"] + q["ln_b"]
    di, N, K = q["A_log"].shape[0], 16, q["conv_w"].shape[1]
    xz = hn @ q["in_w"].T
    xin, z = xz[..., :di], xz[..., di:]
    pre = sum(torch.nn.functional.pad(xin, (0, 0, K - 1 - k, 0))[:, :L] * q["conv_w"][:, k] for k in range(K))
    xc = torch.nn.functional.silu(pre + q["conv_b"])
    dbc = xc @ q["xp_w"].T
    R_ = q["dt_w"].shape[1]
    dt = torch.nn.functional.softplus(dbc[..., :R_] @ q["dt_w"].T + q["dt_bias"])
    B, C = dbc[..., R_:R_ + N], dbc[..., R_ + N:]
    A = -torch.exp(q["A_log"])
    h, ys = torch.zeros(Bt, di, N, dtype=torch.float64), []
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * xc[:, t])[..., None] * B[:, t, None, :]
        ys.append((h * C[:, t, None, :]).sum(-1) + q["D"] * xc[:, t])
    y = torch.stack(ys, 1) * torch.nn.functional.silu(z)
    out = xs + y @ q["out_w"].T
    names = list(q)
    grads = torch.autograd.grad((out * torch.from_numpy(dout).double()).sum(), [xs] + [q[k] for k in names])
    return out.detach().numpy(), dict(zip(["x"] + names, (g.numpy() for g in grads)))


def test_a_blocks_training_step():
    """LayerNorm, in_proj, conv, x_proj, scan, out_proj and all the way back, through the
    library's calls, then one clipping of all gradients; every gradient against
    float64 differentiation of the block.  The bound is the scan backward's, 2e-3 (1 + |g|)."""
    import torch
    import selective_state_space_19_b200 as S
    rng = np.random.default_rng(21)
    Bt, L, dm, di, N, K, Rk = 2, 40, 32, 64, 16, 4, 4

    def f32(*shape, scale=1.0):
        return (scale * rng.standard_normal(shape)).astype(np.float32)
    p = {"ln_w": 1 + f32(dm, scale=0.1), "ln_b": f32(dm, scale=0.1), "in_w": f32(2 * di, dm, scale=dm ** -0.5),
         "conv_w": f32(di, K, scale=0.5), "conv_b": f32(di, scale=0.1),
         "xp_w": f32(Rk + 2 * N, di, scale=di ** -0.5), "dt_w": f32(di, Rk, scale=0.5), "dt_bias": f32(di) - 3.0,
         "A_log": np.log(np.arange(1, N + 1, dtype=np.float32))[None].repeat(di, 0), "D": 1 + f32(di, scale=0.1),
         "out_w": f32(dm, di, scale=di ** -0.5)}
    p = {k: np.ascontiguousarray(v, dtype=np.float32) for k, v in p.items()}
    x, dout = f32(Bt, L, dm), f32(Bt, L, dm)
    ref_out, ref = _block_reference(p, x, dout)

    q = {k: to_dev(v) for k, v in p.items()}
    xd, doutd = to_dev(x), to_dev(dout)
    # forward
    hn, s, mean, rstd = S.s6_layernorm_fwd(xd, q["ln_w"], q["ln_b"])
    xz = hn @ q["in_w"].T
    xin, z = xz[..., :di].contiguous(), xz[..., di:].contiguous()
    xc = S.causal_conv1d_silu_fwd(xin, q["conv_w"], q["conv_b"])
    dbc = xc @ q["xp_w"].T
    dtr = dbc[..., :Rk]
    dt = dtr @ q["dt_w"].T
    B, C = dbc[..., Rk:Rk + N].contiguous(), dbc[..., Rk + N:].contiguous()
    y, _, ckpt = S.s6_scan_fwd_ckpt(xc, dt, q["A_log"], B, C, q["D"], z=z, dt_bias=q["dt_bias"])
    branch = y @ q["out_w"].T
    # the add of the branch, as the next block's LayerNorm does it
    _, out, _, _ = S.s6_layernorm_fwd(s, q["ln_w"], q["ln_b"], r=branch)
    assert np.max(np.abs(out.cpu().numpy() - ref_out) / (1 + np.abs(ref_out))) <= 1e-4
    # backward
    dy = doutd @ q["out_w"]
    g = S.s6_scan_bwd(xc, dt, q["A_log"], B, C, q["D"], dy, z=z, dt_bias=q["dt_bias"], ckpt=ckpt)
    ddbc = torch.cat([g["ddt"] @ q["dt_w"], g["dB"], g["dC"]], -1)
    dxc = g["du"] + ddbc @ q["xp_w"]
    cv = S.causal_conv1d_silu_bwd(xin, q["conv_w"], dxc, conv_b=q["conv_b"])
    dxz = torch.cat([cv["dx"], g["dz"]], -1)
    ln = S.s6_layernorm_bwd(dxz @ q["in_w"], s, mean, rstd, q["ln_w"], ds=doutd)

    def outer(a, b):
        return a.reshape(-1, a.shape[-1]).T @ b.reshape(-1, b.shape[-1])
    got = {"x": ln["dx"], "ln_w": ln["dw"], "ln_b": ln["db"], "in_w": outer(dxz, hn), "conv_w": cv["dconv_w"],
           "conv_b": cv["dconv_b"], "xp_w": outer(ddbc, xc), "dt_w": outer(g["ddt"], dtr), "dt_bias": g["ddt_bias"],
           "A_log": g["dA_log"], "D": g["dD"], "out_w": outer(doutd, y)}
    for k, v in ref.items():
        err = np.max(np.abs(got[k].cpu().numpy() - v) / (1 + np.abs(v)))
        note(f"block training step d{k} (f32)", err)
        assert err <= 2e-3, (k, err)
    # and the clipping of the parameters' gradients
    grads = {k: v for k, v in got.items() if k != "x"}
    before = {k: v.clone() for k, v in grads.items()}
    want = R.grad_norm([v.cpu().numpy() for v in before.values()])
    norm = S.s6_clip_grad_norm(grads, 1.0)
    assert abs(norm.item() - want) <= R.NORM_REL * want and want > 1.0
    for k, v in before.items():
        a = _f64(v) / (want + 1e-6)
        R.within(_f64(grads[k]), a, R.SCALED_REL * np.abs(a), k)
