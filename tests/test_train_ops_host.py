"""CPU checks of the training-step operators: the float64 formulas that the GPU
tests compare with agree with central differences of the forward, and every
call refuses bad arguments before it touches a device."""
import ctypes

import numpy as np
import pytest

import train_reference as R


# ------------------------------------------------- the formulas themselves
def _differences(f, a, h=1e-5):
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        up = f()
        a[i] = keep - h
        down = f()
        a[i] = keep
        out[i] = (up - down) / (2 * h)
    return out


@pytest.mark.parametrize("rows,W,add", [(3, 7, True), (2, 1, False), (5, 4, False)])
def test_layernorm_gradients_are_the_forwards_differences(rows, W, add):
    rng = np.random.default_rng(rows * 10 + W)
    x, dy, ds = (rng.standard_normal((rows, W)) for _ in range(3))
    w, b = 1 + 0.3 * rng.standard_normal(W), rng.standard_normal(W)
    eps = 1e-2

    def loss():
        out, _ = R.ln_fwd(x, w, b, eps)
        return (dy * out["y"]).sum() + ((ds * x).sum() if add else 0.0)
    out, _ = R.ln_fwd(x, w, b, eps)
    got, _ = R.ln_bwd(dy, x, out["mean"], out["rstd"], w, ds if add else None)
    np.testing.assert_allclose(got["dx"], _differences(loss, x), atol=1e-7)
    np.testing.assert_allclose(got["dw"], _differences(loss, w), atol=1e-7)
    np.testing.assert_allclose(got["db"], _differences(loss, b), atol=1e-7)


@pytest.mark.parametrize("L,K", [(1, 4), (2, 4), (6, 4), (5, 3), (4, 2)])
def test_conv_gradients_are_the_forwards_differences(L, K):
    rng = np.random.default_rng(L * 10 + K)
    x, g = rng.standard_normal((2, L, 3)), rng.standard_normal((2, L, 3))
    w, b = rng.standard_normal((3, K)), rng.standard_normal(3)
    got, _ = R.conv_bwd(x, w, b, g)

    def loss():
        return (g * R.conv_fwd(x, w, b)).sum()
    np.testing.assert_allclose(got["dx"], _differences(loss, x), atol=1e-7)
    np.testing.assert_allclose(got["dconv_w"], _differences(loss, w), atol=1e-7)
    np.testing.assert_allclose(got["dconv_b"], _differences(loss, b), atol=1e-7)


# ----------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def S():
    from selective_state_space_19_b200 import _build
    import selective_state_space_19_b200 as S
    _build.build()
    S.lib()
    return S


P = ctypes.c_void_p
OK = P(16)


def _norm_dims(S, **kw):
    d = dict(rows=4, width=64, x_dtype=0, y_dtype=0, eps=1e-5)
    d.update(kw)
    return S.NormDims(**d)


def test_layernorm_forward_host_checks(S):
    def fwd(x=OK, r=None, w=OK, s=None, y=OK, mean=OK, **kw):
        return S.lib().s6_layernorm_fwd(ctypes.byref(_norm_dims(S, **kw)), x, r, w, OK, s, y, mean, OK, None)
    assert S.lib().s6_layernorm_fwd(None, OK, None, OK, OK, None, OK, OK, OK, None) == S.S6_ERR_INVALID_ARG
    assert fwd(rows=-1) == S.S6_ERR_INVALID_ARG
    assert fwd(width=0) == S.S6_ERR_INVALID_ARG
    assert fwd(eps=-1e-5) == S.S6_ERR_INVALID_ARG
    assert fwd(eps=float("nan")) == S.S6_ERR_INVALID_ARG
    assert fwd(eps=float("inf")) == S.S6_ERR_INVALID_ARG
    assert fwd(x=None) == S.S6_ERR_INVALID_ARG
    assert fwd(y=None) == S.S6_ERR_INVALID_ARG
    assert fwd(s=OK) == S.S6_ERR_INVALID_ARG                      # a sum without a summand
    assert fwd(x_dtype=2) == S.S6_ERR_UNSUPPORTED
    assert fwd(x_dtype=1, y_dtype=0) == S.S6_ERR_UNSUPPORTED      # a branch wider than its stream
    assert fwd(width=(1 << 24) + 1) == S.S6_ERR_UNSUPPORTED
    assert fwd(x=P(18)) == S.S6_ERR_ALIGNMENT
    assert fwd(mean=P(18)) == S.S6_ERR_ALIGNMENT
    assert fwd(y=P(17), y_dtype=1) == S.S6_ERR_ALIGNMENT
    assert fwd(rows=0, x=None, y=None) == S.S6_OK


def test_layernorm_backward_host_checks(S):
    big = 1 << 30

    def bwd(x=OK, mean=OK, dy=OK, dx=OK, dw=OK, ds=None, ws=OK, ws_bytes=big, **kw):
        return S.lib().s6_layernorm_bwd(ctypes.byref(_norm_dims(S, **kw)), x, mean, OK, OK, dy, ds, dx, dw, OK, ws,
                                        ws_bytes, None)
    for bad in (dict(x=None), dict(mean=None), dict(dy=None), dict(dx=None), dict(ws=None), dict(ws_bytes=8),
                dict(rows=-1)):
        assert bwd(**bad) == S.S6_ERR_INVALID_ARG, bad
    for bad in (dict(ds=P(18)), dict(dw=P(2)), dict(ws=P(20)), dict(x=P(18))):
        assert bwd(**bad) == S.S6_ERR_ALIGNMENT, bad
    assert bwd(x_dtype=1, y_dtype=0) == S.S6_ERR_UNSUPPORTED

    def ws(**kw):
        return S.lib().s6_layernorm_bwd_workspace(ctypes.byref(_norm_dims(S, **kw)))
    assert ws(rows=0) == 0 and ws(rows=-1) == S.S6_ERR_INVALID_ARG
    assert 0 < ws(rows=1) <= ws(rows=100) <= ws(rows=10 ** 6) == ws(rows=10 ** 7)
    assert ws(rows=3, width=10 ** 5) >= 3 * 8 + 2 * 4 * 10 ** 5


def test_conv_backward_host_checks(S):
    def bwd(x=OK, w=OK, g=OK, gt=0, dx=OK, dw=OK, db=None, ws=OK, ws_bytes=1 << 30, **kw):
        d = dict(batch=2, seqlen=8, d_inner=64, d_state=1, conv_width=4, io_dtype=0)
        d.update(kw)
        return S.lib().causal_conv1d_silu_bwd(ctypes.byref(S.Dims(**d)), x, w, None, g, gt, dx, dw, db, ws, ws_bytes,
                                              None)
    for bad in (dict(x=None), dict(w=None), dict(g=None), dict(dx=None), dict(dw=None), dict(ws=None),
                dict(ws_bytes=16), dict(batch=-1), dict(d_inner=0)):
        assert bwd(**bad) == S.S6_ERR_INVALID_ARG, bad
    for bad in (dict(conv_width=1), dict(conv_width=5), dict(io_dtype=3), dict(gt=1), dict(gt=9),
                dict(seqlen=1 << 31)):
        assert bwd(**bad) == S.S6_ERR_UNSUPPORTED, bad
    for bad in (dict(x=P(18)), dict(dx=P(2)), dict(db=P(2)), dict(ws=P(4))):
        assert bwd(**bad) == S.S6_ERR_ALIGNMENT, bad


def _grads(ptrs, numel, types):
    n = len(ptrs)
    return n, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types)


def test_gradient_host_checks(S):
    L = S.lib()

    def clip(ptrs=(16, 4096), numel=(8, 8), types=(0, 0), max_norm=1.0, eps=1e-6, norm=OK, ws=OK, ws_bytes=1 << 20):
        return L.s6_clip_grad_norm(*_grads(ptrs, numel, types), max_norm, eps, norm, ws, ws_bytes, None)

    def norm(ptrs=(16, 4096), numel=(8, 8), types=(0, 0), out=OK, ws=OK, ws_bytes=1 << 20):
        return L.s6_grad_norm(*_grads(ptrs, numel, types), out, ws, ws_bytes, None)
    for bad in (dict(numel=(8, -1)), dict(ptrs=(16, None)), dict(norm=None), dict(ws=None), dict(ws_bytes=64),
                dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")), dict(eps=-1.0),
                dict(eps=float("inf")),
                dict(ptrs=(16, 16)), dict(ptrs=(16, 44)), dict(ptrs=(44, 16)),       # the same memory twice
                dict(ptrs=(16, 28), types=(1, 0))):
        assert clip(**bad) == S.S6_ERR_INVALID_ARG, bad
    for bad in (dict(types=(0, 2)), dict(numel=(8, 1 << 38))):
        assert clip(**bad) == S.S6_ERR_UNSUPPORTED, bad
        assert norm(**bad) == S.S6_ERR_UNSUPPORTED, bad
    for bad in (dict(ptrs=(18, 4096)), dict(ptrs=(17, 4096), types=(1, 0))):
        assert clip(**bad) == S.S6_ERR_ALIGNMENT, bad
    assert norm(out=None) == S.S6_ERR_INVALID_ARG
    assert norm(out=P(2)) == S.S6_ERR_ALIGNMENT
    assert norm(ws=P(4)) == S.S6_ERR_ALIGNMENT
    n, p, e, t = _grads((16,), (8,), (0,))
    assert L.s6_grad_clip(n, p, e, t, None, 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG
    assert L.s6_grad_clip(-1, p, e, t, OK, 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG
    assert L.s6_grad_clip(1, None, e, t, OK, 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG
    assert L.s6_grad_clip(0, None, None, None, OK, 1.0, 1e-6, None) == S.S6_OK  # nothing to scale
    assert L.s6_grad_workspace(-1, None) == S.S6_ERR_INVALID_ARG
    assert L.s6_grad_workspace(0, None) > 0


def test_binding_refuses_what_it_cannot_pass_on(S):
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        S.s6_layernorm_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        S.s6_layernorm_bwd(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        S.causal_conv1d_silu_bwd(x[None], torch.zeros(8, 4), x[None])
    for call in (lambda: S.s6_grad_norm([x]), lambda: S.s6_clip_grad_norm({"a": x}, 1.0),
                 lambda: S.s6_grad_clip([x], x, 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        S.s6_grad_norm([1.0])
