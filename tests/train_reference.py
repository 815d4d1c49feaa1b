"""The training-step operators in float64 numpy, with bounds on what a float32
evaluation may be off by.

A float32 operation is off by at most u = 2^-24 of its result, a sum of n terms
by at most (its depth) u of the sum of the terms' magnitudes.  DEPTH bounds the
depth of the kernels' sums at the sizes tested here: at most 40 additions in a
thread's registers, 5 across a warp, 16 across the warps of a block, and in
the parameter sums 16 + 8 more over the blocks.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # largest relative rounding error of a stored value
DEPTH = 96


def ln_fwd(x, w, b, eps, r=None):
    """y, s, mean, rstd and the bounds of y (before its rounding), mean, rstd."""
    s = x if r is None else x + r
    mean = s.mean(-1, keepdims=True)
    off = s - mean
    rstd = 1.0 / np.sqrt((off ** 2).mean(-1, keepdims=True) + eps)
    h = off * rstd
    y = h * w + b
    size = np.abs(s).max(-1, keepdims=True)
    e_mean = U * (DEPTH + 2) * np.abs(s).mean(-1, keepdims=True)
    # an error e in every deviation changes the variance by at most 2 e sigma + e^2 of it
    e_off = U * size + U * np.abs(off) + e_mean
    rel = (e_off.max(-1, keepdims=True)) * rstd
    e_rstd = rstd * (0.5 * U * (DEPTH + 4) + rel + rel ** 2 + 2 * U)
    e_y = np.abs(w) * (e_off * rstd + np.abs(off) * e_rstd + 2 * U * np.abs(h)) + U * (np.abs(y) + np.abs(h * w))
    return dict(y=y, s=s, mean=mean[..., 0], rstd=rstd[..., 0]), dict(y=e_y, mean=e_mean[..., 0], rstd=e_rstd[..., 0])


def ln_bwd(dy, x, mean, rstd, w, ds=None):
    mean, rstd = mean[:, None], rstd[:, None]
    h = (x - mean) * rstd
    g = dy * w
    c0, c1 = g.mean(-1, keepdims=True), (g * h).mean(-1, keepdims=True)
    dx = rstd * (g - c0 - h * c1)
    e_h = U * (np.abs(x - mean) * rstd + 2 * np.abs(h))
    e_c0 = U * (DEPTH + 3) * np.abs(g).mean(-1, keepdims=True)
    e_c1 = U * (DEPTH + 3) * np.abs(g * h).mean(-1, keepdims=True) + (np.abs(g) * e_h).mean(-1, keepdims=True)
    e_dx = rstd * (2 * U * np.abs(g) + e_c0 + np.abs(h) * e_c1 + np.abs(c1) * e_h
                   + 3 * U * (np.abs(g) + np.abs(c0) + np.abs(h * c1))) + U * np.abs(dx)
    if ds is not None:
        dx = dx + ds
        e_dx = e_dx + U * np.abs(dx)
    dw, db = (dy * h).sum(0), dy.sum(0)
    e_dw = U * DEPTH * np.abs(dy * h).sum(0) + (np.abs(dy) * e_h).sum(0)
    e_db = U * DEPTH * np.abs(dy).sum(0)
    return dict(dx=dx, dw=dw, db=db), dict(dx=e_dx, dw=e_dw, db=e_db)


def conv_fwd(x, w, b):
    """SiLU of the causal conv of x [Bt, L, d] with taps w [d, K], oldest first."""
    v = conv_pre(x, w, b)
    return v / (1.0 + np.exp(-v))


def conv_pre(x, w, b):
    Bt, L, d = x.shape
    v = np.zeros_like(x) + (0.0 if b is None else b)
    K = w.shape[1]
    for k in range(K):
        back = K - 1 - k
        if back < L:
            v[:, back:] += w[:, k] * x[:, :L - back]
    return v


def conv_bwd(x, w, b, g):
    """dx, dconv_w, dconv_b and their bounds.  p = 1/(1+e^-v) through a power and a
    reciprocal of 2^-22 relative error each, and an argument off by U |v|: p is off by
    (9 + 2 |v|) U of itself."""
    Bt, L, d = x.shape
    K = w.shape[1]
    v = conv_pre(x, w, b)
    e_v = U * (K + 1) * (conv_pre(np.abs(x), np.abs(w), None) + (0.0 if b is None else np.abs(b)))
    p = 1.0 / (1.0 + np.exp(-v))
    f = p * (1.0 + v * (1.0 - p))
    e_p = U * (9 + 2 * np.abs(v)) * p
    # the factor's own second derivative in v is at most 1/2 in magnitude
    e_f = 0.5 * e_v + e_p * (1.0 + np.abs(v)) + U * (2 * np.abs(f) + 3 * p * (1 + np.abs(v)))
    dv, e_dv = g * f, np.abs(g) * e_f + U * np.abs(g * f)
    dx, mag, e_dx = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    dw, e_dw = np.zeros((d, K)), np.zeros((d, K))
    for k in range(K):
        back = K - 1 - k
        if back >= L:
            continue
        dx[:, :L - back] += w[:, k] * dv[:, back:]
        mag[:, :L - back] += np.abs(w[:, k] * dv[:, back:])
        e_dx[:, :L - back] += np.abs(w[:, k]) * e_dv[:, back:]
        xs = x[:, :L - back]
        dw[:, k] = (dv[:, back:] * xs).sum((0, 1))
        e_dw[:, k] = (U * DEPTH * np.abs(dv[:, back:] * xs) + e_dv[:, back:] * np.abs(xs)).sum((0, 1))
    return (dict(dx=dx, dconv_w=dw, dconv_b=dv.sum((0, 1))),
            dict(dx=e_dx + U * K * mag, dconv_w=e_dw, dconv_b=(U * DEPTH * np.abs(dv) + e_dv).sum((0, 1))))


def grad_norm(grads):
    return np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))


# The norm: squares and the sums of 8 of them in float32 (5 u of the sum, half of that of its root), float64 from
# there, one rounding at the end.  The scale: its sum with eps, the division, and the norm's own error.
NORM_REL = 4 * U
SCALED_REL = NORM_REL + 3 * U


def within(got, ref, tol, what=""):
    """Every element finite and within tol; returns the largest error as a share of its bound."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == np.shape(ref), (what, got.shape, np.shape(ref))
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    if got.size == 0:
        return 0.0
    tol = np.broadcast_to(tol, got.shape) + 1e-37
    share = float(np.max(np.abs(got - ref) / tol))
    assert share <= 1.0, f"{what}: {share:.3g} of the bound, at {np.unravel_index(np.argmax(np.abs(got - ref) / tol), got.shape)}"
    return share
