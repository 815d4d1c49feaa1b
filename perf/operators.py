"""The training-step operators around the selective scan, as cases to be timed and compared.

LayerNorm forward (with the residual add in front of it) and backward, the backward of the causal conv + SiLU, and
the clipping of all gradients by their global norm.  ``run`` computes each in its plain form (elementary torch
operations in float32) where ``own`` is false, and through this library where it is true.
"""
import math

import torch

own = False

EPS = 1e-5       # LayerNorm
CLIP_EPS = 1e-6  # added to the norm before the division
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the LayerNorm of one decode step: 256 sequences of the Mamba-mini width; latency counts
        {"name": "ln_fwd_256x384_f32", "op": "ln_fwd", "rows": 256, "width": 384, "x": "f32", "y": "f32", "add": False},
        # the long-sequence workload's tokens, float32 residual stream plus a bfloat16 branch
        {"name": "ln_fwd_add_131072x384_mixed", "op": "ln_fwd", "rows": 131072, "width": 384, "x": "f32", "y": "bf16",
         "add": True},
        # the wide workload's tokens at an odd width: no row but the first is aligned
        {"name": "ln_fwd_8191x2561_bf16", "op": "ln_fwd", "rows": 8191, "width": 2561, "x": "bf16", "y": "bf16",
         "add": False},
        # one Mamba-mini training batch (8 x 256 tokens)
        {"name": "ln_bwd_2048x384_f32", "op": "ln_bwd", "rows": 2048, "width": 384, "x": "f32", "y": "f32",
         "add": False},
        # the long-sequence workload, gradient of the residual stream added
        {"name": "ln_bwd_add_131072x384_mixed", "op": "ln_bwd", "rows": 131072, "width": 384, "x": "f32", "y": "bf16",
         "add": True},
        # the wide workload's tokens at half its inner width
        {"name": "ln_bwd_8192x2560_bf16", "op": "ln_bwd", "rows": 8192, "width": 2560, "x": "bf16", "y": "bf16",
         "add": False},
        # the Mamba-mini block's conv
        {"name": "conv_bwd_8x256x1536_f32", "op": "conv_bwd", "batch": 8, "len": 256, "d": 1536, "k": 4, "x": "f32",
         "g": "f32"},
        # the long-sequence workload's conv: bfloat16 input, the scan's float32 du as the gradient
        {"name": "conv_bwd_16x8192x1536_bf16", "op": "conv_bwd", "batch": 16, "len": 8192, "d": 1536, "k": 4,
         "x": "bf16", "g": "f32"},
        # ragged in every direction, three taps, rows that are not whole 16-byte units
        {"name": "conv_bwd_3x1021x1090_bf16_k3", "op": "conv_bwd", "batch": 3, "len": 1021, "d": 1090, "k": 3,
         "x": "bf16", "g": "bf16"},
        # one block's gradients while nothing has to be clipped: late in training, latency counts
        {"name": "clip_1x64_f32_below", "op": "clip", "layers": 1, "width": 64, "inner": 128, "state": 16, "rank": 4,
         "k": 4, "x": "f32", "clips": False},
        # all gradients of the six Mamba-mini blocks
        {"name": "clip_6x384_f32", "op": "clip", "layers": 6, "width": 384, "inner": 1536, "state": 16, "rank": 24,
         "k": 4, "x": "f32", "clips": True},
        # twelve blocks at the wide workload's inner width, matrices in bfloat16 and the rest in float32
        {"name": "clip_12x2560_mixed", "op": "clip", "layers": 12, "width": 2560, "inner": 5120, "state": 16,
         "rank": 160, "k": 4, "x": "bf16", "clips": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "conv_bwd", "clip"])
    if op in ("ln_fwd", "ln_bwd"):
        width = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            width = max(8, width // 8 * 8)
        rows = _log(rng, 1, min(131072, 131072 * 384 // width))
        x, y = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        return {"op": op, "rows": rows, "width": width, "x": x, "y": y, "add": rng.random() < 0.5}
    if op == "conv_bwd":
        d = _log(rng, 8, 5120)
        if rng.random() < 0.5:
            d = max(8, d // 8 * 8)
        batch = rng.randint(1, 16)
        length = _log(rng, 1, min(65536, 16 * 8192 * 1536 // (d * batch)))
        x, g = rng.choice([("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
        return {"op": op, "batch": batch, "len": length, "d": d, "k": rng.choice([2, 3, 4]), "x": x, "g": g}
    width = _log(rng, 16, 2048)
    return {"op": op, "layers": rng.randint(1, 12), "width": width, "inner": width * rng.choice([2, 4]),
            "state": rng.choice([4, 8, 16]), "rank": max(1, width // 16), "k": rng.choice([2, 3, 4]),
            "x": rng.choice(["f32", "bf16"]), "clips": rng.random() < 0.7}


def _shapes(c):
    """The parameters of one block and whether they are matrices (in the case's type) or small (float32)."""
    w, di, n, r = c["width"], c["inner"], c["state"], c["rank"]
    return [((w,), False), ((w,), False), ((2 * di, w), True), ((di, c["k"]), False), ((di,), False),
            ((r + 2 * n, di), True), ((di, r), True), ((di,), False), ((di, n), False), ((di,), False),
            ((w, di), True)]


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    c = dict(case)
    st = {"case": c}
    if c["op"] in ("ln_fwd", "ln_bwd"):
        m, w = c["rows"], c["width"]
        st["w"] = 1.0 + 0.1 * normal(w)
        st["b"] = 0.1 * normal(w)
        # a residual stream: channels of their own size and offset
        x = normal(m, w).mul_(torch.exp(0.5 * normal(w))).add_(0.3 * normal(w))
        st["x"] = x.to(DT[c["x"]])
        if c["op"] == "ln_fwd":
            st["r"] = normal(m, w, dtype=DT[c["y"]]) if c["add"] else None
        else:
            xs = st["x"].double()
            mean = xs.mean(-1)
            st["mean"] = mean.float()
            st["rstd"] = ((xs - mean[:, None]).square().mean(-1) + EPS).rsqrt().float()
            st["dy"] = normal(m, w, dtype=DT[c["y"]])
            st["ds"] = normal(m, w) if c["add"] else None
    elif c["op"] == "conv_bwd":
        shape = (c["batch"], c["len"], c["d"])
        bound = c["k"] ** -0.5
        st["x"] = normal(*shape, dtype=DT[c["x"]])
        st["dout"] = normal(*shape, dtype=DT[c["g"]])
        st["conv_w"] = (torch.rand(c["d"], c["k"], generator=gen, device="cuda") * 2 - 1) * bound
        st["conv_b"] = (torch.rand(c["d"], generator=gen, device="cuda") * 2 - 1) * bound
    else:
        # gradients as views of one flat buffer for each type, packed without gaps (a bucket of a data-parallel run)
        shapes = _shapes(c) * c["layers"]
        count = {"f32": 0, "bf16": 0}
        places, square = [], 0.0
        for i, (shape, matrix) in enumerate(shapes):
            t = c["x"] if matrix else "f32"
            n = math.prod(shape)
            scale = 10.0 ** (-4 + 2 * ((i * 7) % 11) / 10)
            places.append((t, count[t], shape, n, scale))
            count[t] += n
            square += n * scale * scale
        st["flat"] = [normal(n, dtype=DT[t]) for t, n in count.items() if n]
        by = dict(zip([t for t, n in count.items() if n], st["flat"]))
        st["grads"] = [by[t][at:at + n].view(shape) for t, at, shape, n, _ in places]
        for g, p in zip(st["grads"], places):
            g.mul_(p[4])
        st["max_norm"] = math.sqrt(square) * (0.37 if c["clips"] else 2.0)
    return st


def _next_max_norm(st):
    """The gradients are clipped in place and not made anew between passes: a bound that falls a little with every
    pass keeps each of them one that clips."""
    now = st["max_norm"]
    if st["case"]["clips"]:
        st["max_norm"] = now * 0.9999
    return now


# -------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    if own:
        return _own(c["op"], st)
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "conv_bwd": _conv_bwd, "clip": _clip}[c["op"]](st, c)


def _own(op, st):
    import selective_state_space_19_b200 as S
    if op == "ln_fwd":
        y, s, mean, rstd = S.s6_layernorm_fwd(st["x"], st["w"], st["b"], eps=EPS, r=st["r"],
                                              y_dtype=DT[st["case"]["y"]])
        return {"y": y, "s": s if st["r"] is not None else None, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        return S.s6_layernorm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["w"], ds=st["ds"])
    if op == "conv_bwd":
        return S.causal_conv1d_silu_bwd(st["x"], st["conv_w"], st["dout"], conv_b=st["conv_b"])
    norm = S.s6_clip_grad_norm(st["grads"], _next_max_norm(st), eps=CLIP_EPS)
    return {"norm": norm, "grads": st["flat"]}


def _ln_fwd(st, c):
    s = st["x"].float()
    if st["r"] is not None:
        s = s + st["r"].float()
    mean = s.mean(-1, keepdim=True)
    off = s - mean
    rstd = (off.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = (off * rstd * st["w"] + st["b"]).to(DT[c["y"]])
    return {"y": y, "s": s.to(DT[c["x"]]) if st["r"] is not None else None, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_bwd(st, c):
    dy = st["dy"].float()
    rstd = st["rstd"][:, None]
    xhat = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if st["ds"] is not None:
        dx = dx + st["ds"]
    return {"dx": dx, "dw": (dy * xhat).sum(0), "db": dy.sum(0)}


def _conv_bwd(st, c):
    x, g, w, k = st["x"].float(), st["dout"].float(), st["conv_w"], c["k"]
    n = c["len"]
    pad = torch.zeros(c["batch"], k - 1, c["d"], device=x.device)
    xp = torch.cat([pad, x], 1)
    v = sum(xp[:, i:i + n] * w[:, i] for i in range(k)) + st["conv_b"]
    p = 1.0 / (1.0 + torch.exp(-v))
    dv = g * p * (1.0 + v * (1.0 - p))
    dvp = torch.cat([dv, pad], 1)
    return {"dx": sum(dvp[:, k - 1 - i:k - 1 - i + n] * w[:, i] for i in range(k)),
            "dconv_w": torch.stack([(dv * xp[:, i:i + n]).sum((0, 1)) for i in range(k)], 1),
            "dconv_b": dv.sum((0, 1))}


def _clip(st, c):
    norm = torch.stack([g.float().square().sum() for g in st["grads"]]).sum().sqrt()
    scale = (_next_max_norm(st) / (norm + CLIP_EPS)).clamp(max=1.0)
    [g.mul_(scale) if g.dtype == torch.float32 else g.copy_(g.float() * scale) for g in st["grads"]]
    return {"norm": norm, "grads": st["flat"]}


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("ln_fwd", "ln_bwd"):
        n = c["rows"] * c["width"]
        sx, sy = SIZE[c["x"]], SIZE[c["y"]]
        if c["op"] == "ln_fwd":
            return {"bytes": n * (sx + sy) * (2 if c["add"] else 1) + 8 * c["rows"] + 8 * c["width"], "flops": 8 * n}
        return {"bytes": n * (sx + sy + (8 if c["add"] else 4)) + 8 * c["rows"] + 12 * c["width"], "flops": 14 * n}
    if c["op"] == "conv_bwd":
        n = c["batch"] * c["len"] * c["d"]
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["g"]] + 4) + 8 * c["d"] * (c["k"] + 1),
                "flops": n * (6 * c["k"] + 10)}
    total = sum(math.prod(s) * (SIZE[c["x"]] if m else 4) for s, m in _shapes(c)) * c["layers"]
    count = sum(math.prod(s) for s, _ in _shapes(c)) * c["layers"]
    # nothing has to be written where the norm is below the bound
    return {"bytes": total * (2 if c["clips"] else 1), "flops": count * (3 if c["clips"] else 2)}


# ------------------------------------------------------- the same in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "ln_fwd":
        s = st["x"].double()
        if c["add"]:
            s += st["r"].double()
        mean = torch.einsum("mw->m", s) / c["width"]
        var = torch.einsum("mw,mw->m", s, s) / c["width"] - mean * mean
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(st["b"].double(), (s - mean[:, None]) * st["w"].double(), rstd[:, None])
        return {"y": y, "s": s if c["add"] else None, "mean": mean, "rstd": rstd}
    if c["op"] == "ln_bwd":
        # the vector-Jacobian product of a row, with the projections onto the ones and onto xhat taken out of g
        dy, w = st["dy"].double(), float(c["width"])
        xhat = (st["x"].double() - st["mean"].double()[:, None]).mul_(st["rstd"].double()[:, None])
        dw, db = torch.einsum("mw,mw->w", dy, xhat), torch.einsum("mw->w", dy)
        g = dy * st["w"].double()
        along = torch.einsum("mw,mw->m", g, xhat) / w
        g -= torch.einsum("mw->m", g)[:, None] / w
        g -= along[:, None] * xhat
        g *= st["rstd"].double()[:, None]
        if c["add"]:
            g += st["ds"].double()
        return {"dx": g, "dw": dw, "db": db}
    if c["op"] == "conv_bwd":
        # sequence by sequence, by differentiating the forward's definition
        w = st["conv_w"].double().requires_grad_()
        b = st["conv_b"].double().requires_grad_()
        dx, dw, db = [], torch.zeros_like(w), torch.zeros_like(b)
        for x, g in zip(st["x"], st["dout"]):
            x = x.double().requires_grad_()
            pre = b + w[:, -1] * x
            for back in range(1, min(c["k"], c["len"])):
                late = torch.nn.functional.pad(x[:-back], (0, 0, back, 0))
                pre = pre + w[:, c["k"] - 1 - back] * late
            gx, gw, gb = torch.autograd.grad(pre * torch.sigmoid(pre), (x, w, b), g.double())
            dx.append(gx)
            dw += gw
            db += gb
        return {"dx": torch.stack(dx), "dconv_w": dw.detach(), "dconv_b": db.detach()}
    flat = [f.double() for f in st["flat"]]
    norm = torch.sqrt(sum(torch.dot(f, f) for f in flat))
    scale = min(1.0, st["max_norm"] / (norm.item() + CLIP_EPS))
    return {"norm": norm, "grads": [f * scale for f in flat]}
