"""CPU checks of the training-step operators' edges: what is refused before a device
is touched, and how the two libraries are built."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def S():
    from selective_state_space_19_b200 import _build
    import selective_state_space_19_b200 as S
    _build.build()
    S.lib()
    return S


P = ctypes.c_void_p


def _grads(ptrs, numel, types):
    n = len(ptrs)
    return n, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types)


def test_a_norm_inside_a_gradient_is_refused(S):
    L = S.lib()
    for types in ((0, 0), (1, 1), (0, 1)):
        size = [2 if t else 4 for t in types]
        g = _grads((4096, 8192), (8, 100), types)
        for at in (4096, 4096 + 8 * size[0] - 4, 8192, 8192 + 100 * size[1] - 4):
            assert L.s6_grad_clip(*g, P(at), 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG, (types, at)
            assert L.s6_clip_grad_norm(*g, 1.0, 1e-6, P(at), P(1 << 20), 1 << 20, None) == S.S6_ERR_INVALID_ARG, (types, at)
    # half of the norm's bytes in a bfloat16 tensor of an odd length
    g = _grads((4096,), (3,), (1,))
    assert L.s6_grad_clip(*g, P(4100), 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG
    g = _grads((4098,), (3,), (1,))
    assert L.s6_grad_clip(*g, P(4096), 1.0, 1e-6, None) == S.S6_ERR_INVALID_ARG


def test_a_list_too_long_for_the_hosts_memory_says_so(S):
    """16.7 million tensors want 268 MB for the check that no two overlap: under a limit of the
    address space the call returns a status of its own."""
    import subprocess
    import sys
    code = """
import ctypes, resource, sys
import numpy as np
L = ctypes.CDLL(sys.argv[1])
n = 1 << 24
ptrs = np.arange(1, n + 1, dtype=np.uint64) * 64
numel, types = np.ones(n, np.int64), np.zeros(n, np.int32)
L.s6_grad_clip.argtypes = [ctypes.c_int64] + [ctypes.c_void_p] * 4 + [ctypes.c_float] * 2 + [ctypes.c_void_p]
L.s6_status_string.restype = ctypes.c_char_p
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (128 << 20), resource.RLIM_INFINITY))
st = L.s6_grad_clip(n, ptrs.ctypes.data, numel.ctypes.data, types.ctypes.data, 16, -1.0, 1e-6, None)  # refused in any case
assert st == int(sys.argv[2]), st
assert L.s6_status_string(st).startswith(b"S6_ERR_HOST_MEMORY")
"""
    out = subprocess.run([sys.executable, "-c", code, S.LIB_PATH, str(S.S6_ERR_HOST_MEMORY)], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-2000:]


BASE = 1 << 20


def test_layernorm_forward_refuses_outputs_that_overlap(S):
    """16 rows of 64 (4 KB in float32) at addresses a megabyte apart, but for the one that is moved."""
    at = {k: BASE * (i + 1) for i, k in enumerate(("x", "r", "w", "b", "s", "y", "mean", "rstd"))}
    size = dict(x=4096, r=4096, w=256, b=256, s=4096, y=4096, mean=64, rstd=64)
    dims = S.NormDims(16, 64, S.S6_F32, S.S6_F32, 1e-5)

    def status(**moved):
        p = dict(at, **moved)
        return S.lib().s6_layernorm_fwd(ctypes.byref(dims), P(p["x"]), P(p["r"]), P(p["w"]), P(p["b"]), P(p["s"]),
                                        P(p["y"]), P(p["mean"]), P(p["rstd"]), None)
    for out in ("s", "y", "mean", "rstd"):
        for other in set(at) - {out}:
            for by in (-size[out] + 4, size[other] - 4) + (() if other in "xr" and out in "sy" else (0,)):
                assert status(**{out: at[other] + by}) == S.S6_ERR_INVALID_ARG, (out, other, by)
    assert status(s=at["x"], y=at["x"]) == S.S6_ERR_INVALID_ARG  # both outputs in the stream
    # rows and widths whose product passes 64 bits
    dims = S.NormDims(1 << 40, 1 << 24, S.S6_F32, S.S6_F32, 1e-5)
    assert status() == S.S6_ERR_INVALID_ARG


def test_layernorm_backward_refuses_outputs_that_overlap(S):
    names = ("x", "mean", "rstd", "w", "dy", "ds", "dx", "dw", "db", "ws")
    at = {k: BASE * (i + 1) for i, k in enumerate(names)}
    dims = S.NormDims(16, 64, S.S6_F32, S.S6_F32, 0.0)
    ws = S.lib().s6_layernorm_bwd_workspace(ctypes.byref(dims))
    size = dict(x=4096, mean=64, rstd=64, w=256, dy=4096, ds=4096, dx=4096, dw=256, db=256, ws=ws)

    def status(**moved):
        p = dict(at, **moved)
        return S.lib().s6_layernorm_bwd(ctypes.byref(dims), *(P(p[k]) for k in names), ws, None)
    for out in ("dx", "dw", "db", "ws"):
        for other in set(at) - {out}:
            for by in (-size[out] + 8, size[other] - 8) + (() if (out, other) in (("dx", "x"), ("dx", "dy"), ("dx", "ds")) else (0,)):
                assert status(**{out: at[other] + by}) == S.S6_ERR_INVALID_ARG, (out, other, by)


def test_conv_backward_refuses_outputs_that_overlap(S):
    names = ("x", "w", "b", "g", "dx", "dw", "db", "ws")
    at = {k: BASE * (i + 1) for i, k in enumerate(names)}
    dims = S.Dims(2, 8, 64, 1, 4, 0)
    ws = S.lib().causal_conv1d_silu_bwd_workspace(ctypes.byref(dims))
    size = dict(x=4096, w=1024, b=256, g=4096, dx=4096, dw=1024, db=256, ws=ws)

    def status(**moved):
        p = {k: P(v) for k, v in dict(at, **moved).items()}
        return S.lib().causal_conv1d_silu_bwd(ctypes.byref(dims), p["x"], p["w"], p["b"], p["g"], 0, p["dx"], p["dw"],
                                              p["db"], p["ws"], ws, None)
    assert ws < BASE
    for out in ("dx", "dw", "db", "ws"):
        for other in set(at) - {out}:
            for by in (-size[out] + 8, 0, size[other] - 8):
                assert status(**{out: at[other] + by}) == S.S6_ERR_INVALID_ARG, (out, other, by)


# -------------------------------------------------------------------- build
@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build on a small source tree, with compilers that write down what they are asked for
    (and fail on a source that holds the word broken)."""
    from selective_state_space_19_b200 import _build
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "s6_torch.cpp"):
        (csrc / name).write_text("// " + name + "\n")
    log = tmp_path / "log"
    for name in ("nvcc", "cxx"):
        tool = tmp_path / name
        tool.write_text('#!/bin/sh\necho %s "$@" >> %s\nfor a; do case "$a" in *.cu|*.cpp) grep -q broken "$a" && exit 1;; esac; '
                        '[ "$last" = -o ] && : > "$a"; last="$a"; done; exit 0\n' % (name, log))
        tool.chmod(0o755)
    for k, v in dict(HERE=str(tmp_path), CSRC=str(csrc), OBJ=str(csrc / "obj"), LIB=str(tmp_path / "lib.so"),
                     MODULE=str(tmp_path / "_s6_torch.so"), CXX=str(tmp_path / "cxx")).items():
        monkeypatch.setattr(_build, k, v)
    monkeypatch.setattr(_build, "_nvcc", lambda: str(tmp_path / "nvcc"))

    def calls():
        lines = log.read_text().splitlines() if log.exists() else []
        log.write_text("")
        return sorted(l.split()[0] for l in lines)
    return _build, tmp_path, calls


def test_build_makes_both_and_then_nothing(tree):
    B, at, calls = tree
    B.build()
    assert calls() == ["cxx", "cxx", "nvcc", "nvcc"] and (at / "lib.so").exists() and (at / "_s6_torch.so").exists()
    assert B.up_to_date()
    B.build()
    assert calls() == []


def test_build_without_torch_makes_the_library(tree, monkeypatch, capsys):
    B, at, calls = tree
    monkeypatch.setattr(B, "_torch_dir", lambda: None)
    B.build()
    assert calls() == ["nvcc", "nvcc"] and (at / "lib.so").exists() and not (at / "_s6_torch.so").exists()
    assert "_s6_torch.so is not built" in capsys.readouterr().err
    assert B.up_to_date()
    monkeypatch.undo()


def test_build_makes_the_library_where_the_module_cannot_be_made(tree, monkeypatch):
    import subprocess
    B, at, calls = tree
    (at / "csrc" / "s6_torch.cpp").write_text("broken\n")
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert (at / "lib.so").exists() and not (at / "_s6_torch.so").exists() and not B.up_to_date()
    (at / "csrc" / "s6_torch.cpp").write_text("// mended\n")
    monkeypatch.setattr(B, "CXX", str(at / "no such compiler"))
    (at / "lib.so").unlink()
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert (at / "lib.so").exists() and not (at / "_s6_torch.so").exists()


def test_build_makes_the_module_again_for_another_torch(tree, monkeypatch):
    B, at, calls = tree
    B.build()
    calls()
    was = B._made_for()
    monkeypatch.setattr(B, "_made_for", lambda: was + " and a half")
    assert not B.up_to_date()
    B.build()
    assert calls() == ["cxx", "cxx", "nvcc"]  # the library is linked again, not compiled
    assert B.up_to_date()


def test_the_recorded_traffic_is_of_the_present_scan_kernel():
    """bench.py reports the DRAM bytes of the committed capture as long as the scan's sources are
    those it was taken on; an edit of them asks for another capture."""
    import bench
    traffic, sha = bench.recorded_traffic()
    assert sha == bench.kernel_source_sha() and traffic is not None and 1.4e9 < traffic < 1.7e9
