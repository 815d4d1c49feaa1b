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
