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
