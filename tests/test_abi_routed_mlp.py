"""What the few-sample layer's refusal of too many pairs points to (no GPU)."""
import ctypes as C

import pytest

import volume_rendering_amd as v
from volume_rendering_amd import _binding as B


@pytest.mark.parametrize("act", sorted(B._ACTS))
def test_too_many_pairs(act):
    P = C.c_void_p(256)  # (never dereferenced by a refused call)
    layer = B.nerf_routed_layer(0, 4, 16, 8, 5, B._ACTS[act], 2, 0, 0)
    status = v.lib().nerf_routed_mlp(C.byref(layer), P, P, P, 257, P, P, P, P, C.c_void_p(4096), None, 0, None)
    msg = v.lib().nerf_last_error().decode()
    assert status == 2 and "257 x 2 pairs" in msg and "nerf_expert_linear" in msg
    assert ("no gated hidden layer" in msg) == (act == "gated")  # (nerf_expert_linear knows ReLU and none)
