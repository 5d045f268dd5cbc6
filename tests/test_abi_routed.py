"""Argument checks of the routed-field and distillation calls (no GPU):
everything wrong is refused before anything is launched."""
import ctypes as C

import pytest

import volume_rendering_amd as v
from volume_rendering_amd import _binding as B

P = C.c_void_p(256)   # never dereferenced by a refused call
ODD = C.c_void_p(258)


def _err(text=None):
    msg = v.lib().nerf_last_error().decode()
    assert text is None or text in msg, msg


def test_workspace_sizes():
    assert B.nerf_route_workspace_size(100, 2, 8) == 0  # one workgroup sorts it
    nb = -(-262144 * 2 // 4096)
    assert B.nerf_route_workspace_size(262144, 2, 8) == (nb + 1) * 9 * 4  # counts per workgroup, totals
    for bad in ((-1, 2, 8), (10, 0, 8), (10, 65, 8), (10, 2, 0), (10, 2, 4097), (1 << 31, 1, 8)):
        assert B.nerf_route_workspace_size(*bad) == 0
    assert B.nerf_distill_workspace_size(0, 100) == 0 and B.nerf_distill_workspace_size(10, 0) == 0
    assert B.nerf_distill_workspace_size(1, 100) == 0
    assert B.nerf_distill_workspace_size(1, 100000) > 0
    assert B.nerf_expert_linear_grad_workspace_size(-1, 8, 16, 16) == 0
    assert B.nerf_expert_linear_grad_workspace_size(100, 8, 0, 16) == 0
    # a partial sum per range of slots and one more per expert, each as large as a weight and a bias gradient
    assert B.nerf_expert_linear_grad_workspace_size(1 << 18, 8, 256, 256) % (257 * 256 * 4) == 0


def test_route_plan_refusals():
    f = v.lib().nerf_route_plan
    assert f(P, -1, 2, 8, P, P, P, None, 0, None) == 1
    assert f(P, 4, 0, 8, P, P, P, None, 0, None) == 1
    assert f(P, 4, 65, 8, P, P, P, None, 0, None) == 1
    assert f(P, 4, 2, 0, P, P, P, None, 0, None) == 1
    assert f(P, 4, 2, 4097, P, P, P, None, 0, None) == 2
    assert f(P, 1 << 30, 2, 8, P, P, P, None, 0, None) == 1
    _err("pairs")
    assert f(None, 4, 2, 8, P, P, P, None, 0, None) == 1
    assert f(P, 4, 2, 8, None, P, P, None, 0, None) == 1
    assert f(P, 4, 2, 8, P, None, P, None, 0, None) == 1
    assert f(P, 4, 2, 8, P, P, None, None, 0, None) == 1
    assert f(ODD, 4, 2, 8, P, P, P, None, 0, None) == 1
    _err("misaligned")
    need = B.nerf_route_workspace_size(1 << 20, 2, 8)
    assert f(P, 1 << 20, 2, 8, P, P, P, P, need - 1, None) == 3
    assert f(P, 1 << 20, 2, 8, P, P, P, C.c_void_p(264), need, None) == 1


def test_route_rows_refusals():
    L = v.lib()
    ok = dict(dtype=0, ld=0, n=4, k=2, d=8, E=3)
    bad = [dict(dtype=2), dict(ld=7), dict(ld=-8), dict(n=-1), dict(k=0), dict(d=0), dict(d=65537), dict(E=0)]
    for b in bad:
        a = dict(ok, **b)
        assert L.nerf_route_gather(P, a["dtype"], a["ld"], a["n"], a["k"], a["d"], a["E"], P, P, P, None) == 1, b
        assert L.nerf_route_combine(P, a["dtype"], a["n"], a["k"], a["d"], a["E"], P, P, P, P, a["ld"], None) == 1, b
        assert L.nerf_route_combine_grad(P, a["ld"], P, a["dtype"], a["n"], a["k"], a["d"], a["E"], P, P, P, P, P,
                                         None) == 1, b
    assert L.nerf_route_gather(None, 0, 0, 4, 2, 8, 3, P, P, P, None) == 1
    assert L.nerf_route_gather(P, 0, 0, 4, 2, 8, 3, None, P, P, None) == 1
    assert L.nerf_route_gather(P, 0, 0, 4, 2, 8, 3, P, P, None, None) == 1
    assert L.nerf_route_gather(ODD, 0, 0, 4, 2, 8, 3, P, P, P, None) == 1
    assert L.nerf_route_combine(None, 0, 4, 2, 8, 3, P, P, P, P, 0, None) == 1
    assert L.nerf_route_combine_grad(None, 0, P, 0, 4, 2, 8, 3, P, P, P, P, P, None) == 1
    # no samples: nothing to do
    assert L.nerf_route_gather(None, 0, 0, 0, 2, 8, 3, None, None, None, None) == 0
    assert L.nerf_route_combine(None, 1, 0, 2, 8, 3, None, None, None, None, 0, None) == 0
    assert L.nerf_route_combine_grad(None, 0, None, 1, 0, 2, 8, 3, None, None, None, None, None, None) == 0


def _layer(**kw):
    d = dict(dtype=0, n_experts=4, d_in=16, d_out=8, relu=0, k=2, x_rows=32, ld_x=0, ld_y=0)
    d.update(kw)
    return C.byref(B.nerf_expert_layer(*[d[f] for f, _ in B.nerf_expert_layer._fields_]))


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(n_experts=0), dict(d_in=0), dict(d_out=65537), dict(ld_x=15),
                                 dict(ld_y=7), dict(k=0), dict(x_rows=-1)])
def test_expert_layer_refusals(bad):
    L = v.lib()
    assert L.nerf_expert_linear(_layer(**bad), P, P, None, P, P, 32, P, None) == 1
    assert L.nerf_expert_linear_grad(_layer(**bad), P, P, P, P, P, 32, P, P, P, None, 0, None) == 1


def test_expert_call_refusals():
    L = v.lib()
    f, g = L.nerf_expert_linear, L.nerf_expert_linear_grad
    assert f(None, P, P, None, P, None, 32, P, None) == 1
    assert f(_layer(n_experts=4097), P, P, None, P, None, 32, P, None) == 2
    assert f(_layer(x_rows=1 << 31, d_out=65536), P, P, None, P, None, (1 << 31) - 1, P, None) == 2
    assert f(_layer(), P, P, None, P, None, -1, P, None) == 1
    assert f(_layer(), P, P, None, P, None, 33, P, None) == 1  # fewer rows of x than slots
    _err("rows")
    for i in range(4):
        a = [P, P, P, P]
        a[i] = None
        assert f(_layer(), a[0], a[1], None, a[2], None, 32, a[3], None) == 1
    assert f(_layer(), ODD, P, None, P, None, 32, P, None) == 1
    assert f(_layer(), None, None, None, None, None, 0, None, None) == 0  # no slots
    assert g(_layer(), P, P, P, P, None, 32, None, None, None, None, 0, None) == 1  # nothing asked for
    assert g(_layer(), P, P, P, P, None, 32, P, None, P, None, 0, None) == 1        # dbias without dweights
    assert g(_layer(), None, P, P, P, None, 32, P, P, None, None, 0, None) == 1
    assert g(_layer(), P, None, P, P, None, 32, P, P, None, None, 0, None) == 1
    assert g(_layer(relu=1), P, None, P, P, None, 32, P, None, None, None, 0, None) == 1  # the mask needs x
    assert g(_layer(), P, P, None, P, None, 32, P, P, None, None, 0, None) == 1
    need = B.nerf_expert_linear_grad_workspace_size(1 << 18, 4, 16, 8)
    assert need > 0
    assert g(_layer(x_rows=1 << 18), P, P, P, P, None, 1 << 18, P, P, P, P, need - 1, None) == 3


def test_distill_refusals():
    L = v.lib()

    def f(logits=P, dtype=0, ld=0, n=4, V=100, t=P, ids=P, top=8, T=1.0, loss=P, grad=C.c_void_p(512), ld_g=0):
        return L.nerf_distill_topk(logits, dtype, ld, n, V, t, ids, top, T, None, loss, None, grad, ld_g, None, 0, None)

    def g(logits=P, dtype=0, ld=0, n=4, V=100, t=P, ids=P, top=8, T=1.0, loss=P, grad=C.c_void_p(512), ld_g=0):
        return L.nerf_distill_topk_grad(logits, dtype, ld, n, V, t, ids, top, T, None, loss, grad, ld_g, None)

    for h in (f, g):
        for bad in (dict(dtype=7), dict(ld=99), dict(n=-1), dict(V=0), dict(top=0), dict(top=257), dict(T=0.0),
                    dict(T=-1.0), dict(T=float("inf")), dict(T=float("nan")), dict(logits=None), dict(t=None),
                    dict(ids=None), dict(loss=None), dict(grad=P), dict(ld_g=50), dict(logits=ODD)):
            assert h(**bad) == 1, bad
        assert h(n=1 << 30, V=4096) == 2
        assert h(n=0, logits=None) == 0
    assert g(grad=None) == 1
    need = B.nerf_distill_workspace_size(1, 100000)
    assert L.nerf_distill_topk(P, 0, 0, 1, 100000, P, P, 8, 1.0, None, P, None, None, 0, P, need - 1, None) == 3


def test_binding_refuses_wrong_tensors():
    import torch
    i32 = torch.int32
    with pytest.raises(v.NerfError, match="dtype"):
        v.nerf_route_plan(torch.zeros(4, 2), 3, torch.zeros(4, dtype=i32), torch.zeros(8, dtype=i32),
                          torch.zeros(4, 2, dtype=i32))
    with pytest.raises(v.NerfError, match="not a device tensor"):
        v.nerf_route_plan(torch.zeros(4, 2, dtype=i32), 3, torch.zeros(4, dtype=i32), torch.zeros(8, dtype=i32),
                          torch.zeros(4, 2, dtype=i32))
    with pytest.raises(v.NerfError, match="shape|dimensions"):
        v.nerf_expert_linear(torch.zeros(4, 8), torch.zeros(3, 5, 9), None, torch.zeros(4, dtype=i32),
                             torch.zeros(4, 5))
