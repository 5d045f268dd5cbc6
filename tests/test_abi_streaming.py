"""Argument checks of the streaming-field calls (no GPU): everything wrong is
refused before anything is launched."""
import ctypes as C

import pytest
import torch

import volume_rendering_amd as v
from volume_rendering_amd import _binding as B

P, Q = C.c_void_p(256), C.c_void_p(4096)   # never dereferenced by a refused call
ODD = C.c_void_p(257)
BIG = (1 << 31) - 1


def _err(text):
    msg = v.lib().nerf_last_error().decode()
    assert text in msg, msg


def test_gate_refusals():
    L = v.lib()

    def f(z=P, dtype=0, ld=0, n=4, E=16, k=2, ids=P, w=P, dz=Q):
        return L.nerf_route_gate(z, dtype, ld, n, E, k, 1, ids, w, None)

    def g(z=P, dtype=0, ld=0, n=4, E=16, k=2, ids=P, w=P, dz=Q, dw=P, ld_d=0, renorm=0):
        return L.nerf_route_gate_grad(dw, z, dtype, ld, n, E, k, renorm, ids, w, dz, ld_d, None)

    for h in (f, g):
        for bad in (dict(dtype=2), dict(ld=15), dict(ld=-16), dict(n=-1), dict(E=0), dict(k=0), dict(k=17), dict(k=65, E=100),
                    dict(n=1 << 30, k=2), dict(z=None), dict(ids=None), dict(w=None), dict(z=ODD), dict(ids=ODD),
                    dict(w=C.c_void_p(258))):
            assert h(**bad) == 1, bad
        assert h(E=4097) == 2
        assert h(n=0, z=None, ids=None, w=None) == 0
    for bad in (dict(dw=None), dict(dz=None), dict(dz=P), dict(ld_d=3), dict(dw=ODD), dict(dz=ODD)):
        assert g(**bad) == 1, bad
    _err("misaligned")


def _layer(**kw):
    d = dict(dtype=0, n_experts=4, d_in=16, hidden=8, d_out=5, act=1, k=2, ld_x=0, ld_out=0)
    d.update(kw)
    return C.byref(B.nerf_routed_layer(*[d[f] for f, _ in B.nerf_routed_layer._fields_]))


def test_routed_mlp_refusals():
    L = v.lib()
    f = L.nerf_routed_mlp
    for bad in (dict(dtype=3), dict(n_experts=0), dict(d_in=0), dict(hidden=0), dict(d_out=0), dict(d_in=65537),
                dict(hidden=65537), dict(act=3), dict(act=-1), dict(k=0), dict(k=65), dict(ld_x=15), dict(ld_out=4)):
        assert f(_layer(**bad), P, P, P, 4, P, P, P, P, Q, None, 0, None) == 1, bad
    assert f(None, P, P, P, 4, P, P, P, P, Q, None, 0, None) == 1
    assert f(_layer(n_experts=4097), P, P, P, 4, P, P, P, P, Q, None, 0, None) == 2
    assert f(_layer(), P, P, P, -1, P, P, P, P, Q, None, 0, None) == 1
    assert f(_layer(), P, P, P, 257, P, P, P, P, Q, None, 0, None) == 2
    _err("nerf_expert_linear")
    for i in (0, 1, 4, 6, 8):
        a = [P, P, P, 4, P, P, P, P, Q]
        a[i if i < 3 else i] = None
        assert f(_layer(), *a, None, 0, None) == 1, i
        a[i] = ODD
        assert f(_layer(), *a, None, 0, None) == 1, i
    assert f(_layer(), None, None, None, 0, None, None, None, None, None, None, 0, None) == 0
    need = B.nerf_routed_mlp_workspace_size(4, 2, 8, 5)
    assert need >= 4 * 2 * (8 + 5) * 4
    assert f(_layer(), P, P, P, 4, P, P, P, P, Q, P, need - 1, None) == 3
    assert f(_layer(), P, P, P, 4, P, P, P, P, Q, C.c_void_p(264), need, None) == 1
    for bad in ((0, 2, 8, 5), (4, 0, 8, 5), (257, 2, 8, 5), (4, 2, 0, 5), (4, 2, 8, 0), (1 << 40, 2, 8, 5)):
        assert B.nerf_routed_mlp_workspace_size(*bad) == 0


def _cfg(**kw):
    d = dict(dtype=0, gate_dtype=0, d=16, gates=16, reverse=0, mix=0, rows=64, n_seq=4, ld_a=0, ld_x=0, ld_h=0, ld_dh=0)
    d.update(kw)
    return C.byref(B.nerf_scan_cfg(*[d[f] for f, _ in B.nerf_scan_cfg._fields_]))


def test_scan_refusals():
    L = v.lib()
    R, S, T = C.c_void_p(8192), C.c_void_p(16384), C.c_void_p(32768)

    def f(cfg, a=P, x=Q, off=None, h0=None, h=R, last=None, ws=None, size=0):
        return L.nerf_scan(cfg, a, x, off, h0, h, last, ws, size, None)

    def g(cfg, a=P, x=Q, off=None, h0=None, h=R, last=None, ws=None, size=0, dh=C.c_void_p(1 << 16), da=S, dx=T):
        return L.nerf_scan_grad(cfg, dh, last, a, x, h, h0, off, da, dx, None, ws, size, None)

    for call in (f, g):
        for bad in (dict(dtype=2), dict(gate_dtype=-1), dict(d=0), dict(d=65537), dict(gates=0), dict(gates=17),
                    dict(gates=3), dict(rows=-1), dict(rows=BIG + 1), dict(n_seq=-1), dict(n_seq=BIG), dict(n_seq=5),
                    dict(ld_a=15), dict(ld_x=15), dict(ld_h=3)):
            assert call(_cfg(**bad)) == 1, bad
        assert call(None) == 1
        assert call(_cfg(gate_dtype=1)) == 2
        _err("bfloat16 gates")
        for bad in (dict(a=None), dict(h=None), dict(a=ODD), dict(x=ODD), dict(h=ODD), dict(off=ODD), dict(h0=ODD),
                    dict(last=ODD)):
            assert call(_cfg(), **bad) == 1, bad
        assert call(_cfg(n_seq=0)) == 0
    assert f(_cfg(), x=None) == 1 and f(_cfg(), h=Q) == 1 and f(_cfg(), h=P) == 1
    assert g(_cfg(mix=1), x=None) == 1 and g(_cfg(ld_dh=2)) == 1
    for bad in (dict(dh=None), dict(da=None), dict(dx=None), dict(da=P), dict(dx=R), dict(dx=S), dict(da=ODD), dict(dx=ODD)):
        assert g(_cfg(), **bad) == 1, bad
    need = B.nerf_scan_workspace_size(100000, 8)
    assert need > 0 and f(_cfg(rows=100000, n_seq=1, d=8, gates=8), ws=P, size=need // 100) == 3
    for bad in (dict(rows=-1, d=8), dict(rows=10, d=0), dict(rows=10, d=8, gates=3), dict(rows=10, d=8, n_seq=0)):
        assert B.nerf_scan_workspace_size(**bad) == 0
    assert B.nerf_scan_workspace_size(256, 1024, n_seq=256) == 0  # one step of many states needs none


def _list(*items):
    a = (B.nerf_tensor * max(1, len(items)))()
    for i, (src, dst, count, dtype) in enumerate(items):
        a[i] = B.nerf_tensor(src, dst, count, dtype, 0)
    return C.byref(a), len(items)


def test_gradient_list_refusals():
    L = v.lib()

    def norm(lst, n, out=P):
        return L.nerf_grad_norm(lst, n, out, None, 0, None)

    def clip(lst, n, out=P, most=1.0):
        return L.nerf_grad_clip(lst, n, most, out, None, 0, None)

    good = (1 << 20, 1 << 21, 100, 0)
    for call in (norm, clip):
        assert call(None, 1) == 1 and call(None, -1) == 1 and call(None, (1 << 20) + 1) == 1
        for bad in ((1 << 20, 1 << 21, 100, 2), (1 << 20, 1 << 21, -1, 0), (None, 1 << 21, 4, 0), (1026, 1 << 21, 4, 0),
                    (1025, 1 << 21, 4, 1), (1 << 20, 1 << 21, 1 << 42, 0)):
            assert call(*_list(good, bad)) == 1, bad
            _err("tensor 1")
        assert call(*_list(good), None) == 1 and call(*_list(good), ODD) == 1
    for bad in (float("nan"), -1.0):
        assert clip(*_list(good), P, bad) == 1
    assert clip(*_list((1 << 20, None, 4, 0))) == 1 and clip(*_list((1 << 20, 1025, 4, 0))) == 1
    # destinations overlap a tensor
    M = 1 << 20
    for items in ([(M, M, 100, 0), (M, M, 100, 0)], [(M, 2 * M, 100, 0), (3 * M, 2 * M + 396, 100, 0)],
                  [(M, M + 4, 100, 0)], [(M, 2 * M, 100, 0), (2 * M, 3 * M, 100, 0)], [(M, M, 100, 0), (M + 100, 5 * M, 4, 0)],
                  [(2 * M + 40 * i, 2 * M + 40 * i, 10, 0) for i in range(200)] + [(2 * M + 4, 2 * M + 4, 1, 0)]):
        assert clip(*_list(*items)) == 1, items
        _err("overlaps")
    size = B.nerf_grad_norm_workspace_size(v.nerf_tensor_list([]))
    assert size == 8  # (the norm itself)
    lst, n = _list(good)
    assert L.nerf_grad_norm_workspace_size(lst, n) == 16
    assert L.nerf_grad_clip(lst, n, 1.0, P, P, 15, None) == 3
    assert L.nerf_grad_norm_workspace_size(None, 3) == 0


def test_binding_refuses_wrong_tensors():
    z, i32 = torch.zeros, torch.int32
    for call, why in (
            (lambda: v.nerf_route_gate(z(4, 8), z(4, 2), z(4, 2)), "ids: dtype|not a device"),
            (lambda: v.nerf_route_gate(z(4, 8).half(), z(4, 2, dtype=i32), z(4, 2)), "float32 or bfloat16|not a device"),
            (lambda: v.nerf_route_gate(z(8), z(4, 2, dtype=i32), z(4, 2)), "dimensions"),
            (lambda: v.nerf_route_gate_grad(z(4, 2), None, z(4, 3, dtype=i32), z(4, 3), z(4, 8)), "shape|not a device"),
            (lambda: v.nerf_routed_mlp(z(2, 4), z(2, 1, dtype=i32), None, z(3, 5, 4), None, z(3, 6, 5), None, z(2, 6),
                                       act="tanh"), "act"),
            (lambda: v.nerf_routed_mlp(z(2, 4), z(2, 1, dtype=i32), None, z(5, 4), None, z(3, 6, 5), None, z(2, 6)),
             "dimensions"),
            (lambda: v.nerf_scan(z(4, 2), z(4, 6), z(4, 6)), "not a device tensor"),
            (lambda: v.nerf_scan(z(4), z(4, 6), z(4, 6)), "dimensions"),
            (lambda: v.nerf_scan_grad(z(4, 6), z(4, 2), None, z(4, 6), z(4, 2), z(4, 6)), "not a device tensor"),
            (lambda: v.nerf_tensor_list([z(3)]), "not a device tensor"),
            (lambda: v.nerf_tensor_list([z(3), z(4)], [z(3)]), "2 tensors, 1 outputs|not a device")):
        with pytest.raises(v.NerfError, match=why):
            call()
