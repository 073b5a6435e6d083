"""Argument errors of the expert selection and the low-rank adapters, reported
before anything is launched (no GPU: aligned fake pointers), and the binding's
own checks."""
import ctypes

import pytest

P = 0x10000      # a fake, aligned device pointer: never read
OK, NULL, SHAPE, ALIGN, WORKSPACE, FORMAT = 0, -1, -2, -4, -5, -8


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    return lbq


def _router(L, **kw):
    d = dict(E=64, top_k=4, score=1, groups=8, top_groups=2, group_picks=2, renormalise=1, scale=1.0)
    d.update(kw)
    return ctypes.byref(L.Router(*d.values()))


BAD_ROUTERS = [dict(E=0), dict(E=1025, groups=1, top_groups=1), dict(top_k=0), dict(top_k=33, top_groups=8), dict(top_k=17),
               dict(E=4, top_k=5, groups=1, top_groups=1), dict(groups=0), dict(groups=7), dict(top_groups=0),
               dict(top_groups=9), dict(group_picks=0), dict(group_picks=3)]


@pytest.mark.parametrize("kw", BAD_ROUTERS)
def test_router_shapes(L, kw):
    lib = L.lib()
    assert lib.lbq_moe_select(_router(L, **kw), P, 0, 4, P, P, P, None) == SHAPE
    assert lib.lbq_moe_select_backward(_router(L, **kw), P, P, 0, P, 4, P, None) == SHAPE


def test_select_refusals(L):
    lib, r = L.lib(), _router(L)
    f, b = lib.lbq_moe_select, lib.lbq_moe_select_backward
    assert f(None, P, 0, 4, P, P, P, None) == NULL
    assert f(r, P, 0, -1, P, P, P, None) == SHAPE
    assert f(r, P, 0, 2 ** 22 + 1, P, P, P, None) == SHAPE
    for score in (-1, 2):
        assert f(_router(L, score=score), P, 0, 4, P, P, P, None) == FORMAT
    for dtype in (-1, 3):
        assert f(r, P, dtype, 4, P, P, P, None) == FORMAT
        assert b(r, P, P, dtype, P, 4, P, None) == FORMAT
    for args in ((None, 0, 4, P, P, P), (P, 0, 4, P, None, P), (P, 0, 4, P, P, None)):
        assert f(r, *args, None) == NULL
    for args in ((P + 4, 0, 4, P, P, P), (P, 0, 4, P + 2, P, P), (P, 0, 4, P, P + 2, P), (P, 0, 4, P, P, P + 2)):
        assert f(r, *args, None) == ALIGN
    assert f(r, None, 0, 0, None, None, None, None) == OK          # nothing to do
    for args in ((None, P, 0, P, 4, P), (P, None, 0, P, 4, P), (P, P, 0, None, 4, P), (P, P, 0, P, 4, None)):
        assert b(r, *args, None) == NULL
    for args in ((P + 2, P, 0, P, 4, P), (P, P + 8, 0, P, 4, P), (P, P, 0, P + 1, 4, P), (P, P, 0, P, 4, P + 4)):
        assert b(r, *args, None) == ALIGN
    assert b(r, None, None, 0, None, 0, None, None) == OK


def _ad(lbq, **kw):
    d = dict(L=4, K=256, N=100, r=8, dtype=0, a=P, b=P, scales=P)
    d.update(kw)
    return ctypes.byref(lbq.AdaptersView(*d.values()))


BAD_ADAPTERS = [dict(L=0), dict(L=1025), dict(K=0), dict(K=100), dict(K=2 ** 24 + 128), dict(N=0), dict(N=2 ** 24 + 1),
                dict(r=0), dict(r=129)]


def _forward(L, ad, x=P, M=4, ids=P, off=P, perm=P, base=P, y=P, h=P, ws=P, size=1 << 40):
    return L.lib().lbq_adapters_forward(ad, x, M, ids, off, perm, base, y, h, ws, size, None)


def _backward(L, ad, dy=P, x=P, h=P, M=4, ids=P, off=P, perm=P, base=P, dx=P, da=P, db=P, ws=P, size=1 << 40):
    return L.lib().lbq_adapters_backward(ad, dy, x, h, M, ids, off, perm, base, dx, da, db, ws, size, None)


@pytest.mark.parametrize("kw", BAD_ADAPTERS)
def test_adapter_shapes(L, kw):
    n = ctypes.c_size_t()
    assert _forward(L, _ad(L, **kw)) == SHAPE and _backward(L, _ad(L, **kw)) == SHAPE
    for q in (L.lib().lbq_adapters_workspace, L.lib().lbq_adapters_backward_workspace):
        assert q(_ad(L, **kw), 4, 1, ctypes.byref(n)) == SHAPE


def test_adapter_refusals(L):
    n, ad = ctypes.c_size_t(), _ad(L)
    for call in (_forward, _backward):
        assert call(L, None) == NULL
        for M in (-1, 2 ** 20 + 1):
            assert call(L, ad, M=M) == SHAPE
        for dtype in (-1, 2, 3):
            assert call(L, _ad(L, dtype=dtype)) == FORMAT
        for name in ("a", "b", "scales"):
            assert call(L, _ad(L, **{name: None})) == NULL
            assert call(L, _ad(L, **{name: P + 2})) == ALIGN
        for name in ("x", "ids", "off", "perm"):                 # an order is both or neither
            assert call(L, ad, **{name: None}) == NULL
        for name in ("x", "base", "h", "ids", "off", "perm", "ws"):
            assert call(L, ad, **{name: P + 1}) == ALIGN
    assert _forward(L, ad, y=None) == NULL and _forward(L, ad, y=P + 8) == ALIGN
    for name in ("dy", "h", "dx", "da", "db"):
        assert _backward(L, ad, **{name: None}) == NULL
        assert _backward(L, ad, **{name: P + 1}) == ALIGN
    for q, call in ((L.lib().lbq_adapters_workspace, _forward), (L.lib().lbq_adapters_backward_workspace, _backward)):
        assert q(ad, 4, 1, None) == NULL and q(None, 4, 1, ctypes.byref(n)) == NULL
        assert q(ad, -1, 1, ctypes.byref(n)) == SHAPE
        for M, order in ((4, P), (4, None), (3000, P), (3000, None)):
            assert q(ad, M, order is not None, ctypes.byref(n)) == OK
            if n.value:
                assert call(L, ad, M=M, off=order, perm=order, size=n.value - 1) == WORKSPACE
                assert call(L, ad, M=M, off=order, perm=order, ws=None) == NULL
    assert _forward(L, ad, x=None, M=0, ids=None, off=None, perm=None, base=None, y=None, h=None, ws=None, size=0) == OK


def test_binding_refuses_cpu_tensors_and_shapes(L):
    import torch

    with pytest.raises(L.LbqError):
        L.moe_select(torch.zeros(4, 8), 2)
    with pytest.raises(L.LbqError):
        L.moe_select_backward(torch.zeros(4, 2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(L.LbqError):
        L.Adapters(torch.zeros(2, 4, 128).half(), torch.zeros(2, 16, 4).half(), torch.ones(2))
    with pytest.raises(L.LbqError):
        L.Adapters(torch.zeros(4, 128).half(), torch.zeros(2, 16, 4).half(), torch.ones(2))
    with pytest.raises(L.LbqError):
        L.moe_select(torch.zeros(4, 8), 2 ** 40)


def test_router_holds_what_its_arguments_are_now(L):
    """A tensor or array as scale or switch that changes in place between calls, and settings that are equal as keys."""
    import numpy as np
    import torch

    for of in (torch.tensor, np.array):
        scale, k, on = of(2.0), of(4), of(True)
        for v in ((2.0, 4, True), (3.0, 5, False), (2.0, 4, True)):
            scale[()], k[()], on[()] = v
            s = L._router(64, k, 1, 8, 2, 2, on, scale)._obj
            assert (s.scale, s.top_k, s.renormalise) == v
    assert L._router(64, 4, 1, 8, 2, 2, 2, 1)._obj.renormalise == 1
    with pytest.raises(TypeError):
        L._router(64, 4.5, 1, 8, 2, 2, True, 1.0)


def test_no_tokens_take_the_workspace_of_the_query(L):
    """M = 0: the gradients ask for what their query names (the call itself, with zeros to write, needs a GPU)."""
    n, ad = ctypes.c_size_t(), _ad(L)
    q = L.lib().lbq_adapters_backward_workspace
    assert q(ad, 0, 1, ctypes.byref(n)) == OK and n.value == 0
    assert q(ad, 0, 0, ctypes.byref(n)) == OK and n.value > 0
    assert _backward(L, ad, M=0, off=None, perm=None, size=n.value - 1) == WORKSPACE
    assert _backward(L, ad, M=0, off=None, perm=None, ws=None) == NULL
    for name in ("da", "db"):
        assert _backward(L, ad, M=0, **{name: None}) == NULL
