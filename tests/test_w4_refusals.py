"""Host-side refusals of the 4-bit, router and expert entry points (CPU only: every
call is turned away before a device is touched)."""
import ctypes

import pytest
import torch

import fp8_linear_layers_b200 as ql
from fp8_linear_layers_b200 import build as qbuild

OK, INV, SHAPE, MIS = 0, 1, 2, 3
A = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return ql.lib()


def _w(**kw):
    f = dict(wq=A, sw=A, wz=0, experts=1, N=64, K=64, group=32)
    f.update(kw)
    w = ql._W4(*(f[n] for n in ("wq", "sw", "wz", "experts", "N", "K", "group")))
    return w, ctypes.addressof(w)


@pytest.mark.parametrize("change,want", [
    (dict(wq=0), INV), (dict(sw=0), INV), (dict(wq=A + 8), MIS), (dict(sw=A + 2), MIS), (dict(wz=A + 1), MIS),
    (dict(N=0), INV), (dict(K=0), INV), (dict(K=48), SHAPE), (dict(group=16), SHAPE), (dict(group=256), SHAPE),
    (dict(N=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE), (dict(experts=0), INV)])
def test_weight_shapes(L, change, want):
    w, p = _w(**change)
    assert L.qlinear_forward_w4(A, p, 4, A, None, 0, None) == want
    w, p = _w(**{"experts": 4, **change})
    assert L.qlinear_experts_w4(A, A, None, p, 4, 2, A, None, 0, None) == want


def test_forward_arguments(L):
    w, p = _w()
    assert L.qlinear_forward_w4(A, None, 4, A, None, 0, None) == INV
    assert L.qlinear_forward_w4(None, p, 4, A, None, 0, None) == INV
    assert L.qlinear_forward_w4(A + 2, p, 4, A, None, 0, None) == MIS
    assert L.qlinear_forward_w4(A, p, 4, None, None, 0, None) == INV
    assert L.qlinear_forward_w4(A, p, -1, A, None, 0, None) == INV
    assert L.qlinear_forward_w4(A, p, 1 << 31, A, None, 0, None) == SHAPE
    assert L.qlinear_forward_w4(None, p, 0, None, None, 0, None) == OK
    w, p = _w(experts=2)
    assert L.qlinear_forward_w4(A, p, 4, A, None, 0, None) == INV


def test_experts_arguments(L):
    w, p = _w(experts=8)
    call = L.qlinear_experts_w4
    assert call(None, A, None, p, 4, 2, A, None, 0, None) == INV
    assert call(A, None, None, p, 4, 2, A, None, 0, None) == INV
    assert call(A, A + 4, None, p, 4, 2, A, None, 0, None) == MIS
    assert call(A, A, A + 4, p, 4, 2, A, None, 0, None) == MIS
    assert call(A, A, None, p, 4, 0, A, None, 0, None) == INV
    assert call(A, A, None, p, 4, 33, A, None, 0, None) == INV
    assert call(A, A, None, p, -1, 2, A, None, 0, None) == INV
    assert call(None, None, None, p, 0, 2, None, None, 0, None) == OK
    w, p = _w(experts=1025)
    assert call(A, A, None, p, 4, 2, A, None, 0, None) == SHAPE


def _rc(**kw):
    f = dict(experts=64, top_k=8, groups=1, top_groups=1, group_top=1, score=0, renormalize=1, scale=1.0)
    f.update(kw)
    c = ql._RouteConfig(*f.values())
    return c, ctypes.addressof(c)


@pytest.mark.parametrize("change,want", [
    (dict(score=2), INV), (dict(top_k=0), INV), (dict(top_k=65), INV), (dict(top_k=33), INV), (dict(experts=0), INV),
    (dict(group_top=3), INV), (dict(experts=1025), SHAPE), (dict(groups=5), SHAPE), (dict(groups=64, top_groups=64), SHAPE),
    (dict(groups=8, top_groups=9), SHAPE), (dict(groups=8, top_groups=0), SHAPE), (dict(groups=0), INV),
    (dict(groups=16, top_groups=1), SHAPE), (dict(groups=32, top_groups=32, group_top=2, experts=32), SHAPE)])
def test_route_config(L, change, want):
    c, p = _rc(**change)
    assert L.qlinear_route(A, 0, p, None, 4, A, A, None) == want


def test_route_arguments(L):
    c, p = _rc()
    assert L.qlinear_route(A, 0, None, None, 4, A, A, None) == INV
    assert L.qlinear_route(None, 0, p, None, 4, A, A, None) == INV
    assert L.qlinear_route(A + 4, 0, p, None, 4, A, A, None) == MIS
    assert L.qlinear_route(A, 0, p, A + 4, 4, A, A, None) == MIS
    assert L.qlinear_route(A, 0, p, None, 4, None, A, None) == INV
    assert L.qlinear_route(A, 0, p, None, 4, A, None, None) == INV
    assert L.qlinear_route(A, 0, p, None, -1, A, A, None) == INV
    assert L.qlinear_route(None, 0, p, None, 0, None, None, None) == OK


def test_quantize_arguments(L):
    call = L.qlinear_quantize_weight_w4
    assert call(None, 64, 64, 32, A, A, None, None) == INV
    assert call(A, 64, 64, 32, None, A, None, None) == INV
    assert call(A, 64, 64, 32, A, A + 2, None, None) == MIS
    assert call(A, 64, 80, 32, A, A, None, None) == SHAPE
    assert call(A, 64, 64, 48, A, A, None, None) == SHAPE
    assert call(A, -1, 64, 32, A, A, None, None) == INV


def test_binding_refuses_host_tensors():
    wq, sw = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ql.W4Weight(wq, sw, group=32)
    with pytest.raises(ValueError):
        ql.W4Weight(wq, sw, group=48)
