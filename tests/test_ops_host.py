"""Refusals of the operators around dispatch and combine that come before any
GPU work (no GPU needed): arguments a wrong caller might pass."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import combine_topk_idx_gb300 as ep
    from combine_topk_idx_gb300 import _build_lib
    _build_lib.build()
    return ep.load_library()


P = 0x10000  # an aligned address that is never dereferenced here
INVALID, UNSUPPORTED = 1, 2


def norm(lib, **kw):
    a = dict(T=4, H=256, x=P, xs=256, r=None, rs=0, g=P, f32=0, eps=1e-6, ro=None, y=P, q=None,
             sf=None, ts=2, hs=1, rstd=None)
    a.update(kw)
    return lib.ep_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=252), INVALID),
    (dict(H=65536, xs=65536), UNSUPPORTED), (dict(xs=248), INVALID), (dict(xs=260), INVALID),
    (dict(x=None), INVALID), (dict(x=P + 2), INVALID), (dict(g=None), INVALID),
    (dict(f32=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y=None), INVALID), (dict(y=P + 8), INVALID), (dict(q=P), INVALID),
    (dict(sf=P), INVALID), (dict(q=P, sf=P, ts=0), INVALID), (dict(q=P, sf=P + 2), INVALID),
    (dict(q=P, sf=P, H=264, xs=264), INVALID), (dict(r=P, rs=8), INVALID),
    (dict(r=P, rs=512, ro=P), INVALID), (dict(rstd=P + 1), INVALID),
    (dict(T=0, x=None, y=None, g=None), 0),
])
def test_norm(lib, kw, status):
    assert norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=12), INVALID), (dict(gy=None), INVALID), (dict(r=None), INVALID),
    (dict(g=P + 4), INVALID), (dict(rstd=None), INVALID), (dict(gx=None), INVALID),
    (dict(gg=P + 4), INVALID), (dict(f32=-1), INVALID), (dict(gres=P + 2), INVALID),
    (dict(T=0, gg=None), 0),
])
def test_norm_backward(lib, kw, status):
    a = dict(T=4, H=256, gy=P, r=P, g=P, f32=0, rstd=P, gres=None, gx=P, gg=P)
    a.update(kw)
    assert lib.ep_rmsnorm_backward(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(F=0), INVALID), (dict(F=12), INVALID), (dict(F=136, q=P, sf=P), INVALID),
    (dict(F=65536), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(h=None), INVALID),
    (dict(act=None), INVALID), (dict(q=P), INVALID), (dict(ck=P), INVALID), (dict(w=P + 2), INVALID),
    (dict(act=P + 2), INVALID), (dict(rows=0, h=None, act=None), 0),
])
def test_swiglu(lib, kw, status):
    a = dict(handle=None, rows=4, F=256, h=P, w=None, act=P, q=None, sf=None, ck=None, cs=None)
    a.update(kw)
    assert lib.ep_swiglu(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(F=136), INVALID), (dict(ga=None), INVALID), (dict(ck=None), INVALID),
    (dict(cs=None), INVALID), (dict(gh=None), INVALID), (dict(q=P), INVALID),
    (dict(gw=P + 2), INVALID), (dict(rows=0), 0),
])
def test_swiglu_backward(lib, kw, status):
    a = dict(handle=None, rows=4, F=256, ga=P, ck=P, cs=P, w=None, gh=P, q=None, sf=None, gw=None)
    a.update(kw)
    assert lib.ep_swiglu_backward(*a.values(), None) == status


def test_without_a_handle(lib):
    v = ctypes.c_int64()
    r = ctypes.byref(v)
    assert lib.ep_sf_layout(None, 128, r, r, r, r) == INVALID
    assert lib.ep_combine_weighted_backward(*[None] * 11) == INVALID


def test_expert_gemm_without_a_handle(lib):
    assert lib.ep_expert_gemm(None, 256, 256, P, P, P, P, P, None) == INVALID
