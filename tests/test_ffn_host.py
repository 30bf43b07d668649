"""Refusals of the feed-forward block's products and of clipping that come before
any GPU work (no GPU needed), and the gradients' formulas against differences."""
import ctypes

import numpy as np
import pytest

from oracle import ops_oracle as O


@pytest.fixture(scope="module")
def lib():
    import combine_topk_idx_gb300 as ep
    from combine_topk_idx_gb300 import _build_lib
    _build_lib.build()
    return ep.load_library()


P = 0x10000  # an aligned address that is never dereferenced here
INVALID, UNSUPPORTED = 1, 2
SIZES = [(dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(n=0), INVALID),
         (dict(n=12), INVALID), (dict(n=65544), UNSUPPORTED), (dict(k=4), INVALID),
         (dict(k=20), INVALID), (dict(k=65544, ks=65544), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(n=32776), UNSUPPORTED), (dict(ks=248), INVALID), (dict(ks=260), INVALID),
    (dict(x=None), INVALID), (dict(x=P + 8), INVALID), (dict(w=None), INVALID),
    (dict(w=P + 2), INVALID), (dict(act=None), INVALID), (dict(act=P + 8), INVALID),
    (dict(gu=P + 8), INVALID), (dict(rows=0, act=None, x=None, w=None), 0)])
def test_gated(lib, kw, status):
    a = dict(h=None, rows=4, n=64, k=256, x=P, ks=256, w=P, act=P, gu=None)
    a.update(kw)
    assert lib.ep_ffn_gated(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(ks=248), INVALID), (dict(gy=None), INVALID), (dict(w=None), INVALID),
    (dict(gu=None), INVALID), (dict(ggu=None), INVALID), (dict(act=P + 8), INVALID),
    (dict(rows=0, gy=None), 0)])
def test_gated_backward(lib, kw, status):
    a = dict(h=None, rows=4, n=64, k=256, gy=P, ks=256, w=P, gu=P, ggu=P, act=None)
    a.update(kw)
    assert lib.ep_ffn_gated_backward(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(ks=252), INVALID), (dict(a=None), INVALID), (dict(w=None), INVALID),
    (dict(t=2), INVALID), (dict(t=-1), INVALID), (dict(out=None), INVALID),
    (dict(out=P + 8), INVALID), (dict(rows=0, a=None, out=None), 0)])
def test_product(lib, kw, status):
    a = dict(h=None, rows=4, n=64, k=256, a=P, ks=256, w=P, t=0, out=P)
    a.update(kw)
    assert lib.ep_ffn_product(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(ns=56), INVALID), (dict(ks=252), INVALID), (dict(g=None), INVALID),
    (dict(a=None), INVALID), (dict(gw=None), INVALID), (dict(gw=P + 8), INVALID),
    (dict(f32=2), INVALID), (dict(acc=-1), INVALID), (dict(rows=0, acc=1, g=None, a=None), 0)])
def test_weight_grad(lib, kw, status):
    a = dict(h=None, rows=4, n=64, k=256, g=P, ns=65600, a=P, ks=256, gw=P, f32=1, acc=0)
    a.update(kw)
    assert lib.ep_ffn_weight_grad(*a.values(), None) == status


def clip(lib, count=1, grads=(P,), outs=(P,), numels=(8,), f32=(1,), max_norm=1.0, norm=P):
    def array(kind, v):
        return None if v is None else (kind * len(v))(*v)
    return lib.ep_clip_grads(count, array(ctypes.c_void_p, grads), array(ctypes.c_void_p, outs),
                             array(ctypes.c_int64, numels), array(ctypes.c_uint8, f32), max_norm,
                             norm, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), INVALID), (dict(grads=None), INVALID), (dict(numels=None), INVALID),
    (dict(f32=None), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("nan")), INVALID),
    (dict(outs=None, norm=None), INVALID), (dict(norm=P + 2), INVALID), (dict(numels=(-1,)), INVALID),
    (dict(f32=(2,)), INVALID), (dict(numels=((1 << 40) + 1,)), UNSUPPORTED),
    (dict(grads=(None,)), INVALID), (dict(outs=(None,)), INVALID), (dict(grads=(P + 2,)), INVALID),
    (dict(outs=(P + 2,)), INVALID), (dict(f32=(0,), grads=(P + 1,)), INVALID)])
def test_clip(lib, kw, status):
    assert clip(lib, **kw) == status


def test_gradients_against_differences():
    """The definitions that the GPU tests use: the block's gradients are its differences."""
    r = np.random.RandomState(3)
    rows, k, F, n = 5, 6, 4, 3
    x, w_in, w_out = r.randn(rows, k), r.randn(2, 2 * F, k), r.randn(2, n, F)
    starts, counts, target = [0, 3], [3, 2], r.randn(rows, n)

    def loss(x, w_in, w_out):
        h = O.segment_product(x, w_in, starts, counts)
        return (O.segment_product(O.swiglu(h), w_out, starts, counts) * target).sum()

    h = O.segment_product(x, w_in, starts, counts)
    slopes, act = O.gated_slopes(h)
    d = O.segment_product(target, w_out, starts, counts, True)
    gh = np.tile(d, 2) * slopes
    got = (O.segment_product(gh, w_in, starts, counts, True),
           O.segment_outer(gh, x, starts, counts), O.segment_outer(target, act, starts, counts))
    for i, grad in enumerate(got):
        args = [x, w_in, w_out]
        for at in [tuple(r.randint(s) for s in grad.shape) for _ in range(12)]:
            step = np.zeros_like(grad)
            step[at] = 1e-5
            up, down = ([a + s * step if j == i else a for j, a in enumerate(args)]
                        for s in (1, -1))
            diff = (loss(*up) - loss(*down)) / 2e-5
            assert abs(diff - grad[at]) < 1e-6 * max(1, abs(diff))


def test_global_norm():
    r = np.random.RandomState(4)
    g = [r.randn(7), r.randn(3, 2), np.zeros(0)]
    assert abs(O.global_norm(g) - np.sqrt((g[0] ** 2).sum() + (g[1] ** 2).sum())) < 1e-12
    assert O.global_norm([np.full(4, 1e300)]) == 2e300
    assert O.global_norm([]) == 0.0


@pytest.mark.parametrize("how", ["emptied", "emptied_and_filled", "shrunk", "grown"])
def test_memory_that_was_given_back(how):
    """What a plan holds: a storage keeps its memory until it is resized, which is noticed."""
    import torch
    from combine_topk_idx_gb300._ffn import _Memory
    a, b = torch.ones(1000), torch.ones(500)
    m = _Memory([a, a[:3], b, b[7:], torch.empty(0)])
    assert len(m.storages) == 3 and not m.moved()
    a.mul_(2)
    b.resize_(100)  # within the storage
    at = a.data_ptr()
    a.data = torch.zeros(1000)  # the storage of before is held
    assert not m.moved() and m.storages[0].data_ptr() == at
    s = b.untyped_storage()
    if how == "grown":
        b.resize_(100_000)
    else:
        s.resize_(1000 if how == "shrunk" else 0)
    if how == "emptied_and_filled":
        s.resize_(1200)
    assert m.moved()
