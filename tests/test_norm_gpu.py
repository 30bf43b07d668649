"""GPU tests of ep_rmsnorm and ep_rmsnorm_backward against the 64-bit definition."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import (F32, FP8, assert_bf16, assert_f32, assert_fp8, f64)

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def check_forward(ep, x, residual, gamma, out, eps=EPS):
    xd, rd = f64(x), None if residual is None else f64(residual)
    s, rstd, v = P.rmsnorm(xd, rd, f64(gamma), eps)
    ep.ep_rmsnorm(x, gamma, eps, residual, **out)
    torch.cuda.synchronize()
    if out.get("residual_out") is not None:
        assert_bf16(out["residual_out"], s, what="residual_out")
    if out.get("rstd") is not None:
        assert_f32(out["rstd"], rstd, F32 * rstd, what="rstd")
    if out.get("y") is not None:
        assert_bf16(out["y"], v, what="y")
    if out.get("y_fp8") is not None:
        assert_fp8(out["y_fp8"], out["y_sf"], v, what="y_fp8")


@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (5, 256), (33, 1024), (7, 1152), (130, 2048),
                                 (9, 4096), (301, 7168), (3, 16384), (2, 32768)])
@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("res", [False, True])
def test_forward_fp8(ep, T, H, col, res):
    g = torch.Generator().manual_seed(T + H)
    x, r = normal(g, T, H), normal(g, T, H, std=3.0) if res else None
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    if T % 2:
        gamma = gamma.to(torch.bfloat16)
    out = ep.alloc_rmsnorm(x, residual=res, bf16=H <= 4096, fp8=True, col_major_sf=col, rstd=True)
    check_forward(ep, x, r, gamma, out)


@pytest.mark.parametrize("H", [8, 24, 248, 1000, 1032, 4104, 8200])
def test_forward_bf16_any_width(ep, H):
    """Widths that are no multiple of a block, with row strides of their own."""
    g = torch.Generator().manual_seed(H)
    xs, rs = normal(g, 6, H + 8), normal(g, 6, H + 64)
    gamma = normal(g, H)
    out = ep.alloc_rmsnorm(xs[:, :H], residual=True, bf16=True, fp8=False, rstd=True)
    check_forward(ep, xs[:, :H], rs[:, 8:H + 8], gamma, out)


@pytest.mark.parametrize("H", [16, 496, 504, 512, 520, 528, 784, 8176])
@pytest.mark.parametrize("T", [1, 5, 129])
def test_forward_bf16_rows_of_a_warp_or_more(ep, T, H):
    """Widths about the one up to which a row is a warp's, and partial last warps."""
    g = torch.Generator().manual_seed(T + 3 * H)
    x, r = normal(g, T, H), normal(g, T, H)
    out = ep.alloc_rmsnorm(x, residual=True, bf16=True, fp8=False, rstd=True)
    check_forward(ep, x, r, normal(g, H), out)


@pytest.mark.parametrize("T", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("H", [128, 256])
def test_allocated_scales(ep, T, H):
    """The scales' shapes and strides of few rows, taken by the norm as they are."""
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(H, device="cuda")
    for col in (False, True):
        o = ep.alloc_rmsnorm(x, fp8=True, col_major_sf=col)
        assert o["y_sf"].shape == (T, H // 128)
        assert not col or H == 128 or o["y_sf"].stride(1) % 4 == 0
        ep.ep_rmsnorm(x, gamma, EPS, **o)
        torch.cuda.synchronize()
        assert torch.allclose(o["y_sf"], torch.full_like(o["y_sf"], 1 / 448), rtol=1e-5)


def test_forward_in_place_residual(ep):
    g = torch.Generator().manual_seed(2)
    x, r = normal(g, 40, 2048), normal(g, 40, 2048)
    want = r.clone()
    gamma = normal(g, 2048)
    ref = ep.alloc_rmsnorm(x, residual=True, bf16=True, fp8=True)
    ep.ep_rmsnorm(x, gamma, EPS, want, **ref)
    out = dict(ref, residual_out=r, y=torch.empty_like(x), y_fp8=torch.empty_like(ref["y_fp8"]))
    ep.ep_rmsnorm(x, gamma, EPS, r, **out)
    torch.cuda.synchronize()
    assert torch.equal(r, ref["residual_out"]) and torch.equal(out["y"], ref["y"])
    assert torch.equal(out["y_fp8"], ref["y_fp8"])


def test_forward_special_rows(ep):
    """A zero row, huge and tiny rows, and rows holding an infinity or a NaN,
    which stay in their own row."""
    H = 1024
    g = torch.Generator().manual_seed(4)
    x = normal(g, 8, H)
    x[1] = 0
    x[2] = 1e18  # squares near the top of fp32, below its overflow
    x[3] = 1e-30
    x[4, 5] = float("inf")
    x[5, 700] = float("nan")
    gamma = normal(g, H)
    out = ep.alloc_rmsnorm(x, bf16=True, fp8=True)
    ep.ep_rmsnorm(x, gamma, EPS, **out)
    torch.cuda.synchronize()
    fine = [0, 1, 2, 3, 6, 7]
    v = P.rmsnorm(f64(x[fine]), None, f64(gamma), EPS)[2]
    y = f64(out["y"])
    # the mean of 1024 squares of 1e18 is held exactly enough; 1e-30 sits under eps
    assert np.allclose(y[fine], v, rtol=2 ** -7, atol=1e-30)
    assert not y[1].any() and not f64(out["y_sf"])[1].any() and not out["y_fp8"][1].any()
    assert np.isnan(y[5]).all() and (out["y_fp8"][5] == 0x7F).all()
    assert torch.isnan(out["y_sf"][5]).all()
    assert np.isnan(y[4, 5]) and (y[4, :5] == 0).all()  # rstd 0: inf * 0 at the infinity


def test_scales_feed_prequantised_dispatch(ep):
    """Both scale layouts go straight into ep_dispatch_fp8."""
    T, K, E, H = 50, 2, 8, 512
    g = torch.Generator().manual_seed(9)
    x, gamma = normal(g, T, H), normal(g, H)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).cuda()
    got = []
    for col in (False, True):
        o = ep.alloc_rmsnorm(x, col_major_sf=col)
        ep.ep_rmsnorm(x, gamma, EPS, **o)
        cfg = ep.make_config(T, K, E, 2, H, 25, do_expand=True, use_fp8=True)
        h = ep.ep_layout(cfg, idx)
        r = ep.alloc_recv(h)
        ep.ep_dispatch_fp8(h, o["y_fp8"], o["y_sf"], None, **r)
        dst = h.tensor("dst_buffer_slot_idx").long()
        torch.cuda.synchronize()
        assert torch.equal(r["recv_x"][dst[:, 1]], o["y_fp8"])
        assert torch.equal(r["recv_sf"].view(-1, H // 128)[dst[:, 0]], o["y_sf"])
        got.append(r["recv_x"])
    assert torch.equal(*got)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (2, 128), (37, 1000), (300, 1024), (700, 4096),
                                 (513, 7168), (40, 16384), (5, 32768), (4096, 256)])
@pytest.mark.parametrize("res", [False, True])
def test_backward(ep, T, H, res):
    g = torch.Generator().manual_seed(T * 7 + H)
    r, gy = normal(g, T, H, std=2.0), normal(g, T, H)
    gres = normal(g, T, H) if res else None
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    if T % 2:
        gamma = gamma.to(torch.bfloat16)
    rstd = torch.rsqrt(r.float().square().mean(1) + EPS)
    gx, gg = ep.ep_rmsnorm_backward(gy, r, gamma, rstd, gres)
    gx2, none = ep.ep_rmsnorm_backward(gy, r, gamma, rstd, gres, need_gamma=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(gx, gx2)
    rd, gyd, gd, kd = f64(r), f64(gy), f64(gamma), f64(rstd)
    wx, wg = P.rmsnorm_backward(gyd, rd, gd, kd, None if gres is None else f64(gres))
    xh, t = rd * kd[:, None], gyd * gd
    mag = kd[:, None] * (np.abs(t) + np.abs(xh) * np.abs(t * xh).mean(1, keepdims=True))
    if res:
        mag = mag + np.abs(f64(gres))
    assert_bf16(gx, wx, F32 * mag, "grad_x")
    assert_f32(gg, wg, 4 * F32 * np.abs(gyd * xh).sum(0), "grad_gamma")


def test_backward_in_place_and_repeatable(ep):
    g = torch.Generator().manual_seed(5)
    r, gy, gres = (normal(g, 900, 2048) for _ in range(3))
    gamma = normal(g, 2048)
    rstd = torch.rsqrt(r.float().square().mean(1) + EPS)
    gx, gg = ep.ep_rmsnorm_backward(gy, r, gamma, rstd, gres)
    same, gg2 = ep.ep_rmsnorm_backward(gy, r, gamma, rstd, gres, grad_x=gres)
    torch.cuda.synchronize()
    assert torch.equal(gx, same) and torch.equal(gg, gg2)


def test_backward_follows_differences(ep):
    """The kernel's gradient against central differences of the definition."""
    T, H = 3, 16
    g = torch.Generator().manual_seed(6)
    x, go, gamma = normal(g, T, H), normal(g, T, H), normal(g, H)
    out = ep.alloc_rmsnorm(x, bf16=True, fp8=False, rstd=True)
    ep.ep_rmsnorm(x, gamma, EPS, **out)
    gx, gg = ep.ep_rmsnorm_backward(go, x, gamma, out["rstd"])
    xd, gd, god = f64(x), f64(gamma), f64(go)

    def diff(f, v):
        d = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            e = np.zeros_like(v)
            e[i] = 1e-5
            d[i] = (god * (f(v + e) - f(v - e))).sum() / 2e-5
        return d

    wx = diff(lambda v: P.rmsnorm(v, None, gd, EPS)[2], xd)
    wg = diff(lambda v: P.rmsnorm(xd, None, v, EPS)[2], gd)
    # differences to about 1e-8, sums of at most 16 terms of order 1
    assert_bf16(gx, wx, 1e-4, "grad_x")
    assert_f32(gg, wg, 1e-4, "grad_gamma")


def test_empty_and_refusals(ep):
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(256, device="cuda")
    ep.ep_rmsnorm(x, gamma, EPS, **ep.alloc_rmsnorm(x))
    gx, gg = ep.ep_rmsnorm_backward(x, x, gamma, torch.zeros(0, device="cuda"))
    torch.cuda.synchronize()
    assert gx.shape == (0, 256) and not gg.any()
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    out = ep.alloc_rmsnorm(x, bf16=True)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x.float(), gamma, EPS, **out)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, gamma[:128], EPS, **out)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, gamma, EPS, residual=x[:3], **out)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, gamma, EPS, **dict(out, y_sf=out["y_sf"][:, :1].expand(4, 2)))
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x, gamma, EPS)  # no output
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x, gamma, EPS, y_fp8=out["y_fp8"])  # bytes without scales
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x, gamma, float("nan"), **out)
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x[:1].expand(4, 256), gamma, EPS, **out)  # rows that overlap
    torch.cuda.synchronize()


def test_other_stream_and_graph(ep):
    """On another stream, and captured in a graph with its workspace."""
    g = torch.Generator().manual_seed(8)
    x, gy, gamma = normal(g, 600, 1024), normal(g, 600, 1024), normal(g, 1024)
    rstd = torch.rsqrt(x.float().square().mean(1) + EPS)
    want = ep.ep_rmsnorm_backward(gy, x, gamma, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ep.ep_rmsnorm_backward(gy, x, gamma, rstd, stream=s)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    gx, gg = torch.empty_like(x), torch.empty(1024, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_rmsnorm_backward(gy, x, gamma, rstd, grad_x=gx, grad_gamma=gg)
    for _ in range(2):
        gx.zero_()
        gg.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], gx) and torch.equal(want[1], gg)
