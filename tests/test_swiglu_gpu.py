"""GPU tests of ep_swiglu and ep_swiglu_backward against the 64-bit definition."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import (F32, FP8, assert_bf16, assert_f32, assert_fp8, f64, fp8_f64,
                               routing, row_use, sf_rows)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def slack(h):
    """fp32 arithmetic of sigmoid: the error of exp grows with its argument."""
    F = h.shape[1] // 2
    return F32 + np.abs(h[:, :F]) * 2.0 ** -22


# name: (T, K, E, R, M, A, expand, zero_pad, sync, col, fixed, drop)
LAYOUTS = {
    "aligned_col": (200, 4, 16, 4, 50, 16, True, True, True, True, False, 0.1),
    "aligned_row_no_zero": (100, 3, 8, 2, 50, 128, True, False, True, False, False, 0.1),
    "upper_bound": (90, 4, 32, 4, 25, 8, True, True, False, True, False, 0.2),
    "one_token": (1, 8, 64, 8, 1, 1, True, True, True, False, False, 0.0),
    "fixed_col": (61, 4, 16, 4, 16, 1, True, False, False, True, True, 0.1),
    "fixed_row": (64, 2, 8, 2, 32, 1, True, False, False, False, True, 0.0),
    "rank": (75, 4, 16, 4, 20, 1, False, False, False, False, False, 0.1),
    "no_rows": (9, 2, 8, 2, 5, 4, True, True, True, False, False, 1.0),
}


def layout(ep, name, hidden):
    T, K, E, R, M, A, ex, zp, sync, col, fixed, drop = LAYOUTS[name]
    cfg = ep.make_config(T, K, E, R, hidden, M, A, do_expand=ex, do_zero_padding=zp,
                         do_cpu_sync=sync, use_tma_aligned_col_major_sf=col, fixed_capacity=fixed)
    return ep.ep_layout(cfg, routing(T, K, E, 11, drop).cuda())


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("F,weights", [(128, True), (384, False), (1408, True)])
def test_layouts(ep, name, F, weights):
    h = layout(ep, name, 256)
    rows = h.rows_alloc
    use, pad = row_use(h)
    zero = pad & bool(h.cfg.do_zero_padding)
    g = torch.Generator().manual_seed(F)
    gate_up, ga = normal(g, rows, 2 * F, std=2.0), normal(g, rows, F)
    # rows that are not in use hold anything
    gate_up[torch.from_numpy(~use).cuda()] = float("nan")
    ga[torch.from_numpy(~use).cuda()] = float("nan")
    w = torch.randn(rows, generator=g).cuda() if weights else None
    act = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
    q, sf = ep.alloc_fp8(h, F, zero=True)
    q.fill_(0x55)
    ck = torch.full((rows, 2 * F), 0x33, dtype=torch.uint8, device="cuda")
    cksf = torch.full((rows, F // 64), 5.0, device="cuda")
    ep.ep_swiglu(h, gate_up, w, act=act, act_fp8=q, act_sf=sf, ckpt=ck, ckpt_sf=cksf)
    torch.cuda.synchronize()
    hd, wd = f64(gate_up)[use], None if w is None else f64(w)[use]
    want = P.swiglu(hd, wd)
    sl = slack(hd) * np.abs(want)
    assert_bf16(act[use], want, sl, "act")
    s = sf_rows(ep, h, sf, F) if rows else sf.view(0, F // 128)
    assert_fp8(q[use], s[use], want, sl, "act_fp8")
    assert_fp8(ck[use], cksf[use], hd, what="checkpoint")
    rest = ~(use | zero)
    assert (act[rest] == 7).all() and (q[rest] == 0x55).all(), "unused rows written"
    assert not act[zero].any() and not q[zero].any() and not s[zero].any(), "padding"
    assert (ck[~use] == 0x33).all() and (cksf[~use] == 5).all(), "checkpoint of unused rows"

    # backward, from the checkpoint's own values
    cv = fp8_f64(ck)[use] * np.repeat(f64(cksf)[use], 128, axis=1)
    wgh, wgw = P.swiglu_backward(cv, f64(ga)[use], wd)
    gh = torch.full((rows, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda")
    gq, gsf = ep.alloc_fp8(h, 2 * F, zero=True)
    gq.fill_(0x55)
    gw = torch.full((rows,), 7.0, device="cuda")
    ep.ep_swiglu_backward(h, ga, ck, cksf, w, grad_gate_up=gh, grad_fp8=gq, grad_sf=gsf,
                          grad_row_weights=gw)
    torch.cuda.synchronize()
    d = f64(ga)[use] * (1 if wd is None else wd[:, None])
    g64, u64 = cv[:, :F], cv[:, F:]
    sg = 1 / (1 + np.exp(-g64))
    mag = np.concatenate([np.abs(d * u64 * sg) * (1 + np.abs(g64)), np.abs(d * g64 * sg)], 1)
    sl = np.concatenate([slack(cv)] * 2, 1) * 4 * mag
    assert_bf16(gh[use], wgh, sl, "grad_gate_up")
    s = sf_rows(ep, h, gsf, 2 * F) if rows else gsf.view(0, F // 64)
    assert_fp8(gq[use], s[use], wgh, sl, "grad_fp8")
    terms = np.abs(f64(ga)[use] * g64 * sg * u64) * slack(cv) * 4
    assert_f32(gw[use], wgw, terms.sum(1), "grad_row_weights")
    assert (gh[rest] == 7).all() and (gq[rest] == 0x55).all() and (gw[rest] == 7).all()
    assert not gh[zero].any() and not gq[zero].any() and not gw[zero].any()
    h.free()


@pytest.mark.parametrize("rows,F", [(1, 128), (3, 8), (257, 1024), (5, 32768), (1000, 256), (2, 72)])
def test_without_handle(ep, rows, F):
    g = torch.Generator().manual_seed(rows + F)
    gate_up = normal(g, rows, 2 * F, std=3.0)
    act = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda")
    ep.ep_swiglu(None, gate_up, act=act)
    want = P.swiglu(f64(gate_up))
    sl = slack(f64(gate_up)) * np.abs(want)
    torch.cuda.synchronize()
    assert_bf16(act, want, sl)
    if F % 128:
        return
    q = torch.empty(rows, F, dtype=torch.uint8, device="cuda")
    sf = torch.empty(rows, F // 128, device="cuda")
    ck = torch.empty(rows, 2 * F, dtype=torch.uint8, device="cuda")
    cs = torch.empty(rows, F // 64, device="cuda")
    ep.ep_swiglu(None, gate_up, act_fp8=q, act_sf=sf, ckpt=ck, ckpt_sf=cs)
    gh, gw = torch.empty_like(gate_up), torch.empty(rows, device="cuda")
    ep.ep_swiglu_backward(None, act, ck, cs, grad_gate_up=gh, grad_row_weights=gw)
    torch.cuda.synchronize()
    assert_fp8(q, sf, want, sl)
    cv = fp8_f64(ck) * np.repeat(f64(cs), 128, axis=1)
    wgh, wgw = P.swiglu_backward(cv, f64(act))
    g64, u64, sg = cv[:, :F], cv[:, F:], 1 / (1 + np.exp(-cv[:, :F]))
    mag = np.concatenate([np.abs(f64(act) * u64 * sg) * (1 + np.abs(g64)),
                          np.abs(f64(act) * g64 * sg)], 1)
    assert_bf16(gh, wgh, np.concatenate([slack(cv)] * 2, 1) * 4 * mag)
    assert_f32(gw, wgw, (np.abs(f64(act) * g64 * sg * u64) * slack(cv) * 4).sum(1) + 1e-30)


def test_special_values(ep):
    """Gates far out in both tails, zeros, an infinity and a NaN in one block."""
    F = 256
    h = torch.zeros(4, 2 * F, dtype=torch.bfloat16, device="cuda")
    h[0, :F] = torch.linspace(-300, 300, F)
    h[0, F:] = 1
    h[2] = 1
    h[2, 3] = float("nan")
    h[3] = 1
    h[3, F + 200] = float("inf")
    act = torch.empty(4, F, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(4, F, dtype=torch.uint8, device="cuda")
    sf = torch.empty(4, 2, device="cuda")
    ep.ep_swiglu(None, h, act=act, act_fp8=q, act_sf=sf)
    torch.cuda.synchronize()
    want = P.swiglu(f64(h[:1]))
    assert_bf16(act[:1], want, slack(f64(h[:1])) * np.abs(want) + 1e-30)
    assert not act[1].any() and not q[1].any() and not sf[1].any()
    assert torch.isnan(act[2]).nonzero().flatten().tolist() == [3]
    assert torch.isnan(sf[2, 0]) and (q[2, :128] == 0x7F).all()
    assert torch.isfinite(sf[2, 1])
    assert torch.isinf(sf[3, 1]) and q[3, 200] == 0x7F and not (q[3, 128:200]).any()


def test_backward_follows_differences(ep):
    """The kernel's gradient against central differences of the definition, at
    the checkpoint's values."""
    rows, F = 2, 128
    g = torch.Generator().manual_seed(3)
    h, ga, w = normal(g, rows, 2 * F, std=2.0), normal(g, rows, F), torch.randn(rows).cuda()
    ck = torch.empty(rows, 2 * F, dtype=torch.uint8, device="cuda")
    cs = torch.empty(rows, 2, device="cuda")
    ep.ep_swiglu(None, h, w, ckpt=ck, ckpt_sf=cs)
    gh, gw = torch.empty_like(h), torch.empty(rows, device="cuda")
    ep.ep_swiglu_backward(None, ga, ck, cs, w, grad_gate_up=gh, grad_row_weights=gw)
    torch.cuda.synchronize()
    cv = fp8_f64(ck) * np.repeat(f64(cs), 128, axis=1)
    god, wd = f64(ga), f64(w)
    want = np.zeros_like(cv)
    for i in np.ndindex(cv.shape):
        e = np.zeros_like(cv)
        e[i] = 1e-5
        want[i] = (god * (P.swiglu(cv + e, wd) - P.swiglu(cv - e, wd))).sum() / 2e-5
    ww = (god * P.swiglu(cv)).sum(1)  # linear in the weight
    # differences to about 1e-8; values of order 10
    assert_bf16(gh, want, 1e-4)
    assert_f32(gw, ww, 1e-3)


def test_refusals(ep):
    h = layout(ep, "aligned_col", 256)
    rows = h.rows_alloc
    gu = torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda")
    act = torch.zeros(rows, 256, dtype=torch.bfloat16, device="cuda")
    q, sf = ep.alloc_fp8(h, 256)
    with pytest.raises(ep.EpError):
        ep.ep_swiglu(h, gu)  # no output
    with pytest.raises(ep.EpError):
        ep.ep_swiglu(h, gu, act_fp8=q)  # bytes without scales
    with pytest.raises(ValueError):
        ep.ep_swiglu(h, gu[:-1], act=act)  # not the handle's rows
    with pytest.raises(ValueError):
        ep.ep_swiglu(h, gu, act=act.float())
    with pytest.raises(ValueError):
        ep.ep_swiglu(h, gu, act_fp8=q, act_sf=sf[:-1])
    with pytest.raises(ValueError):
        ep.ep_swiglu(h, gu.cpu(), act=act)
    with pytest.raises(ValueError):
        ep.ep_swiglu(h, gu.t().contiguous().t(), act=act)
    wide = torch.zeros(4, 2 * 72, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ep.EpError):  # a checkpoint needs whole blocks
        ep.ep_swiglu(None, wide, ckpt=torch.zeros(4, 144, dtype=torch.uint8, device="cuda"),
                     ckpt_sf=torch.zeros(4, 1, device="cuda"))
    h.free()
    with pytest.raises(RuntimeError):
        ep.ep_swiglu(h, gu, act=act)
    torch.cuda.synchronize()
