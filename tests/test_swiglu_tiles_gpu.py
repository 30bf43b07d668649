"""GPU tests of ep_swiglu and ep_swiglu_backward where a tile has several rows
(thousands of rows): the walk across rows, warps that hold used and padding
rows, the per-row sums and a ragged last tile, against 64 bits."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import F32, assert_bf16, assert_f32, assert_fp8, f64, fp8_f64, routing, \
    row_use, sf_rows

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


# name: (T, K, E, A, zero_pad, sync, col, F, weights); the rows give tiles of 2 to 20 on
# 152 SMs with 3 and 4 CTAs each
CASES = {
    "narrow_many": (9500, 4, 64, 16, True, True, True, 128, True),
    "narrow_no_zero": (5000, 4, 16, 128, False, True, False, 128, False),
    "three_blocks": (4200, 4, 32, 16, True, True, False, 384, True),
    "two_rows": (2450, 4, 8, 128, True, True, True, 1408, True),
    "bound_rows": (2600, 4, 24, 8, True, False, True, 384, False),
    "padding_rows": (3000, 2, 100, 128, True, True, False, 256, True),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_against_definition(ep, name):
    T, K, E, A, zp, sync, col, F, weights = CASES[name]
    cfg = ep.make_config(T, K, E, 1, 256, T, A, do_expand=True, do_zero_padding=zp,
                         do_cpu_sync=sync, use_tma_aligned_col_major_sf=col)
    h = ep.ep_layout(cfg, routing(T, K, E, 41, 0.1).cuda())
    rows = h.rows_alloc
    assert rows > 2 * 4 * 152 * 4, "tiles of one row"
    use, pad = row_use(h)
    zero, rest = pad & zp, ~(use | (pad & zp))
    g = torch.Generator().manual_seed(F + T)
    gate_up, ga = normal(g, rows, 2 * F, std=2.0), normal(g, rows, F)
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
    s = sf_rows(ep, h, sf, F)
    assert_fp8(q[use], s[use], want, sl, "act_fp8")
    assert_fp8(ck[use], cksf[use], hd, what="checkpoint")
    assert (act[rest] == 7).all() and (q[rest] == 0x55).all(), "unused rows written"
    assert not act[zero].any() and not q[zero].any() and not s[zero].any(), "padding"
    assert (ck[~use] == 0x33).all() and (cksf[~use] == 5).all(), "checkpoint of unused rows"

    cv = fp8_f64(ck)[use] * np.repeat(f64(cksf)[use], 128, axis=1)
    gad = f64(ga)[use]
    wgh, wgw = P.swiglu_backward(cv, gad, wd)
    gh = torch.full((rows, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda")
    gq, gsf = ep.alloc_fp8(h, 2 * F, zero=True)
    gq.fill_(0x55)
    gw = torch.full((rows,), 7.0, device="cuda")
    ep.ep_swiglu_backward(h, ga, ck, cksf, w, grad_gate_up=gh, grad_fp8=gq, grad_sf=gsf,
                          grad_row_weights=gw)
    torch.cuda.synchronize()
    d = gad * (1 if wd is None else wd[:, None])
    g64, u64 = cv[:, :F], cv[:, F:]
    sg = 1 / (1 + np.exp(-g64))
    mag = np.concatenate([np.abs(d * u64 * sg) * (1 + np.abs(g64)), np.abs(d * g64 * sg)], 1)
    sl = np.concatenate([slack(cv)] * 2, 1) * 4 * mag
    assert_bf16(gh[use], wgh, sl, "grad_gate_up")
    s = sf_rows(ep, h, gsf, 2 * F)
    assert_fp8(gq[use], s[use], wgh, sl, "grad_fp8")
    assert_f32(gw[use], wgw, (np.abs(gad * g64 * sg * u64) * slack(cv) * 4).sum(1),
               "grad_row_weights")
    assert (gh[rest] == 7).all() and (gq[rest] == 0x55).all() and (gw[rest] == 7).all()
    assert not gh[zero].any() and not gq[zero].any() and not gw[zero].any()
    assert not s[zero].any()
    h.free()


@pytest.mark.parametrize("rows,F", [(20011, 128), (9001, 72)])
def test_without_handle(ep, rows, F):
    """A row count that no tile divides, and the form of eight elements."""
    g = torch.Generator().manual_seed(rows)
    gate_up = normal(g, rows, 2 * F, std=3.0)
    act = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_swiglu(None, gate_up, act=act)
    torch.cuda.synchronize()
    hd = f64(gate_up)
    want = P.swiglu(hd)
    assert_bf16(act, want, slack(hd) * np.abs(want))
