"""GPU tests of ep_combine_weighted_backward where its kernels run longer than
one item each: CTAs that take many tokens, warps that carry expert sums over
several chunks of tokens, and the wide joining of partial sums; against 64 bits."""
import numpy as np
import pytest
import torch

from tests.ops_harness import F32, assert_bf16, assert_f32, assert_fp8, f64, routing, row_use, \
    sf_rows

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


# name: (T, K, E, H, expand, num_sms): without a cap the row kernel has three CTAs or
# more on each of 152 SMs, so the first two need thousands of tokens
CASES = {
    "many_tokens": (2500, 3, 8, 7168, True, 0),
    "many_tokens_rank": (9001, 3, 16, 128, False, 0),
    "one_sm": (700, 6, 16, 1152, True, 1),
    "one_sm_rank": (700, 6, 16, 512, False, 1),
    "two_sms_odd": (403, 5, 10, 1000, False, 2),
    "three_sms_wide": (150, 4, 8, 12288, True, 3),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("bias", [False, True])
def test_many_tokens_a_cta(ep, name, bias):
    T, K, E, H, expand, cap = CASES[name]
    cfg = ep.make_config(T, K, E, 2, H, -(-T // 2), 8 if expand else 1, do_expand=expand,
                         do_zero_padding=expand, num_sms=cap)
    idx = routing(T, K, E, 19, 0.1)
    h = ep.ep_layout(cfg, idx.cuda())
    rows = h.rows_alloc
    use, pad = row_use(h)
    g = torch.Generator().manual_seed(H + T)
    go, y = normal(g, T, H), normal(g, rows, H)
    y[torch.from_numpy(~use).cuda()] = float("nan")
    w = torch.randn(T, K, generator=g).cuda()
    b = normal(g, E, H) if bias else None
    gy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((T, K), 7.0, device="cuda")
    gb = torch.full((E, H), 7.0, device="cuda") if bias else None
    fp8 = {}
    if H % 128 == 0:
        q, sf = ep.alloc_fp8(h, H, zero=True)
        fp8 = dict(grad_y_fp8=q, grad_y_sf=sf)
    ep.ep_combine_weighted_backward(h, go, y, w, b, grad_y=gy, grad_topk_weights=gw,
                                    grad_expert_bias=gb, **fp8)
    torch.cuda.synchronize()
    dst = h.tensor("dst_buffer_slot_idx").cpu().numpy().astype(np.int64)
    god, wd = f64(go), f64(w)
    # slot by slot over all tokens: the plain definition takes a Python loop a slot
    row_w, row_a, token = np.zeros(rows), np.zeros(rows), np.zeros(rows, np.int64)
    wgw, mgw = np.zeros((T, K)), np.zeros((T, K))
    wgb, mgb = np.zeros((E, H)), np.zeros((E, H))
    yd, bd = f64(y), f64(b) if bias else None
    for k in range(K):
        t = np.nonzero(dst[:, k] >= 0)[0]
        d, e = dst[t, k], idx[:, k].numpy()[t]
        v = yd[d] + (bd[e] if bias else 0)
        m = np.abs(yd[d]) + (np.abs(bd[e]) if bias else 0)
        wgw[t, k] = (v * god[t]).sum(1)
        mgw[t, k] = (m * np.abs(god[t])).sum(1)
        np.add.at(row_w, d, wd[t, k])
        np.add.at(row_a, d, np.abs(wd[t, k]))
        token[d] = t
        if bias:
            for x in range(E):
                i = t[e == x]
                wgb[x] += wd[i, k] @ god[i]
                mgb[x] += np.abs(wd[i, k]) @ np.abs(god[i])
    wgy = row_w[use, None] * god[token[use]]
    off = F32 * row_a[use, None] * np.abs(god[token[use]])
    assert_bf16(gy[use], wgy, off, "grad_y")
    assert_f32(gw, wgw, 2 * F32 * mgw, "grad_topk_weights")
    if bias:
        assert_f32(gb, wgb, (T + 64) * 2.0 ** -24 * mgb, "grad_expert_bias")
    zero, rest = pad & expand, ~(use | (pad & expand))
    assert (gy[rest] == 7).all() and not gy[zero].any()
    if fp8:
        s = sf_rows(ep, h, sf, H)
        assert_fp8(q[use], s[use], wgy, off, "grad_y_fp8")
        assert not q[zero].any() and not s[zero].any()
    h.free()


@pytest.mark.parametrize("T,K,E,H,skew", [(5000, 4, 256, 4096, False), (4000, 3, 512, 2048, True),
                                          (4000, 2, 2048, 512, False)])
def test_bias_sums_over_several_chunks(ep, T, K, E, H, skew):
    """More chunks of 256 tokens than parts (a part is made for 80 warps of each of 152
    SMs, 256 columns and 4 experts a warp), and E * H columns of partial sums."""
    parts = -(-80 * 152 // (H // 256 * (E // 4)))
    assert 1 < parts < -(-T // 256) and E * H >= 65536
    cfg = ep.make_config(T, K, E, 2, H, T // 2, 1)
    idx = routing(T, K, E, 8, 0.1, zipf=skew)
    h = ep.ep_layout(cfg, idx.cuda())
    g = torch.Generator().manual_seed(E)
    go, w = normal(g, T, H), torch.randn(T, K, generator=g).cuda()
    gb, gb2 = torch.full((E, H), 7.0, device="cuda"), torch.empty(E, H, device="cuda")
    ep.ep_combine_weighted_backward(h, go, None, w, grad_expert_bias=gb)
    ep.ep_combine_weighted_backward(h, go, None, w, grad_expert_bias=gb2)
    torch.cuda.synchronize()
    assert torch.equal(gb, gb2)
    dense = np.zeros((T, E))
    for k in range(K):
        m = idx[:, k].numpy() >= 0
        dense[np.arange(T)[m], idx[:, k].numpy()[m]] += f64(w)[m, k]
    god = f64(go)
    tol = (T + 64) * 2.0 ** -24 * (np.abs(dense).T @ np.abs(god))
    assert_f32(gb, dense.T @ god, tol)
    h.free()


def test_refuses_widths_without_whole_blocks(ep):
    """FP8 rows of a width that is no multiple of a scale block, with bytes and scales
    given; and bytes or scales alone where the width would do."""
    lib = ep.load_library()
    for H, q, sf, status in [(72, True, True, ep.EP_ERR_INVALID_ARG),
                             (128, True, False, ep.EP_ERR_INVALID_ARG),
                             (128, False, True, ep.EP_ERR_INVALID_ARG),
                             (128, True, True, ep.EP_OK)]:
        h = ep.ep_layout(ep.make_config(8, 2, 8, 2, H, 4, 1), routing(8, 2, 8, 1).cuda())
        go = torch.zeros(8, H, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros(8, 2, device="cuda")
        b = torch.zeros(h.rows_alloc, 128, dtype=torch.uint8, device="cuda")
        s = torch.zeros(h.rows_alloc, 1, device="cuda")
        st = lib.ep_combine_weighted_backward(
            h.ptr, go.data_ptr(), None, w.data_ptr(), None, None, b.data_ptr() if q else None,
            s.data_ptr() if sf else None, None, None, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == status, (H, q, sf)
        h.free()
