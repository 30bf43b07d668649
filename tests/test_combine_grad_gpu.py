"""GPU tests of ep_combine_weighted_backward against the 64-bit definition."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import (F32, assert_bf16, assert_f32, assert_fp8, f64, routing, row_use,
                               sf_rows)

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


# name: (T, K, E, R, H, M, A, expand, zero_pad, sync, col, fixed, drop, dup)
CASES = {
    "expand_col": (150, 4, 16, 4, 256, 40, 16, True, True, True, True, False, 0.1, False),
    "expand_wide": (40, 8, 64, 8, 7168, 5, 8, True, True, True, True, False, 0.0, False),
    "expand_no_zero": (60, 3, 8, 2, 384, 30, 128, True, False, True, False, False, 0.1, False),
    "upper_bound": (90, 4, 32, 4, 128, 25, 8, True, True, False, False, False, 0.2, False),
    "rank_shared": (120, 6, 16, 2, 512, 60, 1, False, False, True, False, False, 0.1, False),
    "rank_dup": (50, 6, 8, 2, 128, 25, 1, False, False, True, False, False, 0.1, True),
    "fixed": (64, 4, 16, 4, 256, 16, 1, True, False, False, True, True, 0.1, False),
    "one_token": (1, 8, 64, 8, 1152, 1, 64, True, True, True, True, False, 0.0, False),
    "max_topk": (20, 32, 64, 4, 128, 5, 1, True, True, True, False, False, 0.1, False),
    "no_slots": (12, 3, 8, 4, 128, 3, 4, True, True, True, False, False, 1.0, False),
    "no_tokens": (0, 4, 8, 2, 128, 4, 4, True, True, True, False, False, 0.0, False),
    "many_experts": (33, 4, 600, 4, 128, 9, 1, True, True, True, False, False, 0.0, False),
    "widest": (6, 2, 8, 2, 32768, 3, 4, True, True, True, True, False, 0.0, False),
    "wide": (9, 4, 8, 2, 12288, 5, 8, True, True, True, True, False, 0.0, False),
    "odd_wide": (7, 4, 10, 2, 8200, 4, 1, False, False, True, False, False, 0.1, False),
    "many_chunks": (1100, 4, 13, 13, 264, 90, 1, True, True, True, False, False, 0.1, False),
    "odd_width": (70, 4, 16, 4, 1000, 20, 1, False, False, True, False, False, 0.1, False),
    "narrow": (513, 2, 4, 1, 8, 513, 8, True, True, True, False, False, 0.1, False),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("bias", [False, True])
def test_against_definition(ep, name, bias):
    T, K, E, R, H, M, A, ex, zp, sync, col, fixed, drop, dup = CASES[name]
    cfg = ep.make_config(T, K, E, R, H, M, A, do_expand=ex, do_zero_padding=zp, do_cpu_sync=sync,
                         use_tma_aligned_col_major_sf=col, fixed_capacity=fixed)
    idx = routing(T, K, E, 5, drop, dup=dup)
    h = ep.ep_layout(cfg, idx.cuda())
    rows = h.rows_alloc
    use, pad = row_use(h)
    zero = pad & zp
    g = torch.Generator().manual_seed(H)
    go, y = normal(g, T, H), normal(g, rows, H)
    y[torch.from_numpy(~use).cuda()] = float("nan")
    w = torch.randn(T, K, generator=g).cuda()  # of both signs
    if T > 2:
        w[1] = 0
    b = normal(g, E, H) if bias else None
    gy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((T, K), 7.0, device="cuda")
    gb = torch.full((E, H), 7.0, device="cuda") if bias else None
    fp8 = {}
    if H % 128 == 0:
        q, sf = ep.alloc_fp8(h, H, zero=True)
        q.fill_(0x55)
        fp8 = dict(grad_y_fp8=q, grad_y_sf=sf)
    ep.ep_combine_weighted_backward(h, go, y, w, b, grad_y=gy, grad_topk_weights=gw,
                                    grad_expert_bias=gb, **fp8)
    torch.cuda.synchronize()
    dst = h.tensor("dst_buffer_slot_idx").cpu().numpy()
    god, wd = f64(go), f64(w)
    yd = np.where(use[:, None], f64(y), 0.0)
    bd = f64(b) if bias else None
    wgy, row_w, token, wgw, wgb = P.combine_backward(god, yd, dst, idx.numpy(), wd, bd, E)
    wsum = P.combine_backward(god, yd, dst, idx.numpy(), np.abs(wd), bd, E)
    assert_bf16(gy[use], wgy[use], F32 * np.abs(wsum[0][use]), "grad_y")
    rest = ~(use | zero)
    assert (gy[rest] == 7).all() and not gy[zero].any()
    mag = P.combine_backward(np.abs(god), np.abs(yd), dst, idx.numpy(), np.abs(wd),
                             np.abs(bd) if bias else None, E)
    assert_f32(gw, wgw, 2 * F32 * mag[3], "grad_topk_weights")
    if bias:
        assert_f32(gb, wgb, (T + 64) * 2.0 ** -24 * mag[4], "grad_expert_bias")
    if fp8:
        s = sf_rows(ep, h, sf, H) if rows else sf.view(0, H // 128)
        assert (q[rest] == 0x55).all()
        assert not q[zero].any() and not s[zero].any()
        # the bytes are the token's, quantised without the weight
        assert_fp8(q[use], s[use], wgy[use], F32 * np.abs(wsum[0][use]), "grad_y_fp8")
    # each output by itself
    gy2, gw2 = torch.full_like(gy, 7.0), torch.full_like(gw, 7.0)
    if T:
        ep.ep_combine_weighted_backward(h, go, None, w, b, grad_y=gy2)
        ep.ep_combine_weighted_backward(h, go, y, w, b, grad_topk_weights=gw2)
        torch.cuda.synchronize()
        assert torch.equal(gy, gy2) and torch.equal(gw, gw2)
    if bias:
        gb2 = torch.full_like(gb, 7.0)
        ep.ep_combine_weighted_backward(h, go, None, w, b, grad_expert_bias=gb2)
        torch.cuda.synchronize()
        assert torch.equal(gb, gb2)
    h.free()


def test_long_batch_bias_parts(ep):
    """Tokens split over several parts, and their sums joined."""
    T, K, E, H = 3000, 4, 24, 192
    cfg = ep.make_config(T, K, E, 2, H, T // 2, 1)
    idx = routing(T, K, E, 8, 0.1)
    h = ep.ep_layout(cfg, idx.cuda())
    g = torch.Generator().manual_seed(1)
    go, w = normal(g, T, H), torch.randn(T, K, generator=g).cuda()
    gb = torch.empty(E, H, device="cuda")
    ep.ep_combine_weighted_backward(h, go, None, w, grad_expert_bias=gb)
    torch.cuda.synchronize()
    dense = np.zeros((T, E))
    for k in range(K):
        m = idx[:, k].numpy() >= 0
        dense[np.arange(T)[m], idx[:, k].numpy()[m]] += f64(w)[m, k]
    tol = (T + 64) * 2.0 ** -24 * (np.abs(dense).T @ np.abs(f64(go)))
    assert_f32(gb, dense.T @ f64(go), tol)
    gb2 = torch.empty_like(gb)
    ep.ep_combine_weighted_backward(h, go, None, w, grad_expert_bias=gb2)
    assert torch.equal(gb, gb2)


def test_is_the_adjoint_of_combine(ep):
    """<combine(y, w), g> differs by <gy, dy> and <gw, dw> when y or w moves:
    against differences of ep_combine's definition."""
    T, K, E, H = 6, 3, 8, 64
    cfg = ep.make_config(T, K, E, 2, H, 3, 1)
    idx = routing(T, K, E, 2)
    h = ep.ep_layout(cfg, idx.cuda())
    rows = h.rows_alloc
    g = torch.Generator().manual_seed(4)
    go, y, b = normal(g, T, H), normal(g, rows, H), normal(g, E, H)
    w = torch.randn(T, K, generator=g).cuda()
    gy = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    gw, gb = torch.empty(T, K, device="cuda"), torch.empty(E, H, device="cuda")
    ep.ep_combine_weighted_backward(h, go, y, w, b, grad_y=gy, grad_topk_weights=gw,
                                    grad_expert_bias=gb)
    torch.cuda.synchronize()
    dst = h.tensor("dst_buffer_slot_idx").cpu().numpy()
    god, yd, bd, wd = f64(go), f64(y), f64(b), f64(w)
    rng = np.random.default_rng(0)
    for _ in range(3):  # directions; the combine is linear in each argument
        dy, dw, db = rng.normal(size=yd.shape), rng.normal(size=wd.shape), rng.normal(size=bd.shape)
        base = (god * P.combine(yd, dst, idx.numpy(), wd, bd)).sum()
        for got, d, moved in [
                (gy, dy, P.combine(yd + dy, dst, idx.numpy(), wd, bd)),
                (gw, dw, P.combine(yd, dst, idx.numpy(), wd + dw, bd)),
                (gb, db, P.combine(yd, dst, idx.numpy(), wd, bd + db))]:
            # bf16 rows are each off by at most 2^-8 of themselves
            tol = 2.0 ** -8 * (np.abs(f64(got)) * np.abs(d)).sum()
            assert abs((god * moved).sum() - base - (f64(got) * d).sum()) <= tol


def test_stream_and_graph(ep):
    T, K, E, H = 400, 4, 16, 512
    cfg = ep.make_config(T, K, E, 4, H, 100, 8, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False)
    h = ep.ep_layout(cfg, routing(T, K, E, 3).cuda())
    g = torch.Generator().manual_seed(7)
    go, y = normal(g, T, H), normal(g, h.rows_alloc, H)
    w = torch.rand(T, K, generator=g).cuda()

    def outputs():
        return dict(grad_y=torch.zeros(h.rows_alloc, H, dtype=torch.bfloat16, device="cuda"),
                    grad_topk_weights=torch.zeros(T, K, device="cuda"),
                    grad_expert_bias=torch.zeros(E, H, device="cuda"))

    want, got, rep = outputs(), outputs(), outputs()
    ep.ep_combine_weighted_backward(h, go, y, w, **want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ep.ep_combine_weighted_backward(h, go, y, w, stream=s, **got)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_combine_weighted_backward(h, go, y, w, **rep)
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k]) and torch.equal(want[k], rep[k]), k


def test_refusals(ep):
    cfg = ep.make_config(8, 2, 8, 2, 72, 4, 1)
    h = ep.ep_layout(cfg, routing(8, 2, 8, 1).cuda())
    rows = h.rows_alloc
    go = torch.zeros(8, 72, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(rows, 72, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 2, device="cuda")
    gw = torch.zeros(8, 2, device="cuda")
    with pytest.raises(ep.EpError):
        ep.ep_combine_weighted_backward(h, go, y, w)  # no output
    with pytest.raises(ep.EpError):
        ep.ep_combine_weighted_backward(h, go, None, w, grad_topk_weights=gw)  # needs y
    with pytest.raises(ep.EpError):  # 72 is no multiple of a scale block
        ep.ep_combine_weighted_backward(h, go, y, w, grad_y_fp8=torch.zeros(
            rows, 72, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ep.EpError):
        ep.sf_layout(h, 72)
    with pytest.raises(ValueError):
        ep.ep_combine_weighted_backward(h, go[:4], y, w, grad_topk_weights=gw)
    with pytest.raises(ValueError):
        ep.ep_combine_weighted_backward(h, go, y, w.double(), grad_topk_weights=gw)
    with pytest.raises(TypeError):
        ep.ep_combine_weighted_backward(h, go, y, grad_topk_weights=gw)  # weights are required
    h.free()
