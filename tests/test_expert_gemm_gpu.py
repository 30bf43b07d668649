"""GPU tests of ep_expert_gemm against the 64-bit definition."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import FP8, assert_bf16, f64, fp8_f64, routing, row_use, sf_rows

pytestmark = pytest.mark.gpu
# fp32 sums: 128 terms of a block, then at most 64 blocks, 2^-24 each
SUM = 2.0 ** -16


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def weights(E, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(E, n, k, generator=g) * 90).clamp(-448, 448).to(FP8).view(torch.uint8).cuda()
    sf = (0.5 + torch.rand(E, -(-n // 128), k // 128, generator=g)) / 100
    return w, sf.cuda()


def activations(ep, h, k, seed):
    """Random bytes (finite) and scales on every row, in use or not."""
    g = torch.Generator().manual_seed(seed)
    rows = h.rows_alloc
    q, sf = ep.alloc_fp8(h, k)
    v = (torch.randn(rows, k, generator=g) * 60).clamp(-448, 448).to(FP8)
    q.copy_(v.view(torch.uint8))
    sf.copy_(torch.rand(sf.shape, generator=g) + 0.1)
    return q, sf


def check(ep, h, n, k, seed=1, poison=True):
    q, sf = activations(ep, h, k, seed)
    w, wsf = weights(h.E, n, k, seed + 1)
    rows = h.rows_alloc
    use, pad = row_use(h)
    if poison:  # rows not in use hold NaN bytes: they reach no other row
        q[torch.from_numpy(~use).cuda()] = 0x7F
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm(h, q, sf, w, wsf, out=out)
    torch.cuda.synchronize()
    assert int(h.tensor("error_word")[0]) & ep.EP_ERRBIT_TIMEOUT == 0
    s = f64(sf_rows(ep, h, sf, k)) if rows else np.zeros((0, k // 128))
    av = np.where(use[:, None], fp8_f64(q), 0.0)
    cnt = h.tensor("cnt_expert").cpu().numpy()
    psum = h.tensor("psum_expert").cpu().numpy()
    if h.cfg.fixed_capacity:
        cap = int(h.info.expert_capacity)
        starts, counts = np.arange(h.E) * cap, np.minimum(cnt, cap)
    else:
        starts, counts = psum[:-1], np.clip(rows - psum[:-1], 0, cnt)
    wv, ws = fp8_f64(w), f64(wsf)
    want = P.expert_gemm(av, s, wv, ws, starts, counts)
    mag = P.expert_gemm(np.abs(av), s, np.abs(wv), ws, starts, counts)
    assert_bf16(out[use], want[use], SUM * mag[use], "out")
    zero = pad & bool(h.cfg.do_zero_padding)
    assert not out[zero].any(), "padding"
    assert (out[~(use | zero)] == 7).all(), "unused rows written"


# name: (T, K, E, R, M, A, zero_pad, sync, col, fixed, drop, n, k)
CASES = {
    "one_row": (1, 1, 1, 1, 1, 1, True, True, False, False, 0.0, 256, 128),
    "one_tile": (128, 1, 1, 1, 128, 128, True, True, True, False, 0.0, 256, 256),
    "long_k": (64, 1, 1, 1, 64, 1, True, True, False, False, 0.0, 128, 7168),
    "many_stages": (200, 2, 2, 1, 200, 1, True, True, True, False, 0.0, 512, 1280),
    "aligned": (300, 4, 16, 4, 75, 128, True, True, True, False, 0.1, 384, 512),
    "align_256": (90, 2, 4, 2, 45, 256, True, True, True, False, 0.1, 256, 384),
    "unaligned_rows": (333, 4, 16, 4, 90, 1, True, True, True, False, 0.1, 640, 256),
    "no_zero": (100, 3, 8, 2, 50, 16, False, True, False, False, 0.1, 256, 384),
    "upper_bound": (90, 4, 32, 4, 25, 8, True, False, True, False, 0.2, 256, 256),
    "one_token": (1, 8, 64, 8, 1, 1, True, True, False, False, 0.0, 512, 1024),
    "fixed_col": (61, 4, 16, 4, 16, 1, False, False, True, True, 0.1, 256, 384),
    "fixed_row": (64, 2, 8, 2, 200, 1, False, False, False, True, 0.0, 136, 256),
    "odd_columns": (150, 2, 8, 2, 75, 1, True, True, True, False, 0.1, 8, 256),
    "odd_columns_wide": (150, 2, 8, 2, 75, 1, True, True, True, False, 0.1, 1000, 128),
    "no_rows": (9, 2, 8, 2, 5, 4, True, True, False, False, 1.0, 256, 128),
    "many_experts": (700, 2, 2048, 4, 200, 1, True, True, False, False, 0.0, 128, 128),
    "long_segments": (1500, 1, 2, 1, 1500, 16, True, True, True, False, 0.0, 776, 640),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_against_definition(ep, name):
    T, K, E, R, M, A, zp, sync, col, fixed, drop, n, k = CASES[name]
    cfg = ep.make_config(T, K, E, R, 128, M, A, do_expand=True, do_zero_padding=zp,
                         do_cpu_sync=sync, use_tma_aligned_col_major_sf=col, fixed_capacity=fixed)
    h = ep.ep_layout(cfg, routing(T, K, E, 13, drop).cuda())
    check(ep, h, n, k)
    h.free()


@pytest.mark.parametrize("T,E,n,k", [(4500, 2, 520, 128), (9000, 3, 264, 256), (8300, 1, 768, 128)])
def test_many_row_tiles(ep, T, E, n, k):
    """More row tiles per expert than pass over the weights together, several column tiles."""
    K = min(2, E)
    cfg = ep.make_config(T, K, E, 1, 128, T, 1, do_expand=True, do_zero_padding=True)
    h = ep.ep_layout(cfg, routing(T, K, E, 21).cuda())
    check(ep, h, n, k)
    h.free()


@pytest.mark.parametrize("n", [256, 264])
def test_out_alignment(ep, n):
    """Rows of out that start on 32 and on 16 bytes hold the same."""
    cfg = ep.make_config(90, 2, 4, 2, 128, 45, 16, do_expand=True, do_zero_padding=True)
    h = ep.ep_layout(cfg, routing(90, 2, 4, 2, 0.1).cuda())
    q, sf = activations(ep, h, 256, 7)
    w, wsf = weights(4, n, 256, 8)
    rows = h.rows_alloc
    flat = torch.full((rows * n + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    assert flat.data_ptr() % 32 == 0
    outs = [flat[o:o + rows * n].view(rows, n) for o in (0, 8, 16)]
    got = []
    for o in outs:
        flat.fill_(7.0)
        ep.ep_expert_gemm(h, q, sf, w, wsf, out=o)
        torch.cuda.synchronize()
        got.append(o.clone())
        assert (flat[:o.storage_offset()] == 7).all()
        assert (flat[o.storage_offset() + rows * n:] == 7).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    h.free()


def test_repeated_experts_overflow(ep):
    """Rows dropped by an overflowing upper bound are not touched."""
    cfg = ep.make_config(2, 4, 2, 2, 128, 1, 1, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False)
    h = ep.ep_layout(cfg, torch.tensor([[0, 0, 0, 0], [1, 1, 0, 0]]).cuda())
    check(ep, h, 256, 256, poison=False)
    h.free()


def test_special_scales_and_values(ep):
    """Zero scales, NaN bytes and an infinite scale stay in their row."""
    cfg = ep.make_config(6, 1, 1, 1, 128, 6, 1, do_expand=True, do_zero_padding=True)
    h = ep.ep_layout(cfg, torch.zeros(6, 1, dtype=torch.int64).cuda())
    q, sf = activations(ep, h, 256, 3)
    w, wsf = weights(1, 256, 256, 4)
    s = sf.view(6, 2)
    base = ep.ep_expert_gemm(h, q, sf, w, wsf).clone()
    s[1] = 0
    q[2, 130] = 0x7F
    s[3, 0] = float("inf")
    out = ep.ep_expert_gemm(h, q, sf, w, wsf)
    torch.cuda.synchronize()
    assert not out[1].any() and torch.isnan(out[2]).all()
    assert not torch.isfinite(out[3]).any()
    assert torch.equal(out[[0, 4, 5]], base[[0, 4, 5]])
    h.free()


def test_repeats_streams_and_graph(ep):
    cfg = ep.make_config(500, 4, 16, 4, 512, 125, 16, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False, use_tma_aligned_col_major_sf=True)
    h = ep.ep_layout(cfg, routing(500, 4, 16, 3).cuda())
    q, sf = activations(ep, h, 512, 5)
    w, wsf = weights(16, 768, 512, 6)
    outs = [torch.zeros(h.rows_alloc, 768, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ep.ep_expert_gemm(h, q, sf, w, wsf, out=outs[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ep.ep_expert_gemm(h, q, sf, w, wsf, out=outs[1], stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_gemm(h, q, sf, w, wsf, out=outs[2])
    for _ in range(3):
        outs[2].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    h.free()


def test_capped_sms(ep):
    """num_sms bounds the grid: the few CTAs walk all tiles."""
    cfg = ep.make_config(300, 4, 16, 4, 256, 75, 1, do_expand=True, do_zero_padding=True,
                         num_sms=3)
    h = ep.ep_layout(cfg, routing(300, 4, 16, 3, 0.1).cuda())
    check(ep, h, 512, 384)
    h.free()


def test_refusals(ep):
    idx = routing(8, 2, 8, 1).cuda()
    h = ep.ep_layout(ep.make_config(8, 2, 8, 2, 128, 4, 1, do_expand=True), idx)
    q, sf = ep.alloc_fp8(h, 256)
    w, wsf = weights(8, 64, 256, 1)
    ep.ep_expert_gemm(h, q, sf, w, wsf)
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(h, q, sf, w[:4], wsf)  # not the handle's experts
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(h, q[:, :128].contiguous(), sf, w, wsf)
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(h, q, sf, w[:, :, :100].contiguous(), wsf)
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(h, q, sf, w, wsf[:, :, :1].contiguous())
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(h, q, sf, w.cpu(), wsf)
    with pytest.raises(ep.EpError) as e:
        ep.ep_expert_gemm(h, q, sf, w[:, :60].contiguous(), wsf)  # n = 60
    assert e.value.status == ep.EP_ERR_INVALID_ARG
    r = ep.ep_layout(ep.make_config(8, 2, 8, 2, 128, 4, 1), idx)
    q, sf = ep.alloc_fp8(r, 256)
    with pytest.raises(ep.EpError) as e:  # the rank layout has no expert segments
        ep.ep_expert_gemm(r, q, sf, w, wsf)
    assert e.value.status == ep.EP_ERR_UNSUPPORTED
    torch.cuda.synchronize()
