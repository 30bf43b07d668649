"""GPU tests of the operators on arrays of more than 2^31 elements: the last rows
are those of a call on these rows alone."""
import pytest
import torch

from tests.ops_harness import FP8

pytestmark = pytest.mark.gpu
EPS = 1e-6
TAIL = 50


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    yield ep
    torch.cuda.empty_cache()


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def test_norm(ep):
    H = 4096
    T = 2 ** 31 // H + 37
    x, gamma = normal(1, T, H), normal(2, H)
    out = ep.alloc_rmsnorm(x, residual=True, bf16=True, col_major_sf=True, rstd=True)
    ep.ep_rmsnorm(x, gamma, EPS, x, **out)
    xs = x[-TAIL:].contiguous()
    few = ep.alloc_rmsnorm(xs, residual=True, bf16=True, col_major_sf=True, rstd=True)
    ep.ep_rmsnorm(xs, gamma, EPS, xs, **few)
    torch.cuda.synchronize()
    for k, v in few.items():
        assert torch.equal(out[k][-TAIL:], v), k
    y, rstd = out["y"], out["rstd"]
    del out, few
    gx, _ = ep.ep_rmsnorm_backward(y, x, gamma, rstd)
    few, _ = ep.ep_rmsnorm_backward(y[-TAIL:], xs, gamma, rstd[-TAIL:].clone())
    torch.cuda.synchronize()
    assert torch.equal(gx[-TAIL:], few)


def test_swiglu(ep):
    F = 1024
    rows = 2 ** 31 // (2 * F) + 37
    h = normal(3, rows, 2 * F)

    def forward(h):
        n = h.shape[0]
        o = dict(act=torch.empty(n, F, dtype=torch.bfloat16, device="cuda"),
                 act_fp8=torch.empty(n, F, dtype=torch.uint8, device="cuda"),
                 act_sf=torch.empty(n, F // 128, device="cuda"),
                 ckpt=torch.empty(n, 2 * F, dtype=torch.uint8, device="cuda"),
                 ckpt_sf=torch.empty(n, F // 64, device="cuda"))
        ep.ep_swiglu(None, h, **o)
        return o

    def backward(o):
        n = o["act"].shape[0]
        g = dict(grad_gate_up=torch.empty(n, 2 * F, dtype=torch.bfloat16, device="cuda"),
                 grad_fp8=torch.empty(n, 2 * F, dtype=torch.uint8, device="cuda"),
                 grad_sf=torch.empty(n, F // 64, device="cuda"),
                 grad_row_weights=torch.empty(n, device="cuda"))
        ep.ep_swiglu_backward(None, o["act"], o["ckpt"], o["ckpt_sf"], **g)
        return g

    many, few = forward(h), forward(h[-TAIL:].contiguous())
    torch.cuda.synchronize()
    for k, v in few.items():
        assert torch.equal(many[k][-TAIL:], v), k
    del h
    many, few = backward(many), backward(few)
    torch.cuda.synchronize()
    for k, v in few.items():
        assert torch.equal(many[k][-TAIL:], v), k


def test_combine_gradient_and_product(ep):
    """Eight experts that every token goes to: the last tokens of the last expert
    have the last rows."""
    T, K, H, n = 66000, 8, 4096, 4104
    idx = torch.arange(K, device="cuda").expand(T, K).contiguous()
    h = ep.ep_layout(ep.make_config(T, K, K, 1, H, T, 1, do_expand=True), idx)
    rows = h.rows_alloc
    assert rows == T * K and rows * H > 2 ** 31
    go, y = normal(4, T, H), normal(5, rows, H)
    w = torch.rand(T, K, device="cuda")
    gy = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    q, sf = ep.alloc_fp8(h, H)
    gw = torch.empty(T, K, device="cuda")
    ep.ep_combine_weighted_backward(h, go, y, w, grad_y=gy, grad_y_fp8=q, grad_y_sf=sf,
                                    grad_topk_weights=gw)
    t = slice(T - TAIL, T)
    small = ep.ep_layout(ep.make_config(TAIL, K, K, 1, H, TAIL, 1, do_expand=True),
                         idx[:TAIL].contiguous())
    dst = h.tensor("dst_buffer_slot_idx")[t].long().t().reshape(-1)  # expert by expert, as small's
    assert int(dst[-1]) == rows - 1
    gy2, gw2 = torch.empty(TAIL * K, H, dtype=torch.bfloat16, device="cuda"), torch.empty(
        TAIL, K, device="cuda")
    q2, sf2 = ep.alloc_fp8(small, H)
    ep.ep_combine_weighted_backward(small, go[t].contiguous(), y[dst].contiguous(),
                                    w[t].contiguous(), grad_y=gy2, grad_y_fp8=q2, grad_y_sf=sf2,
                                    grad_topk_weights=gw2)
    torch.cuda.synchronize()
    assert torch.equal(gy[dst], gy2) and torch.equal(gw[t], gw2) and torch.equal(q[dst], q2)
    assert torch.equal(sf.view(rows, -1)[dst], sf2.view(TAIL * K, -1))
    del y, gy
    g = torch.Generator(device="cuda").manual_seed(6)
    we = (torch.randn(K, n, H, generator=g, device="cuda") * 90).clamp(-448, 448).to(FP8).view(
        torch.uint8)
    wsf = torch.rand(K, -(-n // 128), H // 128, generator=g, device="cuda")
    out = ep.ep_expert_gemm(h, q, sf, we, wsf)
    few = ep.ep_expert_gemm(small, q2, sf2, we, wsf)
    torch.cuda.synchronize()
    assert rows * n > 2 ** 31 and torch.equal(out[dst], few) and few.any()
    h.free()
    small.free()
