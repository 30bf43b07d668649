"""The example block with a trained shared expert beside the routed ones, forward,
backward and clipped, and a routed feed-forward block whose weights train: runs of
the operators together against fp32 autograd."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("tokens,hidden,ffn,experts,topk,shared", [
    (256, 512, 256, 16, 2, 264), (1, 256, 128, 8, 2, 128), (333, 384, 640, 12, 3, 1024),
    (1500, 256, 256, 4, 4, 72)])
def test_block_against_autograd(tokens, hidden, ffn, experts, topk, shared):
    from examples.moe_layer import MoeHalf, compare
    err = compare(MoeHalf(hidden, ffn, experts, topk, shared=shared), tokens, eight_bit=True)
    # an e4m3 rounding is 2.6% of a value in the mean, as without a shared expert
    assert err["residual"] < 2 ** -8
    assert err["out"] < 0.026 * 2
    for k in ("grad x", "grad gamma", "grad router"):
        assert err[k] < 0.026 * 5, (k, err)
    # BF16 only: roundings of the normed rows, of gate and up, of their gradient and of the
    # activation, at most 2^-8 of a value each; the gradient's factors pass on up to twice
    # what gate and up are off
    for k in ("grad shared in", "grad shared out"):
        assert err[k] < 8 * 2 ** -8, (k, err)


def test_without_a_shared_expert_nothing_changes():
    from examples.moe_layer import MoeHalf
    a, b = MoeHalf(256, 128, 8, 2), MoeHalf(256, 128, 8, 2, shared=64)
    x, r, go, gr = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(4))
    b.s_out.zero_()
    for m in (a, b):
        m.out, m.stream = m.forward(x, r, keep=True)
        m.grads = m.backward(go, gr)
    assert torch.equal(a.out, b.out) and torch.equal(a.stream, b.stream)
    assert len(a.grads) == 3 and len(b.grads) == 5
    for p, q in zip(a.grads, b.grads):
        assert torch.equal(p, q)


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clipped(max_norm):
    from examples.moe_layer import MoeHalf
    m = MoeHalf(256, 128, 8, 2, shared=128)
    x, r, go, gr = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(4))
    m.forward(x, r, keep=True)
    free = m.backward(go, gr)
    held = m.backward(go, gr, max_norm)
    norm = torch.stack([g.double().square().sum() for g in free[1:]]).sum().sqrt()
    assert abs(float(m.grad_norm) / float(norm) - 1) < 1e-5
    by = min(1.0, max_norm / (float(norm) + 1e-6))
    assert torch.equal(free[0], held[0])
    for a, b in zip(free[1:], held[1:]):
        assert torch.allclose(b.double(), a.double() * by, rtol=2 ** -8, atol=0)


@pytest.mark.parametrize("T,E,K,align,hidden,ffn", [
    (96, 8, 2, 16, 128, 200), (700, 4, 2, 1, 264, 136), (3, 16, 4, 8, 64, 64)])
def test_routed_block_that_trains(T, E, K, align, hidden, ffn):
    """Dispatch, gated product, down projection, combine, and all of it back: gradients of
    the tokens, the routing weights and the experts' matrices."""
    import combine_topk_idx_gb300 as ep
    from tests.ops_harness import routing
    g = torch.Generator().manual_seed(T)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).bfloat16().cuda()

    idx = routing(T, K, E, T).cuda()
    w = torch.softmax(torch.randn(T, K, generator=g), 1).cuda()
    x, go = normal(T, hidden), normal(T, hidden)
    w_in, w_out = normal(E, 2 * ffn, hidden, std=hidden ** -0.5), normal(E, hidden, ffn, std=ffn ** -0.5)
    cfg = ep.make_config(T, K, E, 1, hidden, T, align, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False)
    h = ep.ep_layout(cfg, idx)
    recv = ep.alloc_recv(h)
    ep.ep_dispatch(h, x, None, **recv)
    rows = h.rows_alloc
    gate_up = torch.empty(rows, 2 * ffn, dtype=torch.bfloat16, device="cuda")
    act = ep.ep_ffn_gated(h, recv["recv_x"], w_in, gate_up=gate_up)
    y = ep.ep_ffn_product(h, act, w_out)
    out = ep.ep_combine(h, y, w)
    # back
    gy = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
    gw = torch.empty_like(w)
    ep.ep_combine_weighted_backward(h, go, y, w, grad_y=gy, grad_topk_weights=gw)
    act_b = torch.empty_like(act)
    ggu = ep.ep_ffn_gated_backward(h, gy, w_out, gate_up, act=act_b)
    g_out = ep.ep_ffn_weight_grad(h, gy, act_b)
    g_in = ep.ep_ffn_weight_grad(h, ggu, recv["recv_x"])
    gx, _ = ep.ep_dispatch_backward(h, ep.ep_ffn_product(h, ggu, w_in, transposed=True))
    # once more into the same gradients, as a second micro-batch would
    twice = g_in.clone()
    ep.ep_ffn_weight_grad(h, ggu, recv["recv_x"], twice, accumulate=True)
    assert torch.allclose(twice, 2 * g_in, rtol=2 ** -22, atol=0)

    leaves = [t.float().requires_grad_() for t in (x, w, w_in, w_out)]
    xs, ws, a, b = leaves
    want = torch.zeros(T, hidden, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        gg, u = (xs[t] @ a[e].t()).chunk(2, 1)
        want = want.index_add(0, t, (torch.nn.functional.silu(gg) * u) @ b[e].t() * ws[t, k, None])
    want.backward(go.float())
    for got, ref, name in ((out, want, "out"), (gx, xs.grad, "x"), (gw, ws.grad, "w"),
                           (g_in, a.grad, "in"), (g_out, b.grad, "out")):
        off = float((got.float() - ref.detach()).norm() / ref.detach().norm())
        assert off < 8 * 2 ** -8, (name, off)  # a handful of BF16 roundings, at most 2^-8 each
    # all of it clipped
    norm = ep.ep_clip_grads([g_in, g_out], 0.25)
    assert abs(float(ep.ep_grad_norm([g_in, g_out])) - min(0.25, float(norm))) < 1e-5
    h.free()
