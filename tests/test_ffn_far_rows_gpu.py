"""GPU tests of the feed-forward products and of clipping on arrays of more than 2^31
elements: what lies behind them is right, and nothing is read or written at a wrapped
offset."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TAIL = 300


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


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)


def near(got, want):
    """Within a rounding of BF16 and the fp32 sums' error (both far below 2^-7 of the norm)."""
    assert float((got.float() - want).norm() / want.norm()) < 2 ** -8


def test_rows(ep):
    K, F = 2048, 1024
    T = 2 ** 31 // K + 1037
    x, w = normal(1, T, K), normal(2, 2 * F, K, std=K ** -0.5)
    gu = torch.empty(T, 2 * F, dtype=torch.bfloat16, device="cuda")
    act = ep.ep_ffn_gated(None, x, w, gate_up=gu)
    for s in (slice(0, TAIL), slice(T - TAIL, T)):
        h = x[s].float() @ w.float().t()
        near(gu[s], h)
        near(act[s], torch.nn.functional.silu(h[:, :F]) * h[:, F:])
    # back: of rows whose arrays are as long
    ggu = ep.ep_ffn_gated_backward(None, x, normal(3, K, F, std=K ** -0.5), gu)
    for s in (slice(0, TAIL), slice(T - TAIL, T)):
        d = x[s].float() @ normal(3, K, F, std=K ** -0.5).float()
        g, u = gu[s].float().chunk(2, 1)
        sig = torch.sigmoid(g)
        near(ggu[s], torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1))
    out = ep.ep_ffn_product(None, ggu, w, transposed=True, out=x)
    near(out[-TAIL:], ggu[-TAIL:].float() @ w.float())


def test_weight_grad_of_far_rows(ep):
    """Only the last rows hold anything: the sum is theirs."""
    n, k = 64, 2048
    T = 2 ** 31 // k + 1037
    a, g = torch.zeros(T, k, dtype=torch.bfloat16, device="cuda"), normal(5, T, n)
    a[-TAIL:] = normal(6, TAIL, k)
    near(ep.ep_ffn_weight_grad(None, g, a), g[-TAIL:].float().t() @ a[-TAIL:].float())


def test_weight_grad_of_many_experts(ep):
    """More than 2^31 elements of gradient."""
    E, n, k = 140, 4096, 4096
    idx = torch.arange(E, device="cuda")[:, None].repeat(2, 1).contiguous()
    h = ep.ep_layout(ep.make_config(2 * E, 1, E, 1, 128, 2 * E, 1, do_expand=True), idx)
    g, a = normal(7, 2 * E, n), normal(8, 2 * E, k)
    for kind in (torch.bfloat16, torch.float32):
        got = ep.ep_ffn_weight_grad(h, g, a, dtype=kind)
        for e in (0, 127, 128, 139):
            near(got[e], g[2 * e:2 * e + 2].float().t() @ a[2 * e:2 * e + 2].float())
        del got
    w = normal(9, E, n, k, std=k ** -0.5)
    y = ep.ep_ffn_product(h, a, w)
    z = ep.ep_ffn_product(h, g, w, transposed=True)
    for e in (0, 127, 128, 139):
        near(y[2 * e:2 * e + 2], a[2 * e:2 * e + 2].float() @ w[e].float().t())
        near(z[2 * e:2 * e + 2], g[2 * e:2 * e + 2].float() @ w[e].float())
    h.free()


def test_clip(ep):
    n = 2 ** 31 + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1000:] = normal(10, 1000)
    g[:7] = 2.0
    want = float(torch.cat([g[:7], g[-1000:]]).double().norm())
    out = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")[1:]
    norm = ep.ep_clip_grads([g], 1.0, out=[out])
    assert abs(float(norm) / want - 1) < 1e-5
    near(out[-1000:], g[-1000:].float() / want)
    near(out[:7], g[:7].float() / want)
    assert not out[7:-1000].any()
