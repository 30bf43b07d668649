"""The example block: norm, dispatch, experts' products, activation, combine and
all their gradients run together, against fp32 autograd on the same weights."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,ffn,experts,topk,ranks", [
    (256, 512, 256, 16, 2, 4), (1, 256, 128, 8, 2, 1), (333, 384, 640, 12, 3, 2),
    (700, 256, 256, 4, 4, 1)])
def test_block_against_autograd(tokens, hidden, ffn, experts, topk, ranks):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from examples.moe_layer import MoeHalf, compare
    m = MoeHalf(hidden, ffn, experts, topk, ranks)
    # against the block with its experts' inputs in the same 8 bits: for few
    # tokens a weight's gradient, an inner product of nearly orthogonal rows,
    # can lie far from that of unrounded rows
    err = compare(m, tokens, eight_bit=True)
    # an e4m3 rounding is 2.6% of a value in the mean; the output passes two of
    # them, a gradient up to five, independent of one another
    assert err["residual"] < 2 ** -8
    assert err["out"] < 0.026 * 2
    for k in ("grad x", "grad gamma", "grad router"):
        assert err[k] < 0.026 * 5, (k, err)


def test_forward_without_keeping():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from examples.moe_layer import MoeHalf
    m = MoeHalf(256, 128, 8, 2)
    x, r = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(2))
    a, _ = m.forward(x, r)
    b, _ = m.forward(x, r, keep=True)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
