"""GPU tests of the operators' `stream=`: whose memory an output is, the
default stream named from another one, and the gated activation and the norm on
a side stream and in a CUDA graph."""
import pytest
import torch

from tests.ops_harness import routing

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


def owner(t: torch.Tensor) -> int:
    """Handle of the stream that the allocator keeps t's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("named", ["default", "zero", "side"])
def test_outputs_belong_to_the_stream_of_the_call(ep, named):
    """An output that the call allocates is of the stream that writes it: else the
    allocator may hand its memory out while that stream still runs."""
    g = torch.Generator().manual_seed(3)
    r, gy, gamma = normal(g, 64, 1024), normal(g, 64, 1024), normal(g, 1024)
    rstd = torch.rsqrt(r.float().square().mean(1) + EPS)
    want = ep.ep_rmsnorm_backward(gy, r, gamma, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream, current = {"default": (torch.cuda.default_stream(), side), "zero": (0, side),
                       "side": (side, torch.cuda.default_stream())}[named]
    with torch.cuda.stream(current):
        got = ep.ep_rmsnorm_backward(gy, r, gamma, rstd, stream=stream)
    torch.cuda.synchronize()
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    for a, b in zip(want, got):
        assert owner(b) == handle
        assert torch.equal(a, b)
