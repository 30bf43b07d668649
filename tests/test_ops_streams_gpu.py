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


def layout(ep, **kw):
    cfg = ep.make_config(700, 4, 16, 4, 256, 175, 16, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False, **kw)
    return ep.ep_layout(cfg, routing(700, 4, 16, 31, 0.1).cuda())


def run_everywhere(call, outputs):
    """call(outputs, stream) on the current stream, on another one and captured in a
    graph that is replayed twice: the same bits."""
    want, side, graphed = outputs(), outputs(), outputs()
    call(want, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(side, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(graphed, None)
    for _ in range(2):
        for t in graphed.values():
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in want.items():
            if t is not None:
                assert t.any() and torch.equal(t, side[k]) and torch.equal(t, graphed[k]), k


@pytest.mark.parametrize("H,col", [(256, False), (1152, True), (7168, True)])
def test_norm(ep, H, col):
    g = torch.Generator().manual_seed(H)
    x, r, gamma = normal(g, 77, H), normal(g, 77, H), normal(g, H)
    run_everywhere(lambda o, s: ep.ep_rmsnorm(x, gamma, EPS, r, stream=s, **o),
                   lambda: ep.alloc_rmsnorm(x, residual=True, bf16=True, col_major_sf=col,
                                            rstd=True))


@pytest.mark.parametrize("F", [128, 1408])
def test_swiglu(ep, F):
    h = layout(ep, use_tma_aligned_col_major_sf=F == 128)
    rows = h.rows_alloc
    g = torch.Generator().manual_seed(F)
    gu, w = normal(g, rows, 2 * F, std=2.0), torch.randn(rows, generator=g).cuda()

    def outputs():
        q, sf = ep.alloc_fp8(h, F, zero=True)
        return dict(act=torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda"), act_fp8=q,
                    act_sf=sf, ckpt=torch.zeros(rows, 2 * F, dtype=torch.uint8, device="cuda"),
                    ckpt_sf=torch.zeros(rows, F // 64, device="cuda"))

    run_everywhere(lambda o, s: ep.ep_swiglu(h, gu, w, stream=s, **o), outputs)
    h.free()


@pytest.mark.parametrize("F", [128, 1408])
def test_swiglu_backward(ep, F):
    h = layout(ep, use_tma_aligned_col_major_sf=F == 128)
    rows = h.rows_alloc
    g = torch.Generator().manual_seed(F + 1)
    gu, ga = normal(g, rows, 2 * F, std=2.0), normal(g, rows, F)
    w = torch.randn(rows, generator=g).cuda()
    ck = torch.zeros(rows, 2 * F, dtype=torch.uint8, device="cuda")
    cs = torch.zeros(rows, F // 64, device="cuda")
    ep.ep_swiglu(h, gu, w, ckpt=ck, ckpt_sf=cs)

    def outputs():
        q, sf = ep.alloc_fp8(h, 2 * F, zero=True)
        return dict(grad_gate_up=torch.zeros(rows, 2 * F, dtype=torch.bfloat16, device="cuda"),
                    grad_fp8=q, grad_sf=sf, grad_row_weights=torch.zeros(rows, device="cuda"))

    run_everywhere(lambda o, s: ep.ep_swiglu_backward(h, ga, ck, cs, w, stream=s, **o), outputs)
    h.free()
