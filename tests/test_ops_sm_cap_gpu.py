"""GPU tests of cfg.num_sms in the operators that take a handle: no launch of a
call has more CTAs than that many SMs hold, and the results are those of a call
without a cap (each CTA then walks several tiles, tokens, chunks and shares)."""
import ctypes

import pytest
import torch

from tests.ops_harness import routing

pytestmark = pytest.mark.gpu
CTAS_PER_SM = 32  # what an SM of this architecture holds at most


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("args", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kernel", ctypes.c_void_p), ("context", ctypes.c_void_p)]


def grids(call):
    """Numbers of CTAs of the kernels that `call` launches, from a captured graph."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:  # a kernel
            p = _KernelNode()
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(p.grid[0] * p.grid[1] * p.grid[2])
    assert out
    return out


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def layouts(ep, T, K, E, H, cap, **kw):
    idx = routing(T, K, E, 23, 0.1).cuda()
    return [ep.ep_layout(ep.make_config(T, K, E, 2, H, T // 2, num_sms=c, **kw), idx)
            for c in (0, cap)]


def check(free, capped, cap):
    """free, capped: (call, its outputs) without and with the cap."""
    for call, outs in (free, capped):
        for o in outs:
            o.zero_()
        call()
    torch.cuda.synchronize()
    for a, b in zip(free[1], capped[1]):
        assert torch.equal(a, b)
    most = max(grids(free[0]))
    assert most > cap * CTAS_PER_SM, "the case is too small to show a cap"
    assert max(grids(capped[0])) <= cap * CTAS_PER_SM
    for o in capped[1]:
        o.zero_()
    capped[0]()
    torch.cuda.synchronize()
    for a, b in zip(free[1], capped[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cap", [1, 3])
@pytest.mark.parametrize("F", [128, 384])
def test_swiglu(ep, cap, F):
    hs = layouts(ep, 3000, 4, 16, 256, cap, expert_alignment=16, do_expand=True,
                 do_zero_padding=True, do_cpu_sync=True)
    rows = hs[0].rows_alloc
    g = torch.Generator().manual_seed(F)
    gu, w, ga = normal(g, rows, 2 * F, std=2.0), torch.randn(rows, generator=g).cuda(), normal(
        g, rows, F)
    ck = torch.zeros(rows, 2 * F, dtype=torch.uint8, device="cuda")
    cs = torch.zeros(rows, F // 64, device="cuda")
    ep.ep_swiglu(hs[0], gu, w, ckpt=ck, ckpt_sf=cs)

    def forward(h):
        act = torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda")
        q, sf = ep.alloc_fp8(h, F, zero=True)
        k, ks = torch.zeros_like(ck), torch.zeros_like(cs)
        return (lambda: ep.ep_swiglu(h, gu, w, act=act, act_fp8=q, act_sf=sf, ckpt=k, ckpt_sf=ks),
                (act, q, sf, k, ks))

    def backward(h):
        gh = torch.zeros(rows, 2 * F, dtype=torch.bfloat16, device="cuda")
        q, sf = ep.alloc_fp8(h, 2 * F, zero=True)
        gw = torch.zeros(rows, device="cuda")
        return (lambda: ep.ep_swiglu_backward(h, ga, ck, cs, w, grad_gate_up=gh, grad_fp8=q,
                                              grad_sf=sf, grad_row_weights=gw),
                (gh, q, sf, gw))

    check(*map(forward, hs), cap)
    check(*map(backward, hs), cap)
    for h in hs:
        h.free()


@pytest.mark.parametrize("cap", [1, 3])
@pytest.mark.parametrize("expand", [True, False])
@pytest.mark.parametrize("E,H", [(24, 384), (40, 2048)])
def test_combine_gradient(ep, cap, expand, E, H):
    """Rows, weights' gradients, sort, bias sums and their joining (both forms of it)."""
    T, K = 1700, 5
    hs = layouts(ep, T, K, E, H, cap, expert_alignment=8 if expand else 1, do_expand=expand,
                 do_zero_padding=expand, do_cpu_sync=True)
    rows = hs[0].rows_alloc
    g = torch.Generator().manual_seed(H)
    go, y, b = normal(g, T, H), normal(g, rows, H), normal(g, E, H)
    w = torch.randn(T, K, generator=g).cuda()

    def outputs(h):
        gy = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
        q, sf = ep.alloc_fp8(h, H, zero=True)
        gw, gb = torch.zeros(T, K, device="cuda"), torch.zeros(E, H, device="cuda")
        return (lambda: ep.ep_combine_weighted_backward(
            h, go, y, w, b, grad_y=gy, grad_y_fp8=q, grad_y_sf=sf, grad_topk_weights=gw,
            grad_expert_bias=gb), (gy, q, sf, gw, gb))

    check(*map(outputs, hs), cap)
    for h in hs:
        h.free()


@pytest.mark.parametrize("cap", [1, 3])
def test_product(ep, cap):
    T, K, E, n, k = 2600, 2, 4, 1032, 256
    hs = layouts(ep, T, K, E, 256, cap, expert_alignment=16, do_expand=True, do_zero_padding=True,
                 do_cpu_sync=True)
    rows = hs[0].rows_alloc
    g = torch.Generator().manual_seed(5)
    a = torch.randint(0, 120, (rows, k), generator=g, dtype=torch.uint8).cuda()
    w = torch.randint(0, 120, (E, n, k), generator=g, dtype=torch.uint8).cuda()
    wsf = torch.rand(E, -(-n // 128), k // 128, generator=g).cuda()
    _, sf = ep.alloc_fp8(hs[0], k)
    sf.fill_(0.25)

    def product(h):
        out = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
        return lambda: ep.ep_expert_gemm(h, a, sf, w, wsf, out=out), (out,)

    (free, fo), (capped, co) = map(product, hs)
    free()
    capped()
    torch.cuda.synchronize()
    assert torch.equal(fo[0], co[0]) and fo[0].any()
    assert max(grids(free)) > cap >= max(grids(capped))  # one CTA on an SM
    for h in hs:
        h.free()
