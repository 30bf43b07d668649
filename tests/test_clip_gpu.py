"""GPU tests of the global gradient norm and of clipping against 64 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import ops_oracle as P
from tests.ops_harness import f64

pytestmark = pytest.mark.gpu
# fp32 sums of at most 66 squares (each rounding 2^-24), halved by the root, one
# rounding to fp32; then the factor's rounding and the product's
NORM = 34 * 2.0 ** -24
CLIP = NORM + 2 * 2.0 ** -24


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def tensors(sizes, seed, kinds=(torch.float32, torch.bfloat16), std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(kinds[i % len(kinds)]).cuda()
            for i, n in enumerate(sizes)]


def check(ep, grads, max_norm, out=None):
    before = [t.clone() for t in grads]
    norm = ep.ep_clip_grads(grads, max_norm, out=out)
    want = P.global_norm([f64(t) for t in before])
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(float(norm) - want) <= NORM * want + 2.0 ** -149
    c = max_norm / (want + 1e-6) if want + 1e-6 > max_norm else 1.0
    for i, (b, t) in enumerate(zip(before, grads if out is None else out)):
        half = 2.0 ** -8 if b.dtype == torch.bfloat16 else 2.0 ** -24
        tiny = 2.0 ** -133 if b.dtype == torch.bfloat16 else 2.0 ** -149
        w = f64(b) * c
        assert (np.abs(f64(t) - w) <= (half + CLIP) * np.abs(w) + tiny).all(), f"tensor {i}"
        if out is not None:
            assert torch.equal(grads[i], b)
    return norm


SIZES = {
    "one_value": [1],
    "one_each_type": [1, 1],
    "empty_ones": [0, 5, 0, 0, 7, 0],
    "odd": [1, 2, 3, 5, 7, 9, 15, 17, 31, 33, 255, 257],
    "chunk_ends": [8191, 8192, 8193, 16384, 16385, 24575],
    "just_a_small_table": [3] * 64,
    "more_than_a_small_table": [3] * 65,
    "many": [17 * (i % 40) + 1 for i in range(1024)],
    "two_launches": [i % 50 for i in range(2100)],
    "large": [3_000_001, 17, 5_000_000],
}


@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0])
@pytest.mark.parametrize("name", sorted(SIZES))
def test_in_place_and_into_others(ep, name, max_norm):
    grads = tensors(SIZES[name], 3)
    check(ep, grads, max_norm, [torch.full_like(t, 7.0) for t in grads])
    check(ep, grads, max_norm)


# one launch of a cluster up to 64 tensors that are not empty and 1024 pieces of 4 KB, each
# tensor rounded up to whole ones; else two launches
FORMS = {"all_pieces": ([1024 * 1024], torch.float32, 1),
         "a_value_more": ([1024 * 1024 + 1], torch.float32, 2),
         "all_tensors": ([15 * 2048 + 1] * 64 + [0, 0], torch.bfloat16, 1),
         "a_value_more_in_one": ([16 * 2048] * 63 + [16 * 2048 + 1], torch.bfloat16, 2),
         "a_tensor_more": ([0, 1] * 65, torch.bfloat16, 2)}


@pytest.mark.parametrize("name", sorted(FORMS))
def test_where_the_forms_meet(ep, name):
    from tests.test_ops_sm_cap_gpu import grids
    sizes, kind, launches = FORMS[name]
    grads = tensors(sizes, 21, (kind,))
    out = [torch.full_like(t, 7.0) for t in grads]
    check(ep, grads, 1.0, out)
    assert len(grids(lambda: ep.ep_clip_grads(grads, 1.0, out=out))) == launches


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_alignments(ep, kind, shift):
    """Views at every offset, outputs at another one; what lies around them stays."""
    g = torch.Generator().manual_seed(5)
    sizes = [1, 6, 7, 8, 9, 100, 8200, 20001]
    flat = (torch.randn(60000, generator=g) * 3).to(kind).cuda()
    for other in (shift, (shift + 3) % 8):
        to = torch.full((60000,), 7.0, dtype=kind, device="cuda")
        grads, outs, at, free = [], [], shift, torch.ones(60000, dtype=torch.bool)
        for n in sizes:
            grads.append(flat[at:at + n])
            outs.append(to[at - shift + other:at - shift + other + n])
            free[at - shift + other:at - shift + other + n] = False
            at += n + (n % 3)
        check(ep, grads, 1.0, outs)
        assert (to[free.cuda()] == 7).all()


@pytest.mark.parametrize("scale", [1e30, 1e37, 3e38, 1e-18, 1e-25, 1e-38, 1e-41])
def test_squares_outside_the_range(ep, scale):
    """Norms that fp32 holds though the squares leave its range."""
    g = torch.Generator().manual_seed(7)
    grads = [((torch.rand(n, generator=g) * 0.9 + 0.1) * scale).cuda() for n in (3, 8)]
    if scale < 1e38:
        grads += [(torch.randn(9, generator=g) * scale).bfloat16().cuda()]
    else:  # one value, so that the norm stays finite
        grads = [grads[0][:1].contiguous()]
    check(ep, grads, 1.0, [torch.empty_like(t) for t in grads])


def test_large_and_tiny_together(ep):
    big, small = torch.full((4,), 1e25).cuda(), torch.full((100,), 1e-25).cuda()
    assert abs(float(ep.ep_grad_norm([big, small])) / 2e25 - 1) < 1e-6
    mixed = torch.full((8192,), 1e-3)
    mixed[77] = 1e22
    assert abs(float(ep.ep_grad_norm([mixed.cuda()])) / 1e22 - 1) < 1e-6


def test_zero_gradients(ep):
    grads = [torch.zeros(100).cuda(), torch.zeros(9000).bfloat16().cuda()]
    assert float(ep.ep_clip_grads(grads, 1.0)) == 0.0
    assert not any(t.any() for t in grads)


def test_no_gradients(ep):
    assert float(ep.ep_clip_grads([], 1.0)) == 0.0
    assert float(ep.ep_grad_norm([torch.empty(0).cuda()])) == 0.0


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_values_that_are_not_finite(ep, kind):
    grads = [torch.ones(300, dtype=kind).cuda(), torch.ones(5, dtype=kind).cuda()]
    grads[0][7] = float("nan")
    out = [torch.empty_like(t) for t in grads]
    assert math.isnan(float(ep.ep_clip_grads(grads, 1.0, out=out)))
    assert all(t.isnan().all() for t in out)
    grads[0][7] = -float("inf")
    assert float(ep.ep_clip_grads(grads, 1.0, out=out)) == math.inf
    assert out[0][7].isnan() and not out[1].any() and not out[0][:7].any()


def test_norm_only(ep):
    grads = tensors([1000, 20000, 3], 9)
    before = [t.clone() for t in grads]
    want = P.global_norm([f64(t) for t in grads])
    into = torch.empty((), device="cuda")
    got = ep.ep_grad_norm(grads, norm=into)
    assert got is into and abs(float(got) - want) <= NORM * want
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_norm_of_overlapping_gradients(ep):
    """Nothing is written: each counts as often as it is listed."""
    a, b = tensors([1000, 9000], 10, (torch.float32,))
    grads = [a, a, b, b[500:], a[:7]]
    want = P.global_norm([f64(t) for t in grads])
    plan = ep.GradPlan(grads, clips=False)
    for given in (grads, plan):
        assert abs(float(ep.ep_grad_norm(given)) - want) <= NORM * want
    for given in (grads, plan):
        with pytest.raises(ValueError):
            ep.ep_clip_grads(given, 1.0)


def test_plan_is_used_again(ep):
    """A plan follows the values of its tensors."""
    grads = tensors([5000, 40, 8193], 11)
    plan = ep.plan_grads(grads)
    for seed in (12, 13):
        for t, v in zip(grads, tensors([5000, 40, 8193], seed)):
            t.copy_(v)
        check(ep, grads, 1.0, [torch.empty_like(t) for t in grads])
        n = ep.ep_clip_grads(plan, 0.5)
        after = ep.ep_grad_norm(plan)
        assert float(n) > 0.5 and abs(float(after) - 0.5) < 0.5 * 2 ** -7


def test_plan_keeps_the_memory_it_listed(ep):
    """A tensor that is given other memory: the plan works on the memory of before, which stays
    allocated, and on nobody else's."""
    grads = tensors([70000, 33], 14)
    first = list(grads)
    plan = ep.plan_grads(grads)
    want = float(ep.ep_grad_norm(plan))
    old = first[0].data
    at = old.data_ptr()
    first[0].data = torch.zeros_like(old)
    del old
    others = [torch.full_like(first[0], 9.0) for _ in range(8)]
    assert all(t.data_ptr() != at for t in others)
    assert float(ep.ep_clip_grads(plan, 0.5)) == want
    assert (first[0] == 0).all() and all((t == 9).all() for t in others)
    fresh = ep.plan_grads(grads)
    assert float(ep.ep_grad_norm(fresh)) < want


@pytest.mark.parametrize("which", ["grads", "out"])
@pytest.mark.parametrize("how", ["emptied", "emptied_and_filled", "grown"])
def test_plan_of_resized_storages_is_refused(ep, how, which):
    """Their memory may be anybody's."""
    grads = tensors([70000, 33], 15)
    out = [torch.zeros_like(t) for t in grads]
    plan, kept = ep.plan_grads(grads, out), ep.plan_grads(grads[1:])
    want = float(ep.ep_clip_grads(plan, 0.5))
    t = (grads if which == "grads" else out)[0]
    if how == "grown":
        t.resize_(200_000)
    else:
        t.untyped_storage().resize_(0)
    if how == "emptied_and_filled":
        t.untyped_storage().resize_(1000)
    with pytest.raises(ValueError, match="resized"):
        ep.ep_clip_grads(plan, 0.5)
    with pytest.raises(ValueError, match="resized"):
        ep.ep_grad_norm(plan)
    assert want > 0.5 and float(ep.ep_clip_grads(kept, 0.5)) > 0.5


def test_memory_in_use_on_another_stream_is_kept(ep):
    """A tensor leaves the listed memory, the plan is called on another stream and dropped:
    the memory is nobody else's before that stream is done with it."""
    grads = tensors([700_000, 33], 16)
    plan = ep.plan_grads(grads)
    size, at = grads[0].untyped_storage().nbytes(), grads[0].data_ptr()
    grads[0].data = torch.zeros(700_000, device="cuda")
    torch.cuda.synchronize()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # some 0.5 s
    ep.ep_clip_grads(plan, 0.5, stream=side)
    done.record(side)
    del plan
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not done.query()
    assert all(t.data_ptr() != at for t in others)
    torch.cuda.synchronize()


def test_same_bits(ep):
    grads = tensors([123457, 1000, 7, 300000], 17)
    got = []
    for _ in range(3):
        out = [torch.empty_like(t) for t in grads]
        got.append([ep.ep_clip_grads(grads, 1.0, out=out)] + out)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_streams_and_graph(ep):
    grads = tensors([70000, 33, 5], 19)
    plan_out = [torch.empty_like(t) for t in grads]
    plan = ep.plan_grads(grads, plan_out)
    want = ep.ep_clip_grads(plan, 1.0)
    wants = [t.clone() for t in plan_out]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in plan_out:
        t.zero_()
    torch.cuda.synchronize()
    n = ep.ep_clip_grads(plan, 1.0, stream=side)
    side.synchronize()
    assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(plan_out, wants))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    outs = [torch.empty_like(t) for t in grads]
    with torch.cuda.graph(graph):
        norm = ep.ep_clip_grads(plan, 1.0)
    with torch.cuda.graph(other):  # a second graph has a workspace of its own
        norm2 = ep.ep_clip_grads(grads, 2.0, out=outs)
    for _ in range(2):
        for t in plan_out + outs:
            t.zero_()
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and torch.equal(norm2, want)
        assert all(torch.equal(a, b) for a, b in zip(plan_out, wants))
    for t in grads:
        t.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) / (3 * float(want)) - 1) < 2 ** -7


def test_refusals(ep):
    a, b = torch.ones(8).cuda(), torch.ones(8).cuda()
    whole = torch.ones(16).cuda()
    for bad in (float("nan"), -1.0):
        with pytest.raises(ValueError):
            ep.ep_clip_grads([a], bad)
    for grads, out in (([a, a], None), ([whole, whole[4:]], None), ([a], [b, b]),
                       ([a], [torch.ones(9).cuda()]), ([a], [b.bfloat16()]),
                       ([a.cpu()], None), ([a.double()], None), ([a.half()], None),
                       ([whole[::2]], None), ([whole[:8]], [whole[4:12]]),
                       ([whole[:8], whole[8:]], [whole[8:], whole[:8]]),
                       ([a, b], [whole[:8], whole[7:15]])):
        with pytest.raises(ValueError):
            ep.plan_grads(grads, out)
    with pytest.raises(ValueError):
        ep.ep_clip_grads(ep.plan_grads([a]), 1.0, out=[b])
    with pytest.raises(ValueError):
        ep.ep_grad_norm([a], norm=torch.empty(1).cuda())
    ep.plan_grads([a, a], [b, whole[:8]])  # the same gradient twice, outputs apart
