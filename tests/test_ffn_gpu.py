"""GPU tests of the feed-forward block's products (ep_ffn_*) against their 64-bit
definitions: one matrix and all rows, and one matrix per expert of a layout."""
import pytest
import torch

from tests.ffn_harness import OPS, check, make_handle, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


# rows, n (ffn), k: single rows, ends inside a tile, a block and a 16-byte group,
# few and many tiles, a long reduction
DENSE = [(1, 128, 64), (1, 8, 8), (8, 24, 40), (9, 40, 2056), (4, 2504, 104), (1, 520, 1032), (2, 256, 4096), (16, 136, 200), (17, 264, 128),
         (127, 128, 64), (128, 256, 256), (129, 248, 264), (300, 392, 72), (1000, 1000, 328),
         (513, 2056, 192), (64, 512, 7168), (2500, 16, 24)]


@pytest.mark.parametrize("rows,n,k", DENSE)
@pytest.mark.parametrize("op", OPS)
def test_one_matrix(ep, op, rows, n, k):
    check(ep, op, None, rows, n, k, seed=rows + n)


# 129 to some 600 rows: a long reduction is shared by four pairs of CTAs, or two, with rows and
# columns that end inside a tile; and tiles of single CTAs where those of pairs need a round more
SOME_HUNDRED = [(250, 2568, 6200), (129, 3400, 3208), (300, 3400, 3208), (520, 2600, 3200),
                (600, 6704, 200)]


@pytest.mark.parametrize("rows,n,k", SOME_HUNDRED)
@pytest.mark.parametrize("op", ["gated", "gated_bwd", "product", "product_t"])
def test_some_hundred_rows(ep, op, rows, n, k):
    # half as many columns for gate and up, which share a tile
    check(ep, op, None, rows, n // 16 * 8 if op == "gated" else n, k, seed=rows)


@pytest.mark.parametrize("op", ["gated", "gated_bwd", "product", "product_t"])
def test_some_hundred_rows_in_graphs(ep, op):
    """The shared reduction gives the same bits eagerly, on another stream and replayed."""
    call, outputs = calls(ep, None, 300, 3400, 3208)[op]
    want, side, again = (outputs() for _ in range(3))
    call(want, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(side, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(again, None)
    for _ in range(2):
        for t in again.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for name, t in want.items():
            assert torch.equal(side[name], t) and torch.equal(again[name], t)


# name: (T, K, E, R, M, A, zero_pad, sync, fixed, drop, n, k)
LAYOUTS = {
    "one_row": (1, 1, 1, 1, 1, 1, True, True, False, 0.0, 256, 128),
    "one_token": (1, 8, 64, 8, 1, 1, True, True, False, 0.0, 512, 1024),
    "few_slots": (5, 3, 16, 4, 2, 16, True, True, False, 0.1, 136, 264),
    "few_slots_bound": (2, 4, 300, 4, 1, 100, True, False, False, 0.2, 72, 520),
    "few_slots_unpadded": (3, 2, 8, 2, 2, 8, False, True, False, 0.0, 40, 1032),
    "few_slots_fixed": (6, 2, 8, 2, 3, 1, False, False, True, 0.0, 200, 72),
    "sixteen_slots_one_expert": (16, 1, 1, 1, 16, 32, True, True, False, 0.0, 264, 328),
    "aligned": (300, 4, 16, 4, 75, 128, True, True, False, 0.1, 384, 512),
    "align_256": (90, 2, 4, 2, 45, 256, True, True, False, 0.1, 256, 384),
    "unaligned_rows": (333, 4, 16, 4, 90, 1, True, True, False, 0.1, 640, 256),
    "no_zero": (100, 3, 8, 2, 50, 16, False, True, False, 0.1, 256, 392),
    "upper_bound": (90, 4, 32, 4, 25, 8, True, False, False, 0.2, 264, 136),
    "fixed": (61, 4, 16, 4, 16, 1, False, False, True, 0.1, 256, 200),
    "fixed_odd": (64, 2, 8, 2, 200, 1, False, False, True, 0.0, 136, 72),
    "no_rows": (9, 2, 8, 2, 5, 4, True, True, False, 1.0, 256, 128),
    "all_dropped_bound": (9, 2, 8, 2, 5, 4, True, False, False, 1.0, 64, 128),
    "many_experts": (300, 2, 512, 4, 100, 1, True, True, False, 0.0, 32, 40),
    "long_segments": (1500, 1, 2, 1, 1500, 16, True, True, False, 0.0, 328, 264),
}


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("op", OPS)
def test_layouts(ep, op, name):
    T, K, E, R, M, A, zp, sync, fixed, drop, n, k = LAYOUTS[name]
    h = make_handle(ep, T, K, E, R, M, A, zp, sync, fixed, drop)
    check(ep, op, h, h.rows_alloc, n, k)
    h.free()


# no tokens: rows are allocated (fixed slabs, an upper bound with alignment) and none is in use
NO_TOKENS = {"fixed": (1, False, False, True), "bound": (8, True, False, False),
             "bound_unpadded": (100, False, False, False), "no_rows": (8, True, True, False)}


@pytest.mark.parametrize("name", sorted(NO_TOKENS))
@pytest.mark.parametrize("op", OPS)
def test_no_tokens(ep, op, name):
    A, zp, sync, fixed = NO_TOKENS[name]
    h = make_handle(ep, 0, 2, 4, 2, 16, A, zp, sync, fixed)
    assert (h.rows_alloc == 0) == (name == "no_rows")
    check(ep, op, h, h.rows_alloc, 136, 72)
    h.free()


# more rows per expert than a pair of CTAs takes alone, several tiles of each, a last round
# of halved tiles, reductions over several joins
WIDE = {"two_experts": (1300, 1, 2, 1, 1300, 16, 520, 200),
        "uneven": (900, 2, 4, 2, 450, 1, 264, 136),
        "one_expert": (4200, 1, 1, 1, 4200, 128, 72, 264),
        "many_tiles": (700, 3, 3, 1, 700, 1, 2312, 128)}


@pytest.mark.parametrize("name", sorted(WIDE))
@pytest.mark.parametrize("op", OPS)
def test_many_rows_per_expert(ep, op, name):
    T, K, E, R, M, A, n, k = WIDE[name]
    h = make_handle(ep, T, K, E, R, M, A, drop=0.05)
    check(ep, op, h, h.rows_alloc, n, k, seed=3)
    h.free()


@pytest.mark.parametrize("op", OPS)
def test_overflowing_layout(ep, op):
    """Rows dropped by an overflowing upper bound are not touched."""
    cfg = ep.make_config(2, 4, 2, 2, 128, 1, 1, do_expand=True, do_zero_padding=True,
                         do_cpu_sync=False)
    h = ep.ep_layout(cfg, torch.tensor([[0, 0, 0, 0], [1, 1, 0, 0]]).cuda())
    check(ep, op, h, h.rows_alloc, 136, 72)
    h.free()


@pytest.mark.parametrize("rows", [5, 200, 1000])
@pytest.mark.parametrize("keep", [True, False])
def test_outputs_left_out(ep, rows, keep):
    check(ep, "gated", None, rows, 264, 128, keep=keep)
    check(ep, "gated_bwd", None, rows, 264, 128, keep=keep)
    g = torch.Generator().manual_seed(1)
    x, w = normal(g, rows, 128).cuda(), normal(g, 528, 128).cuda()
    act = ep.ep_ffn_gated(None, x, w)
    gu = torch.empty(rows, 528, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(act, ep.ep_ffn_gated(None, x, w, gate_up=gu))


# sums of so many rows that they are joined of parts (131072 rows each): one matrix shared by a
# cluster, by pairs; a layout's by pairs and by single CTAs (num_sms 1; few slots per expert).
# name: (experts, rows, n, k, num_sms)
LONG = {"cluster": (0, (1 << 22) + 37, 40, 24, 0), "just_more": (0, 131073, 72, 48, 0),
        "tiles": (0, 300_001, 1160, 1160, 0), "pairs": (2, (1 << 21) + 5, 40, 264, 0),
        "pairs_aligned": (3, (1 << 21) + 5, 136, 272, 0), "ctas": (2, (1 << 21) + 5, 40, 264, 1),
        "ctas_aligned": (1, 1 << 21, 136, 272, 1), "many_experts": (1024, 140_001, 24, 40, 0)}


@pytest.mark.parametrize("name", sorted(LONG))
def test_weight_gradient_of_very_many_rows(ep, name):
    """Sums of one sign: what the tensor cores cut off adds up, at most two units (2^-23) of the
    sum so far every 16 rows, half of that on average over a growing sum, so 2^-10 in a part."""
    E, T, n, k, sms = LONG[name]
    gen = torch.Generator(device="cuda").manual_seed(T)
    h, rows, starts, counts = None, T, [0], [T]
    if E:
        idx = torch.full((T, 1), E // 2, dtype=torch.int64, device="cuda")
        idx[:1000] = 0
        h = ep.ep_layout(ep.make_config(T, 1, E, 1, 128, T, 1, do_expand=True, num_sms=sms), idx)
        rows, starts = h.rows_alloc, h.tensor("psum_expert").tolist()[:-1]
        counts = h.tensor("cnt_expert").tolist()
    g, a = (torch.rand(rows, c, generator=gen, device="cuda").bfloat16() for c in (n, k))
    for accumulate in (False, True):
        lead = () if h is None else (E,)
        got = torch.full((*lead, n, k), 64.0, dtype=torch.bfloat16, device="cuda")
        ep.ep_ffn_weight_grad(h, g, a, got, accumulate=accumulate)
        for e in {0, E // 2}:
            s = slice(starts[e], starts[e] + counts[e])
            want = sum(g[i:min(i + 65536, s.stop)].double().t() @ a[i:min(i + 65536, s.stop)].double()
                       for i in range(s.start, s.stop, 65536))
            want += 64.0 * accumulate
            err = ((got if h is None else got[e]).double() - want).abs()
            assert (err <= (2.0 ** -8 * (1 + 2.0 ** -9) + 2.0 ** -10 + 2.0 ** -18) * want).all(), (
                e, float((err / want).max()))
        if E > 3:
            assert (got[3] == (64 if accumulate else 0)).all()  # no rows
    if h is not None:
        assert int(h.tensor("error_word")[0]) & ep.EP_ERRBIT_TIMEOUT == 0
        h.free()


# name: (experts, n, k, num_sms): a cluster shares the sum, tiles of pairs, a layout's by pairs and
# by single CTAs
JOINED = {"cluster": (0, 40, 24, 0), "tiles": (0, 1160, 1160, 0), "pairs": (2, 264, 136, 0),
          "ctas": (2, 264, 136, 1)}


@pytest.mark.parametrize("name", sorted(JOINED))
def test_weight_gradient_in_32_bits_is_joined(ep, name):
    """Sums of one sign, where what the tensor cores cut off adds up.  An accumulator takes 512
    rows: 32 times at most two units (2^-23) of a sum that grows, 33 * 2^-23 in all; the parts
    are added up in fp32, 2^-24 of the sum so far each (and of a cluster's four at the end).
    Not joined, 16397 rows are off by 7.5e-5, shared by four by 1.2e-5; the bound is 5.2e-6."""
    E, n, k, sms = JOINED[name]
    T = 16397
    gen = torch.Generator(device="cuda").manual_seed(n)
    h, rows, starts, counts = None, T, [0], [T]
    if E:
        idx = torch.zeros(T + 700, 1, dtype=torch.int64, device="cuda")
        idx[:T] = 1
        h = ep.ep_layout(ep.make_config(T + 700, 1, E, 1, 128, T + 700, 1, do_expand=True,
                                        num_sms=sms), idx)
        rows, starts = h.rows_alloc, h.tensor("psum_expert").tolist()[:-1]
        counts = h.tensor("cnt_expert").tolist()
    g, a = (torch.rand(rows, c, generator=gen, device="cuda").bfloat16() for c in (n, k))
    got = ep.ep_ffn_weight_grad(h, g, a)
    for e, (start, count) in enumerate(zip(starts, counts)):
        s = slice(start, start + count)
        want = g[s].double().t() @ a[s].double()
        err = ((got if h is None else got[e]).double() - want).abs() / want
        parts = -(-count // 512)
        assert float(err.max()) < 33 * 2.0 ** -23 + (parts / 2 + 5) * 2.0 ** -24, (e, float(err.max()))
    if h is not None:
        h.free()


def calls(ep, h, rows, n, k, seed=9):
    """{name: call of (outputs, stream)} and the outputs of each, for one set of inputs."""
    g = torch.Generator().manual_seed(seed)
    lead = () if h is None else (h.E,)
    x, gy, gu = (normal(g, rows, c).cuda() for c in (k, n, 2 * n))
    w_in, w_out, w = (normal(g, *lead, *s, std=0.05).cuda()
                      for s in ((2 * n, k), (n, n), (n, k)))

    def zeros(*shape, kind=torch.bfloat16):
        return torch.zeros(*shape, dtype=kind, device="cuda")

    return {
        "gated": (lambda o, s: ep.ep_ffn_gated(h, x, w_in, stream=s, **o),
                  lambda: dict(act=zeros(rows, n), gate_up=zeros(rows, 2 * n))),
        "gated_bwd": (lambda o, s: ep.ep_ffn_gated_backward(h, gy, w_out, gu, stream=s, **o),
                      lambda: dict(grad_gate_up=zeros(rows, 2 * n), act=zeros(rows, n))),
        "product": (lambda o, s: ep.ep_ffn_product(h, x, w, stream=s, **o),
                    lambda: dict(out=zeros(rows, n))),
        "product_t": (lambda o, s: ep.ep_ffn_product(h, gy, w, transposed=True, stream=s, **o),
                      lambda: dict(out=zeros(rows, k))),
        "wgrad": (lambda o, s: ep.ep_ffn_weight_grad(h, gy, x, stream=s, **o),
                  lambda: dict(grad_w=zeros(*lead, n, k, kind=torch.float32))),
        "wgrad_bf16": (lambda o, s: ep.ep_ffn_weight_grad(h, gy, x, stream=s, **o),
                       lambda: dict(grad_w=zeros(*lead, n, k))),
    }


@pytest.mark.parametrize("form", ["single", "few_rows", "tens", "dense", "layout",
                                  "layout_many_rows"])
@pytest.mark.parametrize("op", OPS)
def test_streams_and_graphs(ep, op, form):
    """The same bits on the current stream, on another one, in a graph that is replayed, and
    in a second graph beside it."""
    h = None
    if form.startswith("layout"):
        T, E = (300, 8) if form == "layout" else (1200, 2)
        h = make_handle(ep, T, 2, E, 1, T, 16)
    rows = {"single": 1, "few_rows": 11, "tens": 40, "dense": 1500}.get(form) or h.rows_alloc
    call, outputs = calls(ep, h, rows, 264, 328)[op]
    want, side, first, second = (outputs() for _ in range(4))
    call(want, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(side, s)
    s.synchronize()
    graphs = []
    for o in (first, second):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(o, None)
    for _ in range(2):
        for o in (first, second):
            for t in o.values():
                t.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for graph, q in zip(graphs, streams):
            with torch.cuda.stream(q):
                graph.replay()
        torch.cuda.synchronize()
        for k, t in want.items():
            assert t.any()
            assert torch.equal(t, side[k]) and torch.equal(t, first[k]) and torch.equal(t, second[k])
    if h is not None:
        h.free()


@pytest.mark.parametrize("op", OPS)
def test_allocated_outputs_belong_to_the_stream(ep, op):
    side = torch.cuda.Stream()
    call, outputs = calls(ep, None, 70, 136, 72)[op]
    want = outputs()
    call(want, None)
    torch.cuda.synchronize()
    o = {"dtype": torch.bfloat16} if op == "wgrad_bf16" else {}
    got = call(o, side)
    side.synchronize()
    main = "grad_gate_up" if op == "gated_bwd" else next(iter(want))
    assert torch.equal(got, want[main])
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= got.data_ptr() < seg["address"] + seg["total_size"]:
            assert seg["stream"] == side.cuda_stream


@pytest.mark.parametrize("rows", [1, 11, 30, 700])
def test_strided_rows(ep, rows):
    """Arrays of rows inside wider ones."""
    g = torch.Generator().manual_seed(4)
    n, k = 136, 200
    wide = [normal(g, rows, c + 40).cuda() for c in (k, n)]
    x, gy = wide[0][:, 16:16 + k], wide[1][:, 24:24 + n]
    xc, gc = x.contiguous(), gy.contiguous()
    w_in, w, gu = (normal(g, *s).cuda() for s in ((2 * n, k), (n, k), (rows, 2 * k)))
    assert torch.equal(ep.ep_ffn_gated(None, x, w_in), ep.ep_ffn_gated(None, xc, w_in))
    assert torch.equal(ep.ep_ffn_product(None, x, w), ep.ep_ffn_product(None, xc, w))
    assert torch.equal(ep.ep_ffn_gated_backward(None, gy, w, gu),
                       ep.ep_ffn_gated_backward(None, gc, w, gu))
    for kind in (torch.float32, torch.bfloat16):
        assert torch.equal(ep.ep_ffn_weight_grad(None, gy, x, dtype=kind),
                           ep.ep_ffn_weight_grad(None, gc, xc, dtype=kind))


@pytest.mark.parametrize("rows", [3, 11, 30, 700])
@pytest.mark.parametrize("op", OPS)
def test_alignment_of_outputs(ep, op, rows):
    """Outputs that start on 16 bytes, not 32, hold the same; what lies around them stays."""
    call, outputs = calls(ep, None, rows, 272, 144)[op]
    want = outputs()
    call(want, None)
    for off in (8, 4) if op == "wgrad" else (8,):
        flat, got = {}, {}
        for name, t in want.items():
            flat[name] = torch.full((t.numel() + 48,), 7.0, dtype=t.dtype, device="cuda")
            got[name] = flat[name][off:off + t.numel()].view(t.shape)
        call(got, None)
        for name, t in want.items():
            assert torch.equal(got[name], t)
            assert (flat[name][:off] == 7).all() and (flat[name][off + t.numel():] == 7).all()


@pytest.mark.parametrize("width", [264, 272])
@pytest.mark.parametrize("form", ["dense", "layout", "layout_many_rows"])
@pytest.mark.parametrize("op", ["gated", "gated_bwd"])
def test_alignment_of_one_output(ep, op, form, width):
    """One of two outputs starts on 16 bytes, not 32, the other where it is allocated."""
    h = None
    if form != "dense":
        T, E = (300, 8) if form == "layout" else (1200, 2)
        h = make_handle(ep, T, 2, E, 1, T, 16)
    rows = 900 if h is None else h.rows_alloc
    call, outputs = calls(ep, h, rows, width, 144)[op]
    want = outputs()
    call(want, None)
    for moved in want:
        got = outputs()
        flat = torch.full((got[moved].numel() + 48,), 7.0, dtype=torch.bfloat16, device="cuda")
        n = got[moved].numel()
        flat[8:8 + n] = 0
        got[moved] = flat[8:8 + n].view(want[moved].shape)
        call(got, None)
        for name, t in want.items():
            assert torch.equal(got[name], t)
        assert (flat[:8] == 7).all() and (flat[8 + n:] == 7).all()


@pytest.mark.parametrize("form", ["dense", "layout", "layout_many_rows"])
def test_alignment_of_the_kept_values(ep, form):
    h = None
    if form != "dense":
        T, E = (300, 8) if form == "layout" else (1200, 2)
        h = make_handle(ep, T, 2, E, 1, T, 16)
    rows, n = 900 if h is None else h.rows_alloc, 272
    g = torch.Generator().manual_seed(12)
    gy, gu = normal(g, rows, n).cuda(), normal(g, rows, 2 * n).cuda()
    w = normal(g, *(() if h is None else (h.E,)), n, n, std=0.05).cuda()
    moved = torch.empty(gu.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(gu.shape)
    moved.copy_(gu)
    want, got = (torch.zeros_like(gu) for _ in range(2))
    ep.ep_ffn_gated_backward(h, gy, w, gu, grad_gate_up=want)
    ep.ep_ffn_gated_backward(h, gy, w, moved, grad_gate_up=got)
    assert torch.equal(got, want)


@pytest.mark.parametrize("op", ["gated", "gated_bwd", "product", "product_t"])
@pytest.mark.parametrize("T", [60, 1000])
def test_other_experts_weights(ep, op, T):
    """Infinities and NaN in an expert's matrix reach its own rows only."""
    h = make_handle(ep, T, 1, 4, 1, T, 1, seed=2)
    rows, n, k = h.rows_alloc, 72, 40
    g = torch.Generator().manual_seed(6)
    x, gu = normal(g, rows, k).cuda(), normal(g, rows, 2 * n).cuda()
    shape = {"gated": (2 * n, k), "gated_bwd": (k, n), "product": (n, k), "product_t": (k, n)}[op]
    w = normal(g, 4, *shape).cuda()
    bad = w.clone()
    bad[1], bad[3] = float("nan"), float("inf")
    run = {"gated": lambda w: ep.ep_ffn_gated(h, x, w),
           "gated_bwd": lambda w: ep.ep_ffn_gated_backward(h, x, w, gu),
           "product": lambda w: ep.ep_ffn_product(h, x, w),
           "product_t": lambda w: ep.ep_ffn_product(h, x, w, transposed=True)}[op]
    psum = h.tensor("psum_expert").tolist()
    a, b = run(w), run(bad)
    for e in range(4):
        rows_e = slice(psum[e], psum[e + 1])
        if e in (1, 3):
            assert not torch.isfinite(b[rows_e]).all()
        else:
            assert torch.equal(a[rows_e], b[rows_e])
    h.free()


def test_values_that_are_not_finite(ep):
    """They stay in their row and column."""
    g = torch.Generator().manual_seed(8)
    for rows in (5, 12, 20, 900):
        x, w = normal(g, rows, 64).cuda(), normal(g, 256, 64).cuda()
        want = ep.ep_ffn_product(None, x, w)
        x[3, 5], w[7, 9] = float("nan"), float("inf")
        got = ep.ep_ffn_product(None, x, w)
        keep = torch.ones(rows, 256, dtype=torch.bool, device="cuda")
        keep[3], keep[:, 7] = False, False
        assert torch.equal(got[keep], want[keep])
        assert got[3].isnan().all() and not torch.isfinite(got[:, 7]).any()
        grad = ep.ep_ffn_weight_grad(None, want, x)
        assert grad[:, 5].isnan().all() and torch.isfinite(grad[:, :5]).all()


def test_gates_at_the_ends(ep):
    """The activation's gradient where the sigmoid is 0 or 1, and at 0."""
    n = 8
    g = torch.tensor([0.0, -0.0, 30.0, -30.0, 120.0, -120.0, 1e30, -1e30])
    gu = torch.cat([g, torch.full((n,), 2.0)])[None].bfloat16().cuda()
    w = torch.eye(n, dtype=torch.bfloat16, device="cuda")
    gy = torch.full((1, n), 3.0, dtype=torch.bfloat16, device="cuda")
    act = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    got = ep.ep_ffn_gated_backward(None, gy, w, gu, act=act)[0].double().cpu()
    v = gu[0, :n].double().cpu()
    s = torch.sigmoid(v)
    # where exp overflows fp32 the gate's sigmoid is 0 and not its tiny value
    want = torch.cat([6 * s * (1 + v * (1 - s)), 3 * v * s])
    assert torch.allclose(got, want, rtol=2 ** -8, atol=1e-10)
    assert torch.allclose(act[0].double().cpu(), 2 * v * s, rtol=2 ** -8, atol=1e-10)


@pytest.mark.parametrize("op", OPS)
def test_no_rows(ep, op):
    call, outputs = calls(ep, None, 0, 72, 40)[op]
    o = {k: t + 1 for k, t in outputs().items()}
    call(o, None)
    for t in o.values():
        assert not t.any() or t.numel() == 0
    if op.startswith("wgrad"):
        t = outputs()["grad_w"] + 1
        e = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
        a = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        ep.ep_ffn_weight_grad(None, e, a, t, accumulate=True)
        assert (t == 1).all()


def test_refusals(ep):
    def b(*s):
        return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    h = make_handle(ep, 20, 2, 4, 1, 20, 4)
    rank = ep.ep_layout(ep.make_config(20, 2, 4, 1, 128, 20),
                        torch.zeros(20, 2, dtype=torch.int64, device="cuda"))
    r = h.rows_alloc
    for bad in (lambda: ep.ep_ffn_gated(None, b(4, 16), b(15, 16)),        # no two halves
                lambda: ep.ep_ffn_gated(None, b(4, 16), b(4, 32, 16)),     # experts without a handle
                lambda: ep.ep_ffn_gated(h, b(r, 16), b(32, 16)),
                lambda: ep.ep_ffn_gated(h, b(r, 16), b(3, 32, 16)),
                lambda: ep.ep_ffn_gated(h, b(r + 1, 16), b(4, 32, 16)),
                lambda: ep.ep_ffn_gated(None, b(4, 24), b(32, 16)),
                lambda: ep.ep_ffn_gated(None, b(4, 16).float(), b(32, 16)),
                lambda: ep.ep_ffn_gated(None, b(4, 16), b(32, 16).float()),
                lambda: ep.ep_ffn_gated(None, b(4, 16), b(16, 32).t()),
                lambda: ep.ep_ffn_gated(None, b(16, 4).t(), b(32, 16)),
                lambda: ep.ep_ffn_gated(None, b(4, 16), b(32, 16), act=b(4, 32)),
                lambda: ep.ep_ffn_gated(None, b(4, 16), b(32, 16), gate_up=b(4, 16)),
                lambda: ep.ep_ffn_gated(None, b(4, 16).cpu(), b(32, 16)),
                lambda: ep.ep_ffn_gated(None, b(16), b(32, 16)),
                lambda: ep.ep_ffn_gated_backward(None, b(4, 16), b(16, 8), b(4, 8)),
                lambda: ep.ep_ffn_gated_backward(None, b(4, 16), b(8, 16), b(4, 32)),
                lambda: ep.ep_ffn_product(None, b(4, 16), b(8, 24)),
                lambda: ep.ep_ffn_product(None, b(4, 16), b(8, 16), transposed=True),
                lambda: ep.ep_ffn_weight_grad(None, b(4, 16), b(5, 16)),
                lambda: ep.ep_ffn_weight_grad(None, b(4, 16), b(4, 8), accumulate=True),
                lambda: ep.ep_ffn_weight_grad(None, b(4, 16), b(4, 8), b(8, 16)),
                lambda: ep.ep_ffn_weight_grad(None, b(4, 16), b(4, 8), dtype=torch.float16),
                lambda: ep.ep_ffn_weight_grad(h, b(r, 16), b(r, 8), b(16, 8))):
        with pytest.raises(ValueError):
            bad()
    for bad, status in (
            (lambda: ep.ep_ffn_gated(None, b(4, 12), b(32, 12)), ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_gated(None, b(4, 16), b(24, 16)), ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_product(None, b(4, 20), b(8, 20)), ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_product(None, b(4, 28)[:, :16], b(8, 16)), ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_product(None, b(4, 32)[:, 4:20], b(8, 16)), ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_product(None, b(1, 16).expand(4, 16), b(8, 16)),
             ep.EP_ERR_INVALID_ARG),
            (lambda: ep.ep_ffn_product(None, b(2, 65544), b(8, 65544)), ep.EP_ERR_UNSUPPORTED),
            (lambda: ep.ep_ffn_product(rank, b(rank.rows_alloc, 16), b(4, 8, 16)),
             ep.EP_ERR_UNSUPPORTED)):
        with pytest.raises(ep.EpError) as e:
            bad()
        assert e.value.status == status
    h.free()
    rank.free()
    with pytest.raises(RuntimeError):
        ep.ep_ffn_product(h, b(r, 16), b(4, 8, 16))


@pytest.mark.parametrize("cap", [1, 2, 5])
@pytest.mark.parametrize("op", OPS)
def test_num_sms(ep, op, cap):
    """A layout's cap on the SMs bounds every launch and changes no bit."""
    from tests.test_ops_sm_cap_gpu import CTAS_PER_SM, grids
    for T, E in ((200, 32), (1500, 2)):
        got = []
        for c in (0, cap):
            h = make_handle(ep, T, 2, E, 1, T, 1, num_sms=c)
            call, outputs = calls(ep, h, h.rows_alloc, 264, 200)[op]
            o = outputs()
            call(o, None)
            torch.cuda.synchronize()
            got.append(o)
            if c:
                assert max(grids(lambda: call(o, None))) <= c * CTAS_PER_SM
            h.free()
        for k, t in got[0].items():
            assert torch.equal(t, got[1][k]), k


@pytest.mark.parametrize("cap", [1, 2, 5])
@pytest.mark.parametrize("op", OPS)
def test_num_sms_by_residency(ep, op, cap):
    """What a capped call launches fits that many SMs at once: of the tensor cores' kernel one
    CTA an SM (its shared memory), of few rows' two, of the small kernel before a weight
    gradient eight.  Uncapped the same calls take more."""
    from tests.test_ops_sm_cap_gpu import grids
    for T, K, E in ((200, 2, 32), (1500, 2, 2), (7, 2, 32)):
        most = {}
        for c in (0, cap):
            h = make_handle(ep, T, K, E, 1, T, 1, num_sms=c)
            call, outputs = calls(ep, h, h.rows_alloc, 1032, 200)[op]
            o = outputs()
            launched = grids(lambda: call(o, None))
            most[c] = launched[-1]
            if op.startswith("wgrad"):
                assert len(launched) == 2
                if c:
                    assert launched[0] <= 8 * c
            else:
                assert len(launched) == 1
            h.free()
        per_sm = 2 if T * K <= 16 and op in ("gated", "product") else 1
        assert most[cap] <= per_sm * cap < most[0]
