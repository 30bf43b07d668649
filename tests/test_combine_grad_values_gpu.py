"""GPU tests of ep_combine_weighted_backward with infinities, NaN and zero weights:
each stays with the rows, slots and experts that it belongs to."""
import pytest
import torch

from tests.ops_harness import routing, sf_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


class Case:
    """One layout, its inputs, and a call with all outputs."""

    def __init__(self, ep, expand=True, T=60, K=3, E=12, H=256, drop=0.1):
        self.ep, self.T, self.K, self.E, self.H = ep, T, K, E, H
        cfg = ep.make_config(T, K, E, 2, H, T // 2, 8 if expand else 1, do_expand=expand,
                             do_zero_padding=expand)
        self.idx = routing(T, K, E, 17, drop)
        self.h = ep.ep_layout(cfg, self.idx.cuda())
        g = torch.Generator().manual_seed(T + H)
        self.go = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.y = torch.randn(self.h.rows_alloc, H, generator=g).to(torch.bfloat16).cuda()
        self.b = torch.randn(E, H, generator=g).to(torch.bfloat16).cuda()
        self.w = torch.randn(T, K, generator=g).cuda()
        self.dst = self.h.tensor("dst_buffer_slot_idx").cpu()

    def run(self):
        rows = self.h.rows_alloc
        q, sf = self.ep.alloc_fp8(self.h, self.H, zero=True)
        gy = torch.zeros(rows, self.H, dtype=torch.bfloat16, device="cuda")
        gw = torch.zeros(self.T, self.K, device="cuda")
        gb = torch.zeros(self.E, self.H, device="cuda")
        self.ep.ep_combine_weighted_backward(self.h, self.go, self.y, self.w, self.b, grad_y=gy,
                                             grad_y_fp8=q, grad_y_sf=sf, grad_topk_weights=gw,
                                             grad_expert_bias=gb)
        torch.cuda.synchronize()
        return (gy.cpu(), q.cpu(), sf_rows(self.ep, self.h, sf, self.H).cpu(), gw.cpu(),
                gb.cpu())


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=123.0), torch.nan_to_num(b, nan=123.0))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_weight_zero_writes_zero_bytes_and_scales(ep, value):
    c = Case(ep)
    t, col = 7, 130  # the second scale block
    c.go[t, col] = value
    c.w[t] = 0
    c.w[t, 1] = -0.0
    gy, q, s, _, gb = c.run()
    rows = [r for r in c.dst[t].tolist() if r >= 0]
    assert rows
    for r in rows:
        assert not q[r].any() and not s[r].any()
        # the BF16 row is the product itself
        assert torch.isnan(gy[r]).nonzero().flatten().tolist() == [col]
    c.w[t] = 2.0
    _, q, s, _, _ = c.run()
    for r in rows:
        assert torch.isfinite(s[r, 0]) and not torch.isfinite(s[r, 1])
        assert q[r, col] & 0x7F == 0x7F


@pytest.mark.parametrize("expand", [True, False])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_gradient_stays_with_its_token_and_experts(ep, expand, value):
    """A token's infinite or NaN gradient reaches its rows, its weights' gradients
    and the biases of its own experts, and nothing else."""
    c = Case(ep, expand)
    base = c.run()
    t, col = 11, 37
    c.go[t, col] = value
    gy, q, s, gw, gb = c.run()
    rows = torch.zeros(c.h.rows_alloc, dtype=torch.bool)
    rows[c.dst[t][c.dst[t] >= 0].long()] = True
    assert rows.any()
    for got, want in ((gy, base[0]), (q, base[1]), (s, base[2])):
        assert same(got[~rows], want[~rows])
    assert not torch.isfinite(gy[rows, col].float()).any()
    assert torch.isfinite(gy[rows][:, torch.arange(c.H) != col].float()).all()
    slots = torch.zeros(c.T, c.K, dtype=torch.bool)
    slots[t] = c.idx[t] >= 0
    assert same(gw[~slots], base[3][~slots]) and not torch.isfinite(gw[slots]).any()
    mine = torch.zeros(c.E, dtype=torch.bool)
    mine[c.idx[t][c.idx[t] >= 0]] = True
    assert not mine.all()
    assert torch.equal(gb[~mine], base[4][~mine]), "reached an expert that the token never chose"
    assert not torch.isfinite(gb[mine, col]).any()
    rest = torch.arange(c.H) != col
    assert torch.equal(gb[mine][:, rest], base[4][mine][:, rest])


def test_a_row_of_y_stays_with_its_slots(ep):
    c = Case(ep)
    base = c.run()
    t = int((c.dst >= 0).all(1).nonzero()[0])
    c.y[c.dst[t, 1]] = float("nan")
    got = c.run()
    for i in (0, 1, 2, 4):
        assert same(got[i], base[i])
    slots = torch.zeros(c.T, c.K, dtype=torch.bool)
    slots[t, 1] = True
    assert torch.isnan(got[3][slots]).all() and torch.equal(got[3][~slots], base[3][~slots])


def test_weights_without_a_row_are_not_read_into_anything(ep):
    """NaN weights on dropped slots."""
    c = Case(ep, drop=0.3)
    base = c.run()
    c.w[(c.idx < 0).cuda()] = float("nan")
    for got, want in zip(c.run(), base):
        assert torch.equal(got, want)
