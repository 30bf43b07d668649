"""Shared helpers of the tests of the feed-forward block's products: inputs,
the rows of each matrix, the five calls against their 64-bit definitions."""
from __future__ import annotations

import numpy as np
import torch

from oracle import ops_oracle as P
from tests.ops_harness import F32, assert_bf16, assert_f32, f64, row_use, routing

OPS = ("gated", "gated_bwd", "product", "product_t", "wgrad", "wgrad_bf16")


def sum_error(terms: int) -> float:
    """Of an fp32 sum of `terms` exact products, relative to the sum of their
    magnitudes: the tensor cores add 16 at a time to the sum so far, and what they
    cut off is at most two units in the last place (2^-23 each) of the magnitudes; up
    to 8 partial sums are joined."""
    return (terms / 16 + 9) * 2.0 ** -22


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def make_handle(ep, T, K, E, R, M, A, zp=True, sync=True, fixed=False, drop=0.0, seed=13, **kw):
    cfg = ep.make_config(T, K, E, R, 128, M, A, do_expand=True, do_zero_padding=zp,
                         do_cpu_sync=sync, fixed_capacity=fixed, **kw)
    return ep.ep_layout(cfg, routing(T, K, E, seed, drop).cuda())


def segments(h, rows):
    """(starts, counts, used, zeroed) of the rows of each matrix."""
    if h is None:
        return [0], [rows], np.ones(rows, bool), np.zeros(rows, bool)
    used, pad = row_use(h)
    cnt = h.tensor("cnt_expert").cpu().numpy()
    psum = h.tensor("psum_expert").cpu().numpy()
    if h.cfg.fixed_capacity:
        cap = int(h.info.expert_capacity)
        starts, counts = np.arange(h.E) * cap, np.minimum(cnt, cap)
    else:
        starts, counts = psum[:-1], np.clip(rows - psum[:-1], 0, cnt)
    return list(starts), list(counts), used, pad & bool(h.cfg.do_zero_padding)


class Rows:
    """Arrays of rows of one case: random values on rows in use, on the others what no
    result may show."""

    def __init__(self, h, rows, seed):
        self.h, self.rows = h, rows
        self.starts, self.counts, self.used, self.zeroed = segments(h, rows)
        self.g = torch.Generator().manual_seed(seed)

    def make(self, n, std=1.0):
        v = normal(self.g, self.rows, n, std=std)
        idle = torch.from_numpy(~self.used)
        v[idle] = float("nan")
        if n > 1:
            v[idle, 0::2] = float("inf")
        return v.cuda()

    def value(self, t):
        return np.where(self.used[:, None], f64(t), 0.0)

    def weights(self, n, k):
        lead = () if self.h is None else (self.h.E,)
        return normal(self.g, *lead, n, k, std=k ** -0.5).cuda()

    def stacked(self, w):
        return f64(w) if self.h is not None else f64(w)[None]

    def out(self, n):
        return torch.full((self.rows, n), 7.0, dtype=torch.bfloat16, device="cuda")

    def compare(self, got, want, slack, what):
        """Rows in use against the definition, zeroed padding, all others untouched."""
        u = self.used
        assert_bf16(got[torch.from_numpy(u).cuda()], want[u], slack[u], what)
        assert not got[torch.from_numpy(self.zeroed).cuda()].any(), f"{what}: padding"
        idle = torch.from_numpy(~(u | self.zeroed)).cuda()
        assert (got[idle] == 7).all(), f"{what}: unused rows written"


def check(ep, op, h, rows, n, k, seed=1, keep=True, **kw):
    """One call of `op` with a matrix [n, k] per expert (n: ffn for the gated ones)."""
    s = Rows(h, rows, seed)
    err = sum_error(k)
    if op == "gated":
        x, w = s.make(k), s.weights(2 * n, k)
        act, gu = s.out(n), s.out(2 * n) if keep else None
        ep.ep_ffn_gated(h, x, w, act=act, gate_up=gu, **kw)
        hv = P.segment_product(s.value(x), s.stacked(w), s.starts, s.counts)
        mag = err * P.segment_product(np.abs(s.value(x)), np.abs(s.stacked(w)), s.starts, s.counts)
        if keep:
            s.compare(gu, hv, mag, "gate_up")
        a = P.swiglu(hv)
        g, u = hv[:, :n], hv[:, n:]
        # |d silu| <= 1.1 |dg|, |silu| <= |g|; the activation's own arithmetic: 2^-20
        slack = 1.1 * mag[:, :n] * (np.abs(u) + mag[:, n:]) + np.abs(g) * mag[:, n:] \
            + 2.0 ** -20 * np.abs(g * u)
        s.compare(act, a, slack, "act")
    elif op == "gated_bwd":
        gy, w, gu = s.make(k, 0.02), s.weights(k, n), s.make(2 * n, 1.5)
        ggu, act = s.out(2 * n), s.out(n) if keep else None
        ep.ep_ffn_gated_backward(h, gy, w, gu, grad_gate_up=ggu, act=act, **kw)
        d = P.segment_product(s.value(gy), s.stacked(w), s.starts, s.counts, True)
        mag = err * P.segment_product(np.abs(s.value(gy)), np.abs(s.stacked(w)), s.starts,
                                      s.counts, True)
        hv = s.value(gu)
        slopes, a = P.gated_slopes(hv)
        # absolute error of the slopes' arithmetic: 2^-18 of |u| and of |g|
        arith = 2.0 ** -18 * np.abs(np.concatenate([hv[:, n:] * 1.2, hv[:, :n]], axis=1))
        d2, m2 = np.tile(d, 2), np.tile(mag, 2)
        s.compare(ggu, d2 * slopes, m2 * np.abs(slopes) + (np.abs(d2) + m2) * arith,
                  "grad_gate_up")
        if keep:
            s.compare(act, a, 2.0 ** -20 * np.abs(hv[:, :n] * hv[:, n:]), "act")
    elif op in ("product", "product_t"):
        flip = op == "product_t"
        a, w = s.make(k), s.weights(*((k, n) if flip else (n, k)))
        out = s.out(n)
        ep.ep_ffn_product(h, a, w, out=out, transposed=flip, **kw)
        args = (s.starts, s.counts, flip)
        s.compare(out, P.segment_product(s.value(a), s.stacked(w), *args),
                  err * P.segment_product(np.abs(s.value(a)), np.abs(s.stacked(w)), *args), "out")
    else:
        f32 = op == "wgrad"
        grad, a = s.make(n), s.make(k)
        for accumulate in (False, True):
            lead = (1,) if h is None else (h.E,)
            before = normal(s.g, *lead, n, k, std=3.0).float().cuda()
            if not f32:
                before = before.bfloat16()
            gw = before.clone()
            ep.ep_ffn_weight_grad(h, grad, a, grad_w=gw[0] if h is None else gw,
                                  accumulate=accumulate, **kw)
            want = P.segment_outer(s.value(grad), s.value(a), s.starts, s.counts)
            mag = P.segment_outer(np.abs(s.value(grad)), np.abs(s.value(a)), s.starts, s.counts)
            slack = sum_error(max(s.counts, default=0)) * mag
            if accumulate:
                want = want + f64(before)
            if f32:
                assert_f32(gw, want, slack + F32 * np.abs(want), "grad_w")
            else:
                assert_bf16(gw, want, slack, "grad_w")
            idle = torch.tensor([c == 0 for c in s.counts])
            left = before[idle.cuda()] if accumulate else torch.zeros_like(before[idle.cuda()])
            assert torch.equal(gw[idle.cuda()], left), "an expert without rows"
    if h is not None:
        assert int(h.tensor("error_word")[0]) & ep.EP_ERRBIT_TIMEOUT == 0
