"""Shared helpers of the tests of the operators around dispatch and combine:
tolerances of one rounding, tensors as 64-bit arrays, seeded routings."""
from __future__ import annotations

import numpy as np
import torch

FP8 = torch.float8_e4m3fn
# relative error of the fp32 arithmetic before an output is rounded: sums of at
# most 64 sequential terms per thread and a tree, 2^-24 each
F32 = 2.0 ** -18


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def fp8_f64(t: torch.Tensor) -> np.ndarray:
    return f64(t.view(FP8).to(torch.float32))


def assert_bf16(got: torch.Tensor, want: np.ndarray, slack=0.0, what=""):
    """One rounding to bf16 (half a unit of 8 bits, 2^-8 of the value) of a
    value that may itself be off by `slack`."""
    err = np.abs(f64(got) - want)
    tol = 2.0 ** -8 * (np.abs(want) + slack) + slack + F32 * np.abs(want) + 2.0 ** -133
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(err / tol)}"


def assert_f32(got: torch.Tensor, want: np.ndarray, tol, what=""):
    err = np.abs(f64(got) - want)
    assert (err <= tol + 1e-37).all(), f"{what}: worst {np.max(err / (tol + 1e-37))}"


def assert_fp8(q: torch.Tensor, sf: torch.Tensor, want: np.ndarray, slack=0.0, what=""):
    """Bytes q [rows, n] and scales sf [rows, n / 128] against the values they
    stand for: the scale within fp32 arithmetic, each value within half a unit
    of e4m3 (2^-4 of a normal value, 2^-10 scales of a subnormal one)."""
    rows, n = want.shape
    s = f64(sf)
    slack = np.broadcast_to(np.asarray(slack, dtype=np.float64), want.shape)
    blk = want.reshape(rows, n // 128, 128)
    amax = np.abs(blk).max(axis=2)
    smax = slack.reshape(blk.shape).max(axis=2)
    assert (np.abs(s - amax / 448.0) <= (F32 * amax + smax) / 448.0 * 1.01 + 1e-40).all(), \
        f"{what} scales"
    got = fp8_f64(q) * np.repeat(s, 128, axis=1)
    full = np.repeat(amax / 448.0, 128, axis=1)
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * full) * (1 + 2.0 ** -6) + 1.1 * slack
    err = np.abs(got - want)
    bad = err > tol + 1e-40
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


def routing(T, K, E, seed, drop=0.0, zipf=False, dup=False):
    g = torch.Generator().manual_seed(seed)
    if dup:
        idx = torch.randint(0, E, (T, K), generator=g)
    else:
        p = torch.rand(T, E, generator=g).log()
        if zipf:
            p = p / (torch.arange(E) + 1.0).pow(-1.2)
        idx = p.topk(min(K, E), dim=1).indices
    if drop > 0:
        idx = idx.masked_fill(torch.rand(idx.shape, generator=g) < drop, -1)
    return idx.to(torch.int64).contiguous()


def sf_rows(ep, handle, flat: torch.Tensor, n: int, rows=None) -> torch.Tensor:
    """Scales [rows, n / 128] of a flat array in the handle's layout."""
    _, ts, hs, es = ep.sf_layout(handle, n)
    r = torch.arange(handle.rows_alloc) if rows is None else torch.as_tensor(rows)
    j = torch.arange(n // 128)
    if es > 0:
        cap = int(handle.info.expert_capacity)
        base = (r // cap) * es + (r % cap) * ts
    else:
        base = r * ts
    return flat[(base[:, None] + j * hs).to(flat.device)]


def row_use(h) -> tuple[np.ndarray, np.ndarray]:
    """(rows in use, alignment padding rows) of a layout, from its own arrays."""
    rows = h.rows_alloc
    used, pad = np.zeros(rows, bool), np.zeros(rows, bool)
    cnt = h.tensor("cnt_expert").cpu().numpy()
    psum = h.tensor("psum_expert").cpu().numpy()
    if not h.cfg.do_expand:
        used[:min(rows, int(h.tensor("totals")[0]))] = True
    elif h.cfg.fixed_capacity:
        cap = int(h.info.expert_capacity)
        for e in range(h.E):
            used[e * cap:e * cap + min(int(cnt[e]), cap)] = True
    else:
        for e in range(h.E):
            used[psum[e]:psum[e] + cnt[e]] = True
            pad[psum[e] + cnt[e]:psum[e + 1]] = True
    return used, pad
