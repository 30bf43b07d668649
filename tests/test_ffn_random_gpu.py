"""GPU parity of the feed-forward block's products and of clipping on seeded random
configurations: layouts, sizes, skews, upper bounds, fixed capacities."""
import random

import pytest
import torch

from tests.ffn_harness import OPS, check, make_handle
from tests.test_clip_gpu import check as check_clip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def size(r, most):
    return 8 * max(1, int(round(most / 8 * r.random() ** 2)))


@pytest.mark.parametrize("seed", range(40))
def test_layouts(ep, seed):
    r = random.Random(seed)
    E, R = r.choice([(1, 1), (2, 1), (3, 3), (6, 2), (16, 4), (48, 8), (130, 2), (450, 1)])
    K = r.randint(1, min(6, E))
    T = r.choice([1, r.randint(2, 40), r.randint(40, 400), r.randint(400, 2500)])
    fixed = r.random() < 0.2
    M = -(-T // R) + (0 if fixed else r.randint(0, 9))
    sync = not fixed and r.random() < 0.5
    align, zero = r.choice([1, 1, 4, 16, 100, 128]), r.random() < 0.5
    if fixed:  # a slab per expert: no alignment, no padding
        align, zero = 1, False
    h = make_handle(ep, T, K, E, R, M, align, zero, sync, fixed, r.choice([0.0, 0.0, 0.1, 0.7]),
                    seed=seed)
    most = 700 if T * K < 2000 else 260
    n, k = size(r, most), size(r, most)
    for op in r.sample(OPS, 3):
        check(ep, op, h, h.rows_alloc, n, k, seed=seed, keep=r.random() < 0.7)
    h.free()


@pytest.mark.parametrize("seed", range(40))
def test_one_matrix(ep, seed):
    r = random.Random(1000 + seed)
    rows = r.choice([r.randint(1, 17), r.randint(16, 140), r.randint(100, 700),
                     r.randint(700, 4000)])
    most = 3000 if rows < 20 else 1000 if rows < 700 else 400
    for op in r.sample(OPS, 3):
        check(ep, op, None, rows, size(r, most), size(r, most), seed=seed,
              keep=r.random() < 0.7)


@pytest.mark.parametrize("seed", range(30))
def test_clip(ep, seed):
    r = random.Random(2000 + seed)
    g = torch.Generator().manual_seed(seed)
    count = r.choice([1, r.randint(2, 64), r.randint(60, 70), r.randint(64, 1300)])
    most = 200_000 if count < 70 else 3000
    flats, at = {}, {}
    for kind in (torch.float32, torch.bfloat16):
        flats[kind] = [torch.empty(count * (most + 8) + 16, dtype=kind, device="cuda")
                       for _ in range(2)]
        at[kind] = [r.randint(0, 8), r.randint(0, 8)]
    grads, outs = [], []
    for _ in range(count):
        kind = r.choice(list(flats))
        n = int(most * r.random() ** 4)
        pair = []
        for flat, i in zip(flats[kind], range(2)):
            pair.append(flat[at[kind][i]:at[kind][i] + n])
            at[kind][i] += n + r.choice([0, 0, 1, 3, 8])
        pair[0].copy_(torch.randn(n, generator=g) * 10.0 ** r.uniform(-6, 1))
        grads.append(pair[0])
        outs.append(pair[1])
    check_clip(ep, grads, r.choice([1.0, 0.01, 1e9]), r.choice([outs, None]))
