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
DENSE = [(1, 128, 64), (1, 8, 8), (1, 520, 1032), (2, 256, 4096), (16, 136, 200), (17, 264, 128),
         (127, 128, 64), (128, 256, 256), (129, 248, 264), (300, 392, 72), (1000, 1000, 328),
         (513, 2056, 192), (64, 512, 7168), (2500, 16, 24)]


@pytest.mark.parametrize("rows,n,k", DENSE)
@pytest.mark.parametrize("op", OPS)
def test_one_matrix(ep, op, rows, n, k):
    check(ep, op, None, rows, n, k, seed=rows + n)


# name: (T, K, E, R, M, A, zero_pad, sync, fixed, drop, n, k)
LAYOUTS = {
    "one_row": (1, 1, 1, 1, 1, 1, True, True, False, 0.0, 256, 128),
    "one_token": (1, 8, 64, 8, 1, 1, True, True, False, 0.0, 512, 1024),
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
