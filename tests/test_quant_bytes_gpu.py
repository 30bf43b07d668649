"""GPU tests of the operators' quantisation, byte by byte, on BF16 blocks that
hold every mantissa of a largest value against every mantissa of the others: the
stated scale, bytes to nearest but for the reciprocal's last place, and how far
the dispatch's bytes of the same rows are."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
# one unit in the last place of the reciprocal (2^-23) and the product's rounding (2^-24)
RECIPROCAL = 2.0 ** -22
BLOCKS = 28  # 128 mantissas x 27 exponents, 127 to a block


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_topk_idx_gb300 as ep
    ep.load_library()
    return ep


def rows(exponent=0):
    """[128, BLOCKS * 128] BF16: row i's blocks have the largest value 1 + i / 128
    (times 2^exponent), in every block another place."""
    m = 1 + np.arange(128) / 128
    v = np.concatenate([m * 2.0 ** -e for e in range(1, 28)])
    v = np.resize(v * np.where(np.arange(v.size) % 3, 1, -1), BLOCKS * 127).reshape(BLOCKS, 127)
    out = np.empty((128, BLOCKS, 128))
    for b in range(BLOCKS):
        out[:, b] = np.insert(v[b], (37 * b) % 128, 0)[None]
        out[:, b, (37 * b) % 128] = m
    x = torch.from_numpy(out.reshape(128, -1) * 2.0 ** exponent).to(torch.bfloat16)
    assert torch.equal(x.double(), torch.from_numpy(out.reshape(128, -1) * 2.0 ** exponent))
    return x


def e4m3(x):
    """Nearest e4m3 value, ties to even, saturating."""
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(x))), -6)
    return np.clip(np.rint(x / 2.0 ** (e - 3)) * 2.0 ** (e - 3), -448, 448)


def values(q):
    return q.cpu().view(torch.float8_e4m3fn).float().double().numpy()


def check(x, q, sf):
    """Bytes q [128, n] and scales sf [128, n / 128] of x."""
    v = x.double().numpy().reshape(128, -1, 128)
    s = sf.cpu().numpy()
    amax = np.abs(v).max(2).astype(np.float32)
    assert np.array_equal(s, amax * (np.float32(1) / np.float32(448)))
    quotient = v / s.astype(np.float64)[..., None]
    got = values(q).reshape(v.shape)
    lo, hi = e4m3(quotient * (1 - RECIPROCAL)), e4m3(quotient * (1 + RECIPROCAL))
    assert ((got == lo) | (got == hi)).all()
    assert (lo != hi).any()  # the rows do hold values next to a middle


@pytest.mark.parametrize("exponent", [0, -60, 90])
def test_checkpoint(ep, exponent):
    x = rows(exponent)
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    sf = torch.empty(128, BLOCKS, device="cuda")
    ep.ep_swiglu(None, x.cuda(), ckpt=q, ckpt_sf=sf)
    torch.cuda.synchronize()
    check(x, q, sf)


@pytest.mark.parametrize("exponent", [0, -60])
def test_combine_gradient_and_dispatch(ep, exponent):
    x = rows(exponent)
    T, H = x.shape
    cfg = ep.make_config(T, 1, 4, 1, H, T, 1, do_expand=True, use_fp8=True)
    h = ep.ep_layout(cfg, (torch.arange(T) % 4)[:, None].cuda())
    dst = h.tensor("dst_buffer_slot_idx")[:, 0].long()
    q, sf = ep.alloc_fp8(h, H)
    ep.ep_combine_weighted_backward(h, x.cuda(), None, torch.ones(T, 1, device="cuda"),
                                    grad_y_fp8=q, grad_y_sf=sf)
    r = ep.alloc_recv(h)
    ep.ep_dispatch(h, x.cuda(), None, **r)
    torch.cuda.synchronize()
    q, sf = q[dst], sf.view(T, BLOCKS)[dst]
    check(x, q, sf)
    # the dispatch: IEEE quotients, so the same or a neighbouring byte
    dq, dsf = r["recv_x"][dst].view(torch.uint8), r["recv_sf"].view(T, BLOCKS)[dst]
    s = dsf.cpu().numpy()
    amax = x.float().abs().view(T, BLOCKS, 128).amax(2).numpy()
    assert np.array_equal(s, amax / np.float32(448))
    assert (np.abs(s - sf.cpu().numpy()) <= np.spacing(s)).all()
    away = (dq.cpu().int() - q.cpu().int()).abs()
    assert int(away.max()) <= 1 and float((away > 0).float().mean()) < 0.01
