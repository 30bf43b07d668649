"""The 64-bit definitions of the operators' gradients against central
differences of their forwards (no GPU)."""
import numpy as np
import pytest

from oracle import ops_oracle as P


def differences(f, x, grad_out, h=1e-6):
    """Gradient of sum(grad_out * f(x)) by central differences."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        out[i] = (grad_out * (f(x + d) - f(x - d))).sum() / (2 * h)
    return out


# central differences: error h^2 * third derivative + 1e-16 / h, about 1e-9
TOL = dict(rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("T,H", [(1, 8), (3, 16), (5, 7)])
def test_rmsnorm(T, H):
    rng = np.random.default_rng(T * H)
    x, g, go, gr = (rng.normal(size=s) for s in [(T, H), (H,), (T, H), (T, H)])
    s, rstd, _ = P.rmsnorm(x, None, g, 1e-5)
    gx, gg = P.rmsnorm_backward(go, s, g, rstd, gr)
    assert np.allclose(gx, differences(lambda v: P.rmsnorm(v, None, g, 1e-5)[2], x, go) + gr, **TOL)
    assert np.allclose(gg, differences(lambda v: P.rmsnorm(x, None, v, 1e-5)[2], g, go), **TOL)
    res = rng.normal(size=(T, H))
    s2, rstd2, _ = P.rmsnorm(x, res, g, 1e-5)
    want = differences(lambda v: P.rmsnorm(x, v, g, 1e-5)[2], res, go)
    assert np.allclose(P.rmsnorm_backward(go, s2, g, rstd2)[0], want, **TOL)


@pytest.mark.parametrize("rows,F", [(1, 4), (3, 6)])
def test_swiglu(rows, F):
    rng = np.random.default_rng(F)
    h, w, ga = rng.normal(size=(rows, 2 * F)) * 2, rng.normal(size=rows), rng.normal(size=(rows, F))
    gh, gw = P.swiglu_backward(h, ga, w)
    assert np.allclose(gh, differences(lambda v: P.swiglu(v, w), h, ga), **TOL)
    assert np.allclose(gw, differences(lambda v: P.swiglu(h, v), w, ga), **TOL)
    assert np.allclose(P.swiglu_backward(h, ga)[0], differences(lambda v: P.swiglu(v), h, ga), **TOL)


def test_combine():
    rng = np.random.default_rng(3)
    T, K, E, H, rows = 4, 3, 5, 6, 9
    idx = np.array([[0, 1, 2], [3, -1, 4], [-1, -1, -1], [2, 2, 0]])
    # slots 0 and 1 of token 0 share a row; a dropped slot; a token without slots
    dst = np.array([[0, 0, 5], [1, -1, 2], [-1, -1, -1], [3, -1, 4]])
    y, b, w = rng.normal(size=(rows, H)), rng.normal(size=(E, H)), rng.normal(size=(T, K))
    go = rng.normal(size=(T, H))
    gy, _, _, gw, gb = P.combine_backward(go, y, dst, idx, w, b, E)
    assert np.allclose(gy, differences(lambda v: P.combine(v, dst, idx, w, b), y, go), **TOL)
    assert np.allclose(gw, differences(lambda v: P.combine(y, dst, idx, v, b), w, go), **TOL)
    assert np.allclose(gb, differences(lambda v: P.combine(y, dst, idx, w, v), b, go), **TOL)


def test_expert_gemm_scales():
    """Block scales multiply whole 128-wide blocks: equal to scaling the operands."""
    rng = np.random.default_rng(5)
    a, w = rng.normal(size=(7, 256)), rng.normal(size=(2, 136, 256))
    asf, wsf = rng.uniform(1, 2, (7, 2)), rng.uniform(1, 2, (2, 2, 2))
    out = P.expert_gemm(a, asf, w, wsf, [0, 4], [3, 2])
    assert not out[3].any() and not out[6].any()
    for r, e in [(0, 0), (2, 0), (4, 1), (5, 1)]:
        for n in (0, 127, 128, 135):
            want = sum(asf[r, j] * wsf[e, n // 128, j]
                       * (a[r, 128 * j:128 * j + 128] @ w[e, n, 128 * j:128 * j + 128])
                       for j in range(2))
            assert np.isclose(out[r, n], want)
