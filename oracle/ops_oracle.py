"""Plain 64-bit definitions of the operators around dispatch and combine.

numpy only, written from the formulas; used by the tests.  Quantisation is
stated by its scale and the quotients an e4m3 byte stands for, so a test can
bound the rounding instead of repeating it.
"""
from __future__ import annotations

import numpy as np


def scales(v: np.ndarray) -> np.ndarray:
    """amax / 448 of the 1x128 blocks of v [rows, n]."""
    rows, n = v.shape
    return np.abs(v).reshape(rows, n // 128, 128).max(axis=2) / 448.0


def rmsnorm(x, residual, gamma, eps):
    """(s, rstd, v): the sum, 1 / sqrt(mean(s^2) + eps), s * rstd * gamma."""
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s, rstd, s * rstd[:, None] * gamma


def rmsnorm_backward(grad_y, normed, gamma, rstd, grad_residual=None):
    """(grad_x, grad_gamma)."""
    xh = normed * rstd[:, None]
    t = grad_y * gamma
    gx = rstd[:, None] * (t - xh * (t * xh).mean(axis=1, keepdims=True))
    if grad_residual is not None:
        gx = gx + grad_residual
    return gx, (grad_y * xh).sum(axis=0)


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(gate_up, row_weights=None):
    F = gate_up.shape[1] // 2
    g, u = gate_up[:, :F], gate_up[:, F:]
    a = g * _sigmoid(g) * u
    return a if row_weights is None else a * row_weights[:, None]


def swiglu_backward(gate_up, grad_act, row_weights=None):
    """(gradient of gate | up, gradient of the row weights)."""
    F = gate_up.shape[1] // 2
    g, u = gate_up[:, :F], gate_up[:, F:]
    sg = _sigmoid(g)
    gw = (grad_act * g * sg * u).sum(axis=1)
    t = grad_act if row_weights is None else grad_act * row_weights[:, None]
    return np.concatenate([t * u * sg * (1 + g * (1 - sg)), t * g * sg], axis=1), gw


def combine(y, dst, topk_idx, w, expert_bias=None):
    """The weighted combine, [T, H]."""
    T, K = dst.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for k in range(K):
            if dst[t, k] >= 0:
                v = y[dst[t, k]]
                if expert_bias is not None:
                    v = v + expert_bias[topk_idx[t, k]]
                out[t] += w[t, k] * v
    return out


def combine_backward(grad_out, y, dst, topk_idx, w, expert_bias=None, num_experts=0):
    """(grad_y, the weight of each row, its token or -1, grad_weights, grad_bias)."""
    T, K = dst.shape
    rows, H = y.shape
    row_w, token = np.zeros(rows), np.full(rows, -1)
    gw, gb = np.zeros((T, K)), np.zeros((num_experts, H))
    for t in range(T):
        for k in range(K):
            r = dst[t, k]
            if r < 0:
                continue
            e = topk_idx[t, k]
            v = y[r] if expert_bias is None else y[r] + expert_bias[e]
            gw[t, k] = grad_out[t] @ v
            row_w[r] += w[t, k]
            token[r] = t
            if num_experts:
                gb[e] += w[t, k] * grad_out[t]
    gy = np.where(token[:, None] >= 0, row_w[:, None] * grad_out[token], 0.0)
    return gy, row_w, token, gw, gb


def expert_gemm(a, a_sf, w, w_sf, starts, counts):
    """a [rows, k] and w [E, n, k] as e4m3 values, scales [rows, k / 128] and
    [E, ceil(n / 128), k / 128]; rows [starts[e], + counts[e]) times w[e]^T,
    other rows 0."""
    E, n, k = w.shape
    out = np.zeros((a.shape[0], n))
    for e in range(E):
        r0, r1 = starts[e], starts[e] + counts[e]
        av = a[r0:r1] * np.repeat(a_sf[r0:r1], 128, axis=1)
        wv = w[e] * np.repeat(np.repeat(w_sf[e], 128, axis=0)[:n], 128, axis=1)
        out[r0:r1] = av @ wv.T
    return out
