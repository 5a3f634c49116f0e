"""fp64 oracle of the operators around the layer (include/vsa_block.h): rotary
positions, head norms with the rotation, linears with their epilogues, and their
gradients.  Plain numpy, one function per formula; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def _np(t):
    return t.detach().cpu().double().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def positions(prefix, grid, offset=(0, 0, 0), step=(1, 1, 1), prefix_pos=None):
    """[N, 3]: the prefix's given positions (zeros without), then the grid, t-major."""
    n_p = int(sum(prefix))
    pre = np.zeros((n_p, 3)) if prefix_pos is None else np.asarray(prefix_pos, dtype=np.float64)
    vid = np.indices(tuple(grid)).reshape(3, -1).T.astype(np.float64)
    return np.concatenate([pre, np.asarray(offset) + np.asarray(step) * vid])


def angles(pos, dims, theta=(1e4, 1e4, 1e4), inv_freq=None):
    """[N, P]: position of a pair's axis times its frequency."""
    cols, k = [], 0
    for a in range(3):
        for i in range(dims[a] // 2):
            f = theta[a] ** (-2.0 * i / dims[a]) if inv_freq is None else inv_freq[k]
            cols.append(pos[:, a] * f)
            k += 1
    return np.stack(cols, 1)


def rotate(x, ang, halves, inverse=False):
    """x [..., N, D]; pair p turns by ang[n, p]."""
    y, P = _np(x).copy(), ang.shape[1]
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    for p in range(P):
        i, j = (p, P + p) if halves else (2 * p, 2 * p + 1)
        a, b = y[..., i].copy(), y[..., j].copy()
        y[..., i] = a * c[:, p] - b * s[:, p]
        y[..., j] = a * s[:, p] + b * c[:, p]
    return y


def head_norm(x, gain, eps):
    x = _np(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if gain is None else _np(gain))


def head_norm_backward(g, x, gain, eps):
    """(dx, d_gain) of head_norm under the gradient g of its output."""
    g, x = _np(g), _np(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    gw = g * (1.0 if gain is None else _np(gain))
    dx = r * (gw - u * (gw * u).mean(-1, keepdims=True))
    return dx, (g * u).sum(axis=tuple(range(x.ndim - 1)))


def act(name, x):
    x = _np(x)
    with np.errstate(over="ignore"):
        if name == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        if name == "silu":
            return x / (1.0 + np.exp(-x))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))
    return x


def act_slope(name, x):
    x = _np(x)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-x))
    if name == "sigmoid":
        return s * (1.0 - s)
    if name == "silu":
        return s * (1.0 + x * (1.0 - s))
    if name == "gelu_tanh":
        c = np.sqrt(2.0 / np.pi)
        t = np.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    return np.ones_like(x)


def rows(x):
    """[B,N,C] from rows or heads [B,H,N,D]."""
    x = _np(x)
    return x if x.ndim == 3 else x.transpose(0, 2, 1, 3).reshape(x.shape[0], x.shape[2], -1)


def heads(x, h):
    """[B,H,N,D] from rows (h = 0: rows as they are)."""
    if not h:
        return x
    return x.reshape(x.shape[0], x.shape[1], h, -1).transpose(0, 2, 1, 3)


def linear(x, w, bias=None):
    p = rows(x) @ _np(w).T
    return p if bias is None else p + _np(bias)


def linear_backward(dy, x, w):
    """(dx, dw, db) in rows."""
    dy, x = rows(dy), rows(x)
    return dy @ _np(w), np.einsum("bno,bnc->oc", dy, x), dy.sum((0, 1))
