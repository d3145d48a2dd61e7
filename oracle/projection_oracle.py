"""fp64 oracle of the projection side: rotary positions with several axes, the
per-head RMS norm with the rotation, the linear product with its epilogue, and
their gradients.

Written from the formulas with complex numbers and explicit sums, on [..., N, D]
arrays, sharing no code with the package. ``positions`` is [N, axes]; ``sections``
holds the rotated channels of each axis.
"""
from __future__ import annotations

import math

import numpy as np


def grid_positions(T, H, W, origin=(0, 0, 0)):
    """[T*H*W, 3] positions of a raster grid, row-major in (t, h, w)."""
    g = np.stack(np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij"), -1).reshape(-1, 3)
    return g.astype(np.float64) + np.asarray(origin, dtype=np.float64)


def angles(positions, sections, base=10000.0, scale=None, shared=False):
    """[N, pairs] radians."""
    rot = sum(sections)
    cols, j = [], 0
    for a, n in enumerate(sections):
        for i in range(n // 2):
            f = base ** (-2.0 * j / rot) if shared else base ** (-2.0 * i / n)
            cols.append(positions[:, a].astype(np.float64) * f * (1.0 if scale is None else scale[a]))
            j += 1
    return np.stack(cols, -1) if cols else np.zeros((positions.shape[0], 0))


def rotate(x, ang, interleaved):
    """x [..., N, D] with pair j of each token turned by ang[n, j]."""
    x = np.asarray(x, dtype=np.float64)
    m = ang.shape[-1]
    y = x.copy()
    u, v = (slice(0, 2 * m, 2), slice(1, 2 * m, 2)) if interleaved else (slice(0, m), slice(m, 2 * m))
    z = (x[..., u] + 1j * x[..., v]) * np.exp(1j * ang)
    y[..., u], y[..., v] = z.real, z.imag
    return y


def norm_rotate(x, w, eps, ang, interleaved):
    x = np.asarray(x, dtype=np.float64)
    return rotate(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w, ang, interleaved)


def norm_rotate_backward(x, w, eps, ang, interleaved, dy):
    """(dx, dw): dw summed over every row of x."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    g = rotate(dy, -ang, interleaved)
    h = g * w
    dx = r * h - x * r ** 3 * np.sum(h * x, -1, keepdims=True) / D
    return dx, np.sum((g * x * r).reshape(-1, D), 0)


# ---------------------------------------------------------------- linear product
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def rows(x):
    """[B, N, channels] of that or of [B, heads, N, D]."""
    x = np.asarray(x, dtype=np.float64)
    return x if x.ndim == 3 else np.concatenate([x[:, h] for h in range(x.shape[1])], -1)


def linear(x, w, b=None, act=None, res=None):
    """(y, z) as rows."""
    z = np.einsum("bnk,fk->bnf", rows(x), np.asarray(w, dtype=np.float64)) + (0 if b is None else b)
    return activate(z, act) + (0 if res is None else rows(res)), z


def linear_backward(x, w, dout, z=None, act=None):
    """(dx, dw, db), dx as rows."""
    dz = rows(dout) * (1 if act is None else slope(rows(z), act))
    return (np.einsum("bnf,fk->bnk", dz, np.asarray(w, dtype=np.float64)), np.einsum("bnf,bnk->fk", dz, rows(x)),
            dz.sum((0, 1)))
