"""Plain 64-bit forms of the norm and rotation and of their gradients (numpy), for the tests."""

import numpy as np


def cos_sin(positions, freqs, pair_axis):
    """cos and sin [B, 1, S, R/2]: positions [axes, B, S] integers, freqs float32, angles in extended precision."""
    ld = np.longdouble
    a = positions.astype(ld)[np.asarray(pair_axis)] * freqs.astype(ld)[:, None, None]  # [R/2, B, S]
    two_pi = ld("6.283185307179586476925286766559")
    a = a - two_pi * np.rint(a / two_pi)
    a = np.moveaxis(a, 0, -1)[:, None]
    return np.cos(a).astype(np.float64), np.sin(a).astype(np.float64)


def pairs(D, R, interleaved):
    """Indices (u, v) of the members of every pair."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def turn(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    u, v = pairs(x.shape[-1], R, interleaved)
    y = x.copy()
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., u] * sin + x[..., v] * cos
    return y


def pair_size(x, R, interleaved):
    """|x_u| + |x_v| at both members of every pair, |x_j| elsewhere: what bounds a rotated value's rounding."""
    u, v = pairs(x.shape[-1], R, interleaved)
    m = np.abs(x)
    m[..., u] = m[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    return m


def forward(x, w, eps, cos, sin, interleaved):
    """(y, the size its rounding errors scale with)."""
    n = x
    if eps is not None:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return turn(n, cos, sin, interleaved), pair_size(n, 2 * cos.shape[-1], interleaved)


def backward(g, x, w, eps, cos, sin, interleaved):
    """(dx, its rounding size, dw, its rounding size); dw is None without the norm."""
    u = turn(g, cos, -sin, interleaved)
    size = pair_size(g, 2 * cos.shape[-1], interleaved)
    if eps is None:
        return u, size, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * r
    w = np.ones(x.shape[-1]) if w is None else w
    wu = w * u
    dx = r * (wu - z * (wu * z).mean(-1, keepdims=True))
    dx_size = r * (np.abs(w) * size + np.abs(z) * (np.abs(w) * size * np.abs(z)).mean(-1, keepdims=True))
    return dx, dx_size, (u * z).sum((0, 1, 2)), (size * np.abs(z)).sum((0, 1, 2))
