"""Rotary positions from their definition, in 64 bits (numpy)."""
import numpy as np


def rotate(x, positions, inv_freq, axis, adjacent):
    """x [T, H, D] fp64, positions int [axes, T]: pair f of the first 2 len(inv_freq) dims turned by
    positions[axis[f]] * inv_freq[f]."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for f in range(n):
        a = positions[axis[f]].astype(np.float64) * inv_freq[f]
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        i, j = (2 * f, 2 * f + 1) if adjacent else (f, f + n)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def magnitude(x, n, adjacent):
    """Of each dim, |x0| + |x1| of its pair (0 for dims that do not turn)."""
    m = np.zeros_like(x)
    for f in range(n):
        i, j = (2 * f, 2 * f + 1) if adjacent else (f, f + n)
        m[..., i] = m[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return m
