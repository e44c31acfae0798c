"""Rotary positions over several axes, in float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A head of D elements is D/2 pairs; an axis of d dimensions owns d/2 of them,
in the order of the axes, and its pair j turns by pos * theta^(-2j/d):
    (x, y) -> (x cos - y sin, x sin + y cos)
Pairs are (2i, 2i+1) or, half-split, (i, i + D/2).  Before it, optionally,
x * w / sqrt(mean x^2 + eps) over the head.
"""
import numpy as np


def norm(x, w, eps):
    return x * w / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def rope(x, pos, axis_dims, theta=10000.0, half=False, inverse=False, w=None, eps=1e-6):
    """x [M, heads, D], pos [M, axes] -> [M, heads, D] float64."""
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = norm(x, w, eps)
    angle = np.concatenate([np.asarray(pos, dtype=np.float64)[:, a:a + 1] * theta ** (-2.0 * np.arange(d // 2) / d)
                            for a, d in enumerate(axis_dims)], axis=1)[:, None, :]
    c, s = np.cos(angle), np.sin(-angle if inverse else angle)
    n = x.shape[-1] // 2
    a, b = (x[..., :n], x[..., n:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * s, a * s + b * c
    out = np.empty_like(x)
    if half:
        out[..., :n], out[..., n:] = u, v
    else:
        out[..., 0::2], out[..., 1::2] = u, v
    return out
