"""Plain fp64 CPU definition of QK-norm with RoPE at given positions, and of
its gradient.

TEST INFRASTRUCTURE.  Part of the oracle the CUDA path is checked against;
only the test suite may import it, and nothing here is shared with the CUDA
kernels.

Written from "The Mathematics of Karpathy's nanochat": §Rotary Position
Embeddings (half split, RoPE(u) = (u1 cos + u2 sin, -u1 sin + u2 cos) with angle
t base^(-2i/D); `reverse` negates the angles) and §QK-Norm with Sharpening:
    y = alpha RoPE(x) / sqrt(mean(RoPE(x)^2) + eps).
The gradient is the vector-Jacobian product of these two steps, each with its
own Jacobian, last step first.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def _angles(positions, D, base):
    theta = np.power(F64(base), -2.0 * np.arange(D // 2, dtype=F64) / D)
    return np.asarray(positions, F64)[:, None] * theta          # [N, D/2]


def rope(x, positions, base: float, reverse: bool = False):
    x = np.asarray(x, F64)
    a = _angles(positions, x.shape[-1], base)[:, None]
    c, s = np.cos(a), np.sin(a) * (-1.0 if reverse else 1.0)
    lo, hi = np.split(x, 2, axis=-1)
    return np.concatenate([lo * c + hi * s, hi * c - lo * s], axis=-1)


def forward(x, positions, alpha: float, base: float, eps: float, reverse: bool = False):
    """x [N, heads, D] at positions [N]."""
    r = rope(x, positions, base, reverse)
    return alpha * r / np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + eps)


def backward(x, positions, dy, alpha: float, base: float, eps: float, reverse: bool = False):
    r, dy = rope(x, positions, base, reverse), np.asarray(dy, F64)
    D = r.shape[-1]
    rho = np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + eps)
    # d(r / rho) / dr = I / rho - r r^T / (D rho^3)
    dr = alpha * (dy / rho - r * np.sum(r * dy, axis=-1, keepdims=True) / (D * rho ** 3))
    return rope(dr, positions, base, not reverse)
