"""Plain fp64 CPU definition of the clipped policy loss with a KL term and of
its gradient with respect to the logits.

TEST INFRASTRUCTURE.  Part of the oracle the CUDA path is checked against;
only the test suite may import it, and nothing here is shared with the CUDA
kernels.

Per token with a target y != -1: lp = z_y - logsumexp(z) ("The Mathematics of
Karpathy's nanochat", §Cross-Entropy Loss), r = exp(lp - old), d = ref - lp,
    L = -min(r A, clip(r, 1 - cl, 1 + ch) A) + beta (e^d - d - 1),
    loss = sum_t w_t L_t.
The gradient is the chain rule through lp; where the two arguments of the
minimum are equal it is that of r A.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def weights(targets, norm: int):
    """w [B, T]: 0 = the same for every token, 1 = the same for every sequence."""
    valid = np.asarray(targets) != -1
    if norm == 0:
        return valid / max(1, valid.sum())
    per = valid.sum(axis=1, keepdims=True)
    return valid / np.maximum(per, 1) / max(1, (per > 0).sum())


def log_probs(logits, targets):
    z, y = np.asarray(logits, F64), np.maximum(np.asarray(targets), 0)
    m = z.max(axis=-1, keepdims=True)
    lse = m[..., 0] + np.log(np.exp(z - m).sum(axis=-1))
    return np.take_along_axis(z, y[..., None], -1)[..., 0] - lse, lse


def policy_loss(logits, targets, advantages, old=None, ref=None, clip_low=0.2, clip_high=0.2, beta=0.0, norm=0):
    """Returns dict(stats [3], lp [B, T], dz [B, T, V], slope [B, T], p [B, T, V], size [B, T]); size bounds
    the terms that slope is the sum of."""
    z, y = np.asarray(logits, F64), np.asarray(targets)
    w = weights(y, norm)
    lp, lse = log_probs(z, y)
    A = np.asarray(advantages, F64)
    A = np.broadcast_to(A if A.ndim == 2 else A[:, None], y.shape)
    r = np.exp(lp - (lp if old is None else np.asarray(old, F64)))
    free, cut = r * A, np.clip(r, 1 - clip_low, 1 + clip_high) * A
    loss, slope, size, kl = -np.minimum(free, cut), np.where(free <= cut, -r * A, 0.0), np.abs(r * A), np.zeros(y.shape)
    if ref is not None:
        d = np.asarray(ref, F64) - lp
        kl = np.expm1(d) - d
        loss, slope, size = loss + beta * kl, slope - beta * np.expm1(d), size + beta * (1 + np.exp(d))
    p = np.exp(z - lse[..., None])
    hot = np.zeros(z.shape)
    np.put_along_axis(hot, np.maximum(y, 0)[..., None], 1.0, -1)
    valid = y != -1
    keep = lambda x: np.where(valid, x, 0.0)
    stats = np.array([(w * keep(x)).sum() for x in (loss, kl, (free > cut).astype(F64))])
    g = w * keep(slope)
    return {"stats": stats, "lp": keep(lp), "dz": g[..., None] * (hot - p), "slope": g, "p": p, "size": w * keep(size),
            "hot": hot}
