"""Plain fp64 CPU definition of the attention of rows that share a prefix.

TEST INFRASTRUCTURE.  Part of the oracle the CUDA path is checked against;
only the test suite may import it, and nothing here is shared with the CUDA
kernels.

Written from "The Mathematics of Karpathy's nanochat", §Scaled Dot-Product
Attention with Sliding Window, for a row whose key sequence is its group's
prefix followed by its own keys: query i of Tq has position P + S - Tq + i and
sees key j iff j <= position and position - j < w.  A query that sees nothing
has output 0 and log-sum-exp -inf.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def row_attention(q, k, v, window: int, scale: float):
    """q [Tq, H, D] at the last Tq of the positions of k, v [L, H_kv, D].
    Returns (o [Tq, H, D], lse [Tq, H], mag [Tq, H, D]) with mag = sum p |v|."""
    q, k, v = (np.asarray(t, F64) for t in (q, k, v))
    Tq, H, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    o, mag = np.zeros((Tq, H, D)), np.zeros((Tq, H, D))
    lse = np.full((Tq, H), -np.inf)
    for i in range(Tq):
        pos = L - Tq + i
        lo = 0 if window <= 0 else max(0, pos - window + 1)
        if pos < lo:
            continue
        for h in range(H):
            kh, vh = k[lo:pos + 1, h // (H // Hkv)], v[lo:pos + 1, h // (H // Hkv)]
            s = scale * (kh @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            p /= p.sum()
            o[i, h], mag[i, h] = p @ vh, p @ np.abs(vh)
    return o, lse, mag


def prefix_attention(q, k_prefix, v_prefix, prefix_lens, k_suffix, v_suffix, suffix_lens, window: int, scale: float):
    """q [B, Tq, H, D]; caches [G, P_max, H_kv, D] and [B, S_max, H_kv, D]."""
    B, G = q.shape[0], k_prefix.shape[0]
    outs = []
    for b in range(B):
        g = b // (B // G)
        P, S = int(prefix_lens[g]), int(suffix_lens[b])
        k = np.concatenate([k_prefix[g, :P], k_suffix[b, :S]])
        v = np.concatenate([v_prefix[g, :P], v_suffix[b, :S]])
        outs.append(row_attention(q[b], k, v, window, scale))
    return tuple(np.stack(x) for x in zip(*outs))
