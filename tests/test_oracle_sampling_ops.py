"""Pins of the fp64 definitions behind nc_qk_norm_rope, nc_prefix_attention and
nc_policy_loss: closed forms, brute force, and differences for the gradients.

Central differences with step h of a smooth f of size O(1) are off by
O(h^2) + 2^-52 / h; with h = 1e-5 both are near 1e-10, held at 1e-6."""
import numpy as np
import pytest

from oracle import nanochat_fwd as O
from oracle import policy_loss as PL
from oracle import prefix_attention as PA
from oracle import qk_norm_rope as QK

RNG = np.random.default_rng


def test_qk_norm_keeps_norm_and_depends_on_distance_only():
    rng = RNG(1)
    x, y = rng.standard_normal((5, 2, 128)), rng.standard_normal((5, 2, 128))
    pos = np.array([0, 1, 17, 4096, 2 ** 31 - 1])
    a = QK.forward(x, pos, 1.15, 1e5, 0.0)
    assert np.allclose(np.linalg.norm(a, axis=-1), 1.15 * np.sqrt(128), atol=1e-9)
    assert np.allclose(QK.forward(x, np.zeros(5), 1.15, 1e5, 0.0)[0], a[0], atol=0)  # position 0 turns nothing
    s1 = np.sum(QK.rope(x[:4], pos[:4], 1e5) * QK.rope(y[:4], pos[:4] + 9, 1e5), -1)
    s2 = np.sum(QK.rope(x[:4], pos[:4] + 100, 1e5) * QK.rope(y[:4], pos[:4] + 109, 1e5), -1)
    assert np.allclose(s1, s2, atol=1e-8)


def test_qk_norm_is_that_of_the_model():
    x, pos = RNG(5).standard_normal((6, 3, 128)), np.array([0, 1, 2, 77, 2047, 100000])
    want = O.qk_norm(O.rope(x, pos, 1e5), 1.15, 1e-6)
    assert np.allclose(QK.forward(x, pos, 1.15, 1e5, 1e-6), want, atol=1e-12)
    assert np.allclose(QK.rope(QK.rope(x, pos, 1e5), pos, 1e5, reverse=True), x, atol=1e-12)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_qk_norm_gradient_against_differences(eps):
    rng = RNG(2)
    x, dy, pos = rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 2, 16)), np.array([0, 5, 1000])
    got = QK.backward(x, pos, dy, 1.15, 1e4, eps)
    h = 1e-5
    for idx in [(0, 0, 0), (0, 1, 9), (1, 0, 3), (1, 1, 15), (2, 0, 8), (2, 1, 7)]:
        e = np.zeros_like(x)
        e[idx] = h
        f = lambda t: np.sum(dy * QK.forward(t, pos, 1.15, 1e4, eps))
        assert abs((f(x + e) - f(x - e)) / (2 * h) - got[idx]) < 1e-6


@pytest.mark.parametrize("P,S,window", [(9, 0, 0), (0, 9, 0), (5, 4, 0), (5, 4, 3), (8, 1, 1)])
def test_prefix_attention_equals_causal_attention_of_the_joined_sequence(P, S, window):
    rng = RNG(3)
    L, H, Hkv, D = P + S, 4, 2, 8
    k, v = rng.standard_normal((L, Hkv, D)), rng.standard_normal((L, Hkv, D))
    q = rng.standard_normal((L, H, D))
    ref = O.attention(q, k, v, window or L, D ** -0.5)
    Tq = 3
    pad = np.full((1, 2, Hkv, D), np.nan)
    kp, vp = np.concatenate([k[None, :P], pad], 1), np.concatenate([v[None, :P], pad], 1)
    ks, vs = np.concatenate([k[None, P:], pad], 1), np.concatenate([v[None, P:], pad], 1)
    o, lse, _ = PA.prefix_attention(q[None, -Tq:], kp, vp, [P], ks, vs, [S], window, D ** -0.5)
    assert np.allclose(o[0], ref[-Tq:], atol=1e-12)
    s = (q[-1, 3] @ k[(0 if not window else L - min(L, window)):, 1].T) * D ** -0.5
    assert np.allclose(lse[0, -1, 3], np.log(np.exp(s).sum()), atol=1e-12)


def test_prefix_attention_without_keys():
    q = np.ones((2, 2, 1, 4))
    e = np.zeros((1, 3, 1, 4))
    o, lse, _ = PA.prefix_attention(q, e, e, [0], np.zeros((2, 2, 1, 4)), np.ones((2, 2, 1, 4)), [0, 1], 0, 1.0)
    assert np.all(o[0] == 0) and np.all(lse[0] == -np.inf)
    # row 1 has one key: its first query stands before it, its second sees it alone
    assert np.all(o[1, 0] == 0) and np.all(o[1, 1] == 1) and lse[1, 0, 0] == -np.inf and lse[1, 1, 0] == 0


def test_policy_loss_closed_forms():
    # two words, logits (0, 0): lp = -log 2; r = 1 without an old policy, so L = -A
    z = np.zeros((1, 3, 2))
    got = PL.policy_loss(z, [[0, 1, -1]], np.array([2.0]))
    assert np.allclose(got["stats"], [-2.0, 0, 0]) and np.allclose(got["lp"], [[-np.log(2), -np.log(2), 0]])
    assert np.allclose(got["dz"], [[[-0.5, 0.5], [0.5, -0.5], [0, 0]]])
    # r = 2 with A > 0 is cut at 1.2 and has no gradient; with A < 0 it is not cut
    old = np.full((1, 3), -2 * np.log(2))
    up = PL.policy_loss(z, [[0, -1, -1]], np.array([1.0]), old=old)
    assert np.allclose(up["stats"], [-1.2, 0, 1]) and np.all(up["dz"] == 0)
    down = PL.policy_loss(z, [[0, -1, -1]], np.array([-1.0]), old=old)
    assert np.allclose(down["stats"], [2.0, 0, 0]) and np.allclose(down["dz"][0, 0], [1.0, -1.0])
    # by sequences: one token of the first row weighs as much as two of the second
    w = PL.weights(np.array([[0, -1], [0, 0], [-1, -1]]), 1)
    assert np.allclose(w, [[0.5, 0], [0.25, 0.25], [0, 0]])
    assert np.all(PL.weights(np.full((2, 2), -1), 0) == 0) and np.all(PL.weights(np.full((2, 2), -1), 1) == 0)


@pytest.mark.parametrize("norm,beta", [(0, 0.0), (1, 0.3)])
def test_policy_loss_gradient_against_differences(norm, beta):
    rng = RNG(4)
    B, T, V = 2, 4, 7
    z = rng.standard_normal((B, T, V))
    y = rng.integers(0, V, (B, T))
    y[1, 2:] = -1
    lp, _ = PL.log_probs(z, y)
    x = np.array([[0.1, 0.5, -0.5, -0.1], [0.6, -0.4, 0, 0]])      # away from both borders
    kw = dict(old=lp - x, ref=lp + rng.standard_normal((B, T)), beta=beta, norm=norm)
    if not beta:
        kw["ref"] = None
    A = np.array([1.3, -0.7])
    got = PL.policy_loss(z, y, A, **kw)
    h = 1e-5
    for idx in np.ndindex(B, T, V):
        e = np.zeros_like(z)
        e[idx] = h
        f = lambda t: PL.policy_loss(t, y, A, **kw)["stats"][0]
        assert abs((f(z + e) - f(z - e)) / (2 * h) - got["dz"][idx]) < 1e-6
