"""nc_policy_loss where old, reference and present log-probabilities lie far
apart, in each form of the kernel, against the fp64 definition
(oracle/policy_loss.py).

Gradients are held to the bound that test_gpu_policy_loss.py derives.  A KL
term is the difference of an exponential's excess and d, each within 2^-23
relative (expm1f within 1 ulp, d rounded once from fp64), beside what follows
from lp: the statistics may be off by 2^-22 of the terms' sizes more."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import synth
from oracle import policy_loss as PL
from test_gpu_policy_loss import HALF, _run

pytestmark = pytest.mark.gpu
LOW, HIGH = float(np.float32(0.2)), float(np.float32(0.28))
FORMS = [(300, "fp32"), (300, "bf16"), (4099, "fp32"), (9001, "fp32"), (20491, "bf16")]  # warp, rows, ring


def _logits(seed, T, V, dtype):
    rng = np.random.default_rng(seed)
    z = (2 * rng.standard_normal((1, T, V))).astype(np.float32)
    if dtype == "bf16":
        z = synth.round_bf16(z)
    y = rng.integers(0, V, (1, T)).astype(np.int32)
    return z, y, PL.log_probs(z, y)[0]


def _gradient_close(dz, want, dtype):
    bound = HALF[dtype] * np.abs(want["dz"]) + 2.0 ** -15 * want["size"][..., None] * (want["p"] + want["hot"]) + 2.0 ** -126
    assert np.isfinite(want["dz"]).all() and np.all(np.abs(dz - want["dz"]) <= bound), float(np.max(np.abs(dz - want["dz"]) / bound))


@pytest.mark.parametrize("V,dtype", FORMS)
def test_a_reference_that_gives_the_token_almost_no_probability(V, dtype):
    """d far below 0: the KL term grows like -d and its gradient tends to beta, also for a reference of -inf."""
    ds = [-0.6, -20.0, -300.0, -2.0 ** 26, -2.0 ** 31, -np.inf]
    z, y, lp = _logits(V, len(ds), V, dtype)
    ref = (lp + np.array([ds])).astype(np.float32)
    adv = np.array([[0.0, 1e-3, -1e-3, 0.5, -0.5, 2e-2]], np.float32)
    for n in (len(ds), len(ds) - 1):                         # with and without the infinite one
        y1 = y.copy()
        y1[:, n:] = -1
        stats, logp, dz = _run(z, y1, adv, None, ref, dtype, 0.2, 0.28, 0.25, 0)
        want = PL.policy_loss(z, y1, adv, None, ref, LOW, HIGH, 0.25, 0)
        _gradient_close(dz, want, dtype)
        if n == len(ds):
            assert stats[0] == np.inf and stats[1] == np.inf
        else:
            kl = want["stats"][1]
            assert abs(stats[1] - kl) <= 2.0 ** -16 * want["size"].sum() + (2.0 ** -22 + 2.0 ** -24) * kl
            assert abs(stats[0] - want["stats"][0]) <= 2.0 ** -16 * want["size"].sum() + (2.0 ** -22 + 2.0 ** -24) * 0.25 * kl
        assert stats[2] == 0


@pytest.mark.parametrize("V,dtype", FORMS)
def test_a_term_of_weight_zero_is_left_out_however_large(V, dtype):
    """No KL weight and a token that the reference finds e^100 times as likely (the KL statistic alone passes fp32);
    no advantage and a ratio beyond fp32's and fp64's range, or of an old policy that could not draw the token."""
    z, y, _ = _logits(V + 1, 6, V, dtype)
    np.put_along_axis(z[0, :3], y[0, :3, None], -100.0, -1)
    lp = PL.log_probs(z, y)[0]
    ref = np.where(np.arange(6) < 3, -5.0, lp - 0.3).astype(np.float32)
    adv = np.array([[0.7, -0.7, 0.0, 0.0, 0.0, 0.0]], np.float32)
    old = (lp - np.array([[0.05, 0.05, 0.05, 100.0, 1000.0, np.inf]])).astype(np.float32)
    stats, logp, dz = _run(z, y, adv, old, ref, dtype, 0.2, 0.28, 0.0, 0)
    want = PL.policy_loss(z, y, adv, np.where(adv == 0, lp, old), ref, LOW, HIGH, 0.0, 0)
    _gradient_close(dz, want, dtype)
    assert np.all(dz[0, 2:] == 0) and stats[1] == np.inf and stats[2] == 0
    assert abs(stats[0] - want["stats"][0]) <= 2.0 ** -16 * np.abs(want["slope"]).sum() + 2.0 ** -24 * abs(want["stats"][0])
    # no KL term at all gives the same loss and gradient
    stats2, _, dz2 = _run(z, y, adv, old, None, dtype, 0.2, 0.28, 0.0, 0)
    assert stats2[0] == stats[0] and np.array_equal(dz2, dz) and stats2[1] == 0


@pytest.mark.parametrize("V", [300, 4099, 9001])
def test_logits_that_are_not_numbers_show_in_the_loss_without_an_advantage(V):
    z, y, lp = _logits(V + 2, 3, V, "fp32")
    z[0, 1, 5] = np.nan
    stats, logp, dz = _run(z, y, np.zeros((1, 3), np.float32), lp.astype(np.float32), None, "fp32", 0.2, 0.28, 0.0, 0)
    assert np.isnan(stats[0]) and np.isnan(logp[0, 1]) and np.isnan(dz[0, 1]).all()
    assert np.isfinite(logp[0, ::2]).all() and np.all(dz[0, ::2] == 0)


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("V,dtype", FORMS)
def test_exponentials_beyond_fp32_whose_weighted_terms_fit(V, dtype, norm):
    """Ratios and KL terms of e^90 = 1.2e39: with the weight (1/8 here), the advantage and kl_beta they fit fp32 again.
    The statistic of the KL term has the weight alone, its error follows lp's (2^-17 + 2^-24 |lp| in the exponent)."""
    T, beta = 8, 0.02
    z, y, _ = _logits(V + 3, T, V, dtype)
    np.put_along_axis(z[0, 4:6], y[0, 4:6, None], -100.0, -1)
    lp = PL.log_probs(z, y)[0]
    d = np.array([[0.1, -0.2, 0.3, 0.0, 90.0, 85.0, -0.1, 0.2]])
    x = np.array([[90.0, 85.0, 82.0, 90.0, 0.1, -0.1, 0.1, 79.0]])
    adv = np.array([[-0.1, -1e-30, -0.5, 0.9, 0.5, -0.5, 0.3, -0.1]], np.float32)
    old, ref = (lp - x).astype(np.float32), (lp + d).astype(np.float32)
    stats, logp, dz = _run(z, y, adv, old, ref, dtype, 0.2, 0.28, beta, norm)
    want = PL.policy_loss(z, y, adv, old, ref, LOW, HIGH, beta, norm)
    assert np.abs(want["dz"]).max() > 1e36 and want["stats"][1] > 1e38
    _gradient_close(dz, want, dtype)
    assert abs(stats[0] - want["stats"][0]) <= 2.0 ** -16 * want["size"].sum() + 2.0 ** -24 * abs(want["stats"][0])
    assert abs(stats[1] - want["stats"][1]) <= 2.0 ** -15 * want["stats"][1] and abs(stats[2] - want["stats"][2]) <= 2.0 ** -24
