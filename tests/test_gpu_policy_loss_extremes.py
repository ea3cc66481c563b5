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
