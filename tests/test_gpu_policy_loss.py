"""GPU parity of nc_policy_loss against the fp64 definition
(oracle/policy_loss.py).

Tolerance.  A weight exp(z - max) is off by 2^-22 (the exponential) and by
2^-24 times its argument (at most 2^-19 where it counts: e^-x x < 0.37), and
passes through at most 50 roundings of a thread's sum in fp32 (words of a
chunk first, then the chunks); what lies across threads and the logarithm are
fp64.  Together that is below
2^-17 relative, so lp is off by at most 2^-17 + 2^-24 |lp|.  The ratio and the
KL term follow lp: dL/dlp is off by at most 2^-16 of its terms' size, a
gradient element by 2^-15 of that size times (p + [v = y]), plus half a step of
its type (2^-8 in bf16, 2^-24 in fp32, relative); the statistics by 2^-16 of
the sum of the terms' sizes plus 2^-24 relative.  Elements below 2^-126 may be
flushed to zero.  The inputs keep every ratio at least 1e-2 from both borders,
so the branch taken does not depend on rounding."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import nc, synth
from oracle import policy_loss as PL

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _t(a, dtype=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if dtype is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def _case(seed, B, T, V, dtype, low=0.2, high=0.28, scale=2.0):
    rng = np.random.default_rng(seed)
    z = (scale * rng.standard_normal((B, T, V))).astype(np.float32)
    y = rng.integers(0, V, (B, T)).astype(np.int32)
    if dtype == "bf16":
        z = synth.round_bf16(z)
    if B * T > 2:
        y[rng.random((B, T)) < 0.3] = -1
    lp, _ = PL.log_probs(z, y)
    lo, hi = np.log(1 - low) if low < 1 else -9.0, np.log(1 + high)
    x = rng.uniform(-0.8, 0.8, (B, T))
    for edge in (lo, hi):
        x = np.where(np.abs(x - edge) < 0.02, x + 0.05, x)
    old = (lp - x).astype(np.float32)
    ref = (lp + rng.normal(0, 0.5, (B, T))).astype(np.float32)
    return z, y, old, ref, rng.standard_normal((B, T)).astype(np.float32)


def _run(z, y, adv, old, ref, dtype, low, high, beta, norm, ldl=None, lddl=None, grad=True, shift=0):
    """Logits in rows ldl apart that start `shift` elements into their buffer, surrounded by NaN."""
    import torch
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, T, V = z.shape

    def rows(ld):
        return torch.full((B * T * ld + 16,), float("nan"), dtype=td, device="cuda")[shift:shift + B * T * ld].view(B, T, ld)

    zb = rows(ldl or V)
    zb[:, :, :V] = _t(z, td)
    db = rows(lddl or V) if grad else None
    stats, logp = torch.full((3,), float("nan"), device="cuda"), torch.full((B, T), float("nan"), device="cuda")
    nc.nc_policy_loss(zb[:, :, :V], _t(y), _t(adv), stats, logp, db[:, :, :V] if grad else None,
                      old_logp=None if old is None else _t(old), ref_logp=None if ref is None else _t(ref),
                      clip_low=low, clip_high=high, kl_beta=beta, norm=norm)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0 and nc.nc_last_launch_count() == 2
    if grad and (lddl or V) > V:
        assert bool(torch.isnan(db[:, :, V:]).all())          # columns behind the vocabulary are not written
    f = lambda t: t.double().cpu().numpy()
    return f(stats), f(logp), f(db[:, :, :V]) if grad else None


def _check(got, want, dtype):
    stats, logp, dz = got
    size, p, hot = want["size"], want["p"], want["hot"]
    lp = want["lp"]
    assert np.all(np.abs(logp - lp) <= (2.0 ** -17 + 2.0 ** -24 * np.abs(lp)) * (lp != 0))
    if dz is not None:
        bound = HALF[dtype] * np.abs(want["dz"]) + 2.0 ** -15 * size[..., None] * (p + hot) + 2.0 ** -126
        assert np.all(np.abs(dz - want["dz"]) <= bound), float(np.max(np.abs(dz - want["dz"]) / bound))
    assert np.all(np.abs(stats - want["stats"]) <= 2.0 ** -16 * (size.sum() + 1e-9) + 2.0 ** -24 * np.abs(want["stats"]))


@pytest.mark.parametrize("B,T,V,dtype,norm,beta,per_token", [
    (1, 1, 1, "fp32", 0, 0.0, False),                        # one word: p = 1, no gradient
    (1, 1, 5, "bf16", 1, 0.1, True),
    (2, 3, 33, "fp32", 0, 0.05, False),
    (3, 5, 1000, "fp32", 1, 0.05, True),
    (3, 7, 1001, "bf16", 1, 0.05, False),                    # odd rows: every alignment
    (2, 300, 513, "fp32", 0, 0.0, True),
    (5, 1100, 40, "fp32", 1, 0.1, True),                     # two rows per warp
    (2, 7, 2048, "fp32", 0, 0.05, False),                    # the border of 8 KB a row, and beyond
    (2, 7, 2049, "fp32", 0, 0.05, False),
    (3, 400, 2051, "fp32", 1, 0.05, False),                  # several rows per CTA
    (4, 90, 4099, "bf16", 0, 0.2, True),                     # more rows than CTAs
    (1, 5, 32768, "fp32", 0, 0.05, False),
    (1, 3, 40009, "fp32", 1, 0.05, False),
    (1, 3, 40009, "bf16", 0, 0.05, False),
    (2, 2, 8193, "fp32", 0, 0.05, True),
    (2, 2, 16391, "bf16", 1, 0.05, True),
    (2, 3, 5121, "fp32", 0, 0.05, True),                     # the borders of 20 and 40 KB a row, few rows
    (2, 3, 20480, "bf16", 1, 0.05, True),
    (3, 150, 5120, "fp32", 0, 0.05, True),                   # and many
    (3, 150, 5123, "fp32", 1, 0.05, True),
    (3, 130, 20479, "bf16", 0, 0.05, True),
    (3, 130, 12289, "fp32", 0, 0.05, True),                  # the border of 48 KB
    (1, 3, 60001, "fp32", 0, 0.05, False),                   # a row longer than shared memory
    (3, 150, 9001, "fp32", 1, 0.0, False),                   # several long rows per CTA
    (3, 150, 20011, "bf16", 1, 0.05, True),
    (2, 600, 17, "fp32", 1, 0.05, True),                     # more tokens than threads
])
def test_against_the_definition(B, T, V, dtype, norm, beta, per_token):
    low, high = 0.2, 0.28
    z, y, old, ref, adv = _case(B * T + V, B, T, V, dtype, low, high)
    adv = adv if per_token else adv[:, 0]
    ref = ref if beta else None
    got = _run(z, y, adv, old, ref, dtype, low, high, beta, norm)
    low32, high32 = float(np.float32(low)), float(np.float32(high))
    _check(got, PL.policy_loss(z, y, adv, old, ref, low32, high32, beta, norm), dtype)


def test_on_policy_without_clipping_range():
    """No old log-probabilities: r = 1, on both borders of an empty range, and the gradient is that of r A."""
    z, y, _, ref, adv = _case(1, 2, 9, 257, "fp32")
    got = _run(z, y, adv, None, ref, "fp32", 0.0, 0.0, 0.1, 0)
    want = PL.policy_loss(z, y, adv, None, ref, 0.0, 0.0, 0.1, 0)
    assert want["stats"][2] == 0 and got[0][2] == 0
    _check(got, want, "fp32")


@pytest.mark.parametrize("dtype,ldl,lddl,shift", [("fp32", 261, 259, 0), ("fp32", 260, 264, 1), ("bf16", 259, 259, 3),
                                                  ("bf16", 264, 257, 0)])
def test_strided_rows_and_odd_starts(dtype, ldl, lddl, shift):
    z, y, old, ref, adv = _case(2, 2, 6, 257, dtype)
    got = _run(z, y, adv[:, 0], old, ref, dtype, 0.2, 0.28, 0.05, 0, ldl, lddl, shift=shift)
    _check(got, PL.policy_loss(z, y, adv[:, 0], old, ref, float(np.float32(0.2)), float(np.float32(0.28)), 0.05, 0), dtype)


@pytest.mark.parametrize("dtype,V,ldl,lddl,shift", [("fp32", 9001, 9002, 9003, 1), ("bf16", 20011, 20013, 20016, 5)])
def test_strided_long_rows(dtype, V, ldl, lddl, shift):
    z, y, old, ref, adv = _case(10, 2, 3, V, dtype)
    got = _run(z, y, adv[:, 0], old, ref, dtype, 0.2, 0.28, 0.05, 0, ldl, lddl, shift=shift)
    _check(got, PL.policy_loss(z, y, adv[:, 0], old, ref, float(np.float32(0.2)), float(np.float32(0.28)), 0.05, 0), dtype)


@pytest.mark.parametrize("V", [700, 9001, 60001])
def test_loss_alone_equals_the_loss_with_gradient(V):
    z, y, old, ref, adv = _case(3, 3, 8, V, "fp32")
    a = _run(z, y, adv, old, ref, "fp32", 0.2, 0.28, 0.05, 1)
    b = _run(z, y, adv, old, ref, "fp32", 0.2, 0.28, 0.05, 1, grad=False)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_gradient_in_the_place_of_the_logits():
    import torch
    for dtype, td, V in (("fp32", torch.float32, 1003), ("bf16", torch.bfloat16, 1003), ("fp32", torch.float32, 4099),
                         ("bf16", torch.bfloat16, 12001), ("fp32", torch.float32, 9001), ("fp32", torch.float32, 60001)):
        z, y, old, _, adv = _case(4, 2, 40 if V < 2000 else 4, V, dtype)
        want = _run(z, y, adv, old, None, dtype, 0.2, 0.28, 0.0, 0)
        zd, stats, logp = _t(z, td), torch.empty(3, device="cuda"), torch.empty(y.shape, device="cuda")
        nc.nc_policy_loss(zd, _t(y), _t(adv), stats, logp, zd, old_logp=_t(old), clip_low=0.2, clip_high=0.28)
        torch.cuda.synchronize()
        assert np.array_equal(zd.double().cpu().numpy(), want[2]) and np.array_equal(stats.double().cpu().numpy(), want[0])


def test_nothing_to_learn_from():
    z, y, old, ref, adv = _case(5, 2, 4, 50, "fp32")
    y[:] = -1
    for norm in (0, 1):
        stats, logp, dz = _run(z, y, adv, old, ref, "fp32", 0.2, 0.28, 0.1, norm)
        assert np.all(stats == 0) and np.all(logp == 0) and np.all(dz == 0)
    y[1, 2] = 7                                              # one token of one sequence
    for norm in (0, 1):
        _check(_run(z, y, adv, old, ref, "fp32", 0.2, 0.28, 0.1, norm),
               PL.policy_loss(z, y, adv, old, ref, float(np.float32(0.2)), float(np.float32(0.28)), 0.1, norm), "fp32")


def test_masked_words_and_padding_of_any_value():
    """-inf and the type's lowest value have probability 0; rows without a target may hold NaN."""
    z, y, old, ref, adv = _case(6, 2, 4, 300, "fp32")
    y[0, 0], y[1, 1], y[1, 3] = 5, 6, -1
    hide = np.ones((2, 4, 300), bool)
    np.put_along_axis(hide, np.maximum(y, 0)[..., None], False, -1)
    hide[:, :, ::2] = False
    z[hide] = -np.inf
    z[0][hide[0]] = np.finfo(np.float32).min
    lp, _ = PL.log_probs(z, y)
    old, ref = (lp - 0.1).astype(np.float32), (lp + 0.3).astype(np.float32)
    want = PL.policy_loss(z, y, adv, old, ref, float(np.float32(0.2)), float(np.float32(0.28)), 0.1, 0)
    pad = z.copy()
    pad[1, 3] = np.nan
    got = _run(pad, y, adv, old, ref, "fp32", 0.2, 0.28, 0.1, 0)
    _check(got, want, "fp32")
    assert np.all(got[2][hide] == 0) and np.all(got[2][1, 3] == 0)


def test_large_logits_keep_their_differences():
    """Adding 2^12 to integer logits changes nothing: the maximum is subtracted first, exactly."""
    rng = np.random.default_rng(7)
    z = rng.integers(-20, 20, (1, 6, 999)).astype(np.float32)
    y, adv = rng.integers(0, 999, (1, 6)).astype(np.int32), np.ones((1, 6), np.float32)
    a = _run(z, y, adv, None, None, "fp32", 0.2, 0.2, 0.0, 0)
    b = _run(z + 4096, y, adv, None, None, "fp32", 0.2, 0.2, 0.0, 0)
    assert np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])


def test_bad_targets_are_flagged_and_left_out():
    import torch
    z, y, old, ref, adv = _case(8, 2, 5, 60, "fp32")
    y[:] = 3
    want_y = y.copy()
    y[0, 1], y[1, 4] = 60, -2
    want_y[0, 1] = want_y[1, 4] = -1
    for norm in (0, 1):
        stats, logp, dz = torch.empty(3, device="cuda"), torch.empty(2, 5, device="cuda"), torch.empty(2, 5, 60, device="cuda")
        nc.nc_policy_loss(_t(z), _t(y), _t(adv), stats, logp, dz, kl_beta=0.1, ref_logp=_t(ref), norm=norm)
        torch.cuda.synchronize()
        rc, bits = nc.nc_get_status()
        assert rc == nc.STATUS_CODES["NC_ERR_DATA"] and bits == 1 << rc
        _check(tuple(t.double().cpu().numpy() for t in (stats, logp, dz)), PL.policy_loss(z, want_y, adv, None, ref, 0.2, 0.2, 0.1, norm), "fp32")


def test_captured_and_replayed_is_bit_identical():
    import torch
    z, y, old, ref, adv = _case(9, 4, 200, 2001, "fp32")
    t = [_t(a) for a in (z, y, adv, old, ref)]
    ws = torch.empty(nc.nc_policy_loss_workspace_bytes(), dtype=torch.uint8, device="cuda")
    new = lambda: (torch.empty(3, device="cuda"), torch.empty(4, 200, device="cuda"), torch.empty_like(t[0]))
    got, want = new(), new()
    call = lambda o: nc.nc_policy_loss(t[0], t[1], t[2], *o, old_logp=t[3], ref_logp=t[4], kl_beta=0.05, workspace=ws)
    call(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
