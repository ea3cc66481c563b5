"""GPU parity of nc_qk_norm_rope and its backward against the fp64 definition
(oracle/qk_norm_rope.py).

Tolerance, per element.  Storing rounds by at most half a step, h = 2^-8 |y|
in bf16 and 2^-24 |y| in fp32.  Before that, in fp32: the phase is truncated to
2^-32 turns and rounded to 2^-25 turns (together below 2^-22 radians), sin and
cos of it are off by at most 2 units of 2^-24, the two products and their sum
by 3 more, the mean of 128 squares by (16 + 3) 2^-24, halved by the root, and
rsqrt and the scale by 4: together below 2^-19 times the pair's length, which
the rotation keeps.  The gradient has the same terms on |dy|'s pair and, for
the projection, on |x| |x||dy| / (D rho^2), whose dot product and mean add
2 (16 + 3) 2^-24: 2^-18 covers both."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import nc, synth
from oracle import qk_norm_rope as QK

pytestmark = pytest.mark.gpu
D, ALPHA, BASE, EPS = 128, 1.15, 1e5, 1e-6
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _dev(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _draw(rng, shape, dtype):
    a = rng.standard_normal(shape, dtype=np.float32)
    return synth.round_bf16(a) if dtype == "bf16" else a


def _pair(x):
    lo, hi = np.split(np.abs(x), 2, -1)
    n = np.hypot(lo, hi)
    return np.concatenate([n, n], -1)


def _close(got, ref, dtype):
    bound = HALF[dtype] * np.abs(ref) + 2.0 ** -19 * _pair(ref) + 1e-30
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / bound))


def _positions(rng, N):
    p = rng.integers(0, 1 << 17, N)
    p[: min(N, 4)] = [0, 2 ** 31 - 1, 1, 123456789][: min(N, 4)]
    return p


def _status_ok():
    import torch
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0


@pytest.mark.parametrize("N,H,Hkv,dtype", [(1, 1, 1, "bf16"), (1, 12, 12, "bf16"), (33, 12, 4, "bf16"), (7, 3, 1, "fp32"),
                                           (257, 4, 2, "fp32"), (4097, 5, 5, "bf16"), (4099, 2, 1, "fp32")])
def test_forward_dense(N, H, Hkv, dtype):
    import torch
    rng = np.random.default_rng(N + H)
    q, k, pos = _draw(rng, (N, H, D), dtype), _draw(rng, (N, Hkv, D), dtype), _positions(rng, N)
    q[0, 0] = 0.0                                       # a vector of norm 0 stays 0
    qd, kd = _dev(q, dtype), _dev(k, dtype)
    qo, ko = torch.full_like(qd, float("nan")), torch.full_like(kd, float("nan"))
    nc.nc_qk_norm_rope(qd, kd, torch.from_numpy(pos.astype(np.int32)).cuda(), qo, ko)
    _status_ok()
    assert nc.nc_last_launch_count() == 1
    _close(_host(qo), QK.forward(q, pos, ALPHA, BASE, EPS), dtype)
    _close(_host(ko), QK.forward(k, pos, ALPHA, BASE, EPS), dtype)


@pytest.mark.parametrize("N,H,Hkv,dtype", [(1, 4, 4, "bf16"), (50, 12, 3, "bf16"), (31, 2, 2, "fp32"), (5000, 4, 2, "bf16")])
def test_forward_packed_projection_into_a_cache(N, H, Hkv, dtype):
    """q, k, v are slices of one projection; rows of the cache that no token names keep their contents."""
    import torch
    rng = np.random.default_rng(N)
    rows = 2 * N + 3
    qkv, pos = _draw(rng, (N, H + 2 * Hkv, D), dtype), _positions(rng, N)
    slots = rng.permutation(rows)[:N]
    slots[rng.random(N) < 0.2] = -1
    if N > 1:
        slots[N // 2] = -1
    x = _dev(qkv, dtype)
    cache = torch.full((2, rows, Hkv + 1, D), 7.0, dtype=x.dtype, device="cuda")   # a wider row: strided rows
    qo = torch.full((N, 2 * H, D), 5.0, dtype=x.dtype, device="cuda")
    nc.nc_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], torch.from_numpy(pos.astype(np.int32)).cuda(), qo[:, :H],
                       cache[0][:, :Hkv], v=x[:, H + Hkv:], v_out=cache[1][:, :Hkv],
                       slots=torch.from_numpy(slots.astype(np.int32)).cuda())
    _status_ok()
    _close(_host(qo[:, :H]), QK.forward(qkv[:, :H], pos, ALPHA, BASE, EPS), dtype)
    assert np.all(_host(qo[:, H:]) == 5.0)
    keep = slots >= 0
    kc, vc = _host(cache[0]), _host(cache[1])
    _close(kc[slots[keep], :Hkv], QK.forward(qkv[:, H:H + Hkv], pos, ALPHA, BASE, EPS)[keep], dtype)
    assert np.array_equal(vc[slots[keep], :Hkv], qkv[keep, H + Hkv:].astype(np.float64))
    rest = np.setdiff1d(np.arange(rows), slots[keep])
    assert np.all(kc[rest] == 7.0) and np.all(vc[rest] == 7.0) and np.all(kc[:, Hkv:] == 7.0) and np.all(vc[:, Hkv:] == 7.0)


def test_reverse_turns_the_other_way():
    import torch
    rng = np.random.default_rng(9)
    q, k, pos = _draw(rng, (60, 3, D), "fp32"), _draw(rng, (60, 1, D), "fp32"), _positions(rng, 60)
    qd, kd, pd = _dev(q, "fp32"), _dev(k, "fp32"), torch.from_numpy(pos.astype(np.int32)).cuda()
    qo, ko, dq, dk = (torch.empty_like(t) for t in (qd, kd, qd, kd))
    nc.nc_qk_norm_rope(qd, kd, pd, qo, ko, reverse=True)
    _close(_host(qo), QK.forward(q, pos, ALPHA, BASE, EPS, reverse=True), "fp32")
    _close(_host(ko), QK.forward(k, pos, ALPHA, BASE, EPS, reverse=True), "fp32")
    # (dy = x)
    nc.nc_qk_norm_rope_backward(qd, kd, pd, qd, kd, dq, dk, reverse=True)
    _status_ok()
    for got, x in ((dq, q), (dk, k)):
        x64 = x.astype(np.float64)
        ref = QK.backward(x, pos, x, ALPHA, BASE, EPS, reverse=True)
        rho2 = np.mean(x64 ** 2, -1, keepdims=True) + EPS
        size = _pair(x64) + np.abs(x64) * np.sum(x64 ** 2, -1, keepdims=True) / (D * rho2)
        assert np.all(np.abs(_host(got) - ref) <= HALF["fp32"] * np.abs(ref) + 2.0 ** -18 * ALPHA / np.sqrt(rho2) * size)


def test_forward_in_place_equals_out_of_place():
    import torch
    rng = np.random.default_rng(5)
    q, k = _dev(_draw(rng, (100, 6, D), "bf16"), "bf16"), _dev(_draw(rng, (100, 2, D), "bf16"), "bf16")
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    nc.nc_qk_norm_rope(q, k, pos, qo, ko)
    nc.nc_qk_norm_rope(q, k, pos, q, k)
    _status_ok()
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_bad_positions_and_slots_are_flagged():
    import torch
    rng = np.random.default_rng(6)
    q, k = _draw(rng, (3, 2, D), "bf16"), _draw(rng, (3, 1, D), "bf16")
    qd, kd = _dev(q, "bf16"), _dev(k, "bf16")
    for pos, slots in (([5, -3, 9], [0, 1, 2]), ([5, 0, 9], [0, 4, 2]), ([5, 0, 9], [0, -2, 2])):
        qo, cache = torch.empty_like(qd), torch.full((4, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
        nc.nc_qk_norm_rope(qd, kd, torch.tensor(pos, dtype=torch.int32, device="cuda"), qo, cache,
                           slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        rc, bits = nc.nc_get_status()
        assert rc == nc.STATUS_CODES["NC_ERR_DATA"] and bits == 1 << rc
        # a negative position is taken as 0, a slot out of range as -1
        p = np.maximum(pos, 0)
        _close(_host(qo), QK.forward(q, p, ALPHA, BASE, EPS), "bf16")
        kept = [n for n in range(3) if 0 <= slots[n] < 4]
        _close(_host(cache)[[slots[n] for n in kept]], QK.forward(k, p, ALPHA, BASE, EPS)[kept], "bf16")
        rest = [r for r in range(4) if r not in [slots[n] for n in kept]]
        assert np.all(_host(cache)[rest] == 3.0)
    _status_ok()


@pytest.mark.parametrize("N,H,Hkv,dtype", [(1, 2, 1, "bf16"), (40, 12, 12, "bf16"), (333, 6, 3, "fp32"), (4098, 4, 1, "bf16"),
                                           (4100, 1, 1, "fp32")])
def test_backward(N, H, Hkv, dtype):
    import torch
    rng = np.random.default_rng(N + 1)
    qkv, pos = _draw(rng, (N, H + Hkv, D), dtype), _positions(rng, N)
    g = _draw(rng, (N, H + Hkv, D), dtype)
    x, gd = _dev(qkv, dtype), _dev(g, dtype)
    out = torch.full((N, H + Hkv + 1, D), 9.0, dtype=x.dtype, device="cuda")
    nc.nc_qk_norm_rope_backward(x[:, :H], x[:, H:], torch.from_numpy(pos.astype(np.int32)).cuda(), gd[:, :H], gd[:, H:],
                                out[:, :H], out[:, H:H + Hkv])
    _status_ok()
    got = _host(out)
    assert np.all(got[:, H + Hkv:] == 9.0)
    ref = QK.backward(qkv, pos, g, ALPHA, BASE, EPS)
    x64, g64 = qkv.astype(np.float64), g.astype(np.float64)
    rho2 = np.mean(x64 ** 2, -1, keepdims=True) + EPS
    size = _pair(g64) + np.abs(x64) * np.linalg.norm(x64, axis=-1, keepdims=True) * np.linalg.norm(g64, axis=-1, keepdims=True) / (D * rho2)
    bound = HALF[dtype] * np.abs(ref) + 2.0 ** -18 * ALPHA / np.sqrt(rho2) * size
    assert np.all(np.abs(got[:, :H + Hkv] - ref) <= bound), float(np.max(np.abs(got[:, :H + Hkv] - ref) / bound))


def test_backward_against_differences_of_the_forward():
    """Central differences of the fp32 forward along random directions: with step h = 2^-6 the cubic term is about
    h^2 and the rounding 2^-24 sqrt(2 D) |dy| |y| / h, both below 1e-2 of the derivative's size (about |dy| |u| = D)."""
    import torch
    torch.manual_seed(7)
    N, H = 5, 2
    q, dy, u = (torch.randn(N, H, D, device="cuda") for _ in range(3))
    pos = torch.tensor([0, 3, 700, 65536, 999999], dtype=torch.int32, device="cuda")

    def f(x):
        y, k = torch.empty_like(x), torch.empty_like(x)
        nc.nc_qk_norm_rope(x, x, pos, y, k)
        return (y.double() * dy.double()).sum(-1)

    dq, dk = torch.empty_like(q), torch.empty_like(q)
    nc.nc_qk_norm_rope_backward(q, q, pos, dy, dy, dq, dk)
    _status_ok()
    assert torch.equal(dq, dk)
    h = 2.0 ** -6
    diff = (f(q + h * u) - f(q - h * u)) / (2 * h)
    assert float((diff - (dq.double() * u.double()).sum(-1)).abs().max()) <= 1e-2 * D


def test_captured_and_replayed_on_another_stream():
    import torch
    rng = np.random.default_rng(8)
    q, k = _dev(_draw(rng, (9, 4, D), "bf16"), "bf16"), _dev(_draw(rng, (9, 2, D), "bf16"), "bf16")
    pos, slots = torch.arange(9, dtype=torch.int32, device="cuda"), torch.arange(9, dtype=torch.int32, device="cuda")
    qo, cache = torch.zeros_like(q), torch.zeros(30, 2, D, dtype=q.dtype, device="cuda")
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        nc.nc_qk_norm_rope(q, k, pos, qo, cache, slots=slots)
    for step in range(3):                                # the next tokens: other positions, other slots
        graph.replay()
        torch.cuda.synchronize()
        q2, c2 = torch.empty_like(q), torch.zeros_like(cache)
        nc.nc_qk_norm_rope(q, k, pos, q2, c2, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(q2, qo) and torch.equal(c2[9 * step:9 * step + 9], cache[9 * step:9 * step + 9])
        pos += 1
        slots += 9
    _status_ok()
