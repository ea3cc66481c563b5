"""GPU parity of nc_prefix_attention against the fp64 definition
(oracle/prefix_attention.py), per element.

Tolerance.  A score scale q.k is summed in fp32 over 128 products: off by at
most e = 128 * 2^-23 * scale * sum|q_d k_d|, which scale |q| |k| bounds.  A
weight p = 2^(s - m) is off by e, 2^-22 from the exponential and 2^-20 from the
arguments' rounding, and by 2^-8 when it enters P V in bf16; the sum of the
weights by the first three.  So o is off by at most
  (2^-8 + 2 e + 2^-18) sum p|v| + 2^-8 |o|  (its own rounding to bf16),
and the log-sum-exp by e + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import nc, synth
from oracle import prefix_attention as PA

pytestmark = pytest.mark.gpu
D = 128


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)


def _i32(a):
    import torch
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def _bf(rng, *shape):
    return synth.round_bf16(rng.standard_normal(shape, dtype=np.float32))


def _inputs(seed, B, G, Tq, H, Hkv, P, S, sharp=1.0):
    rng = np.random.default_rng(seed)
    q = synth.round_bf16(rng.standard_normal((B, Tq, H, D), dtype=np.float32) * np.float32(sharp))
    return q, _bf(rng, G, P, Hkv, D), _bf(rng, G, P, Hkv, D), _bf(rng, B, S, Hkv, D), _bf(rng, B, S, Hkv, D)


def _check(got, lse, q, kp, vp, pl, ks, vs, sl, window, scale):
    o, l, mag = PA.prefix_attention(q, kp, vp, pl, ks, vs, sl, window, scale)
    kmax = max([np.linalg.norm(c[i, :n].astype(np.float64), axis=-1).max() for c, ns in ((kp, pl), (ks, sl))
                for i, n in enumerate(ns) if n > 0], default=0.0)
    e = 2.0 ** -16 * scale * np.linalg.norm(q.astype(np.float64), axis=-1) * kmax
    bound = (2.0 ** -8 + 2 * e + 2.0 ** -18)[..., None] * mag + 2.0 ** -8 * np.abs(o) + 1e-30
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - o) <= bound), float(np.max(np.abs(got - o) / bound))
    empty = l == -np.inf
    assert np.array_equal(empty, lse == -np.inf) and np.all(got[empty] == 0)
    l0 = np.where(empty, 0.0, l)
    assert np.all(np.abs(np.where(empty, 0.0, lse) - l0) <= e + 2.0 ** -20 * (1 + np.abs(l0)))


def _run(q, kp, vp, pl, ks, vs, sl, window=0, scale=None):
    """Through the binding; cache rows behind the lengths hold NaN."""
    import torch
    t = [_dev(x) for x in (kp, vp, ks, vs)]
    for c, ns in ((t[0], pl), (t[1], pl), (t[2], sl), (t[3], sl)):
        for i, n in enumerate(ns):
            c[i, n:] = float("nan")
    qd = _dev(q)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    nc.nc_prefix_attention(qd, t[0], t[1], _i32(pl), t[2], t[3], _i32(sl), out, out_lse=lse, window=window, softmax_scale=scale)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("B,G,Tq,H,Hkv,pl,sl,window", [
    (1, 1, 1, 1, 1, [1], [0], 0),                                    # one key in all
    (1, 1, 1, 1, 1, [0], [1], 0),
    (2, 1, 1, 2, 2, [64], [0, 1], 0),                                # a whole tile, then one key
    (3, 1, 1, 4, 2, [65], [63, 64, 65], 0),
    (4, 2, 1, 3, 1, [200, 7], [5, 0, 130, 1], 0),                    # ragged groups
    (4, 2, 3, 4, 4, [129, 300], [3, 2, 77, 1], 0),                   # rows with fewer own keys than queries
    (2, 1, 5, 6, 2, [0], [3, 5], 0),                                 # queries before the first key: empty rows
    (2, 2, 2, 2, 1, [0, 40], [0, 0], 0),                             # a row without any key
    (3, 1, 1, 2, 2, [500], [10, 200, 0], 64),                        # window: prefix seen in part, not at all, at its end
    (3, 1, 4, 2, 2, [500], [10, 200, 0], 1),                         # each query sees itself alone
    (3, 1, 2, 4, 2, [0], [0, 0, 0], 0),                              # no keys at all
    (3, 1, 2, 4, 2, [0], [0, 0, 0], 5),
    (2, 1, 130, 1, 1, [70], [130, 200], 0),                          # several query tiles per row
    (2, 1, 130, 2, 1, [70], [131, 190], 50),
    (40, 1, 1, 12, 3, [333], [0] * 20 + list(range(1, 21)), 0),      # 160 query rows per key head: two tiles
    (2, 1, 1, 128, 1, [100], [3, 9], 0),                             # 128 query heads on one key head
    (6, 3, 1, 96, 2, [100, 1, 64], [3, 9, 0, 1, 2, 64], 0),          # 48 rows per token: two tokens fit a tile
    (5, 1, 2, 4, 4, [3000], [900, 1, 450, 30, 2], 0),                # many splits
    (1, 1, 1, 12, 1, [9000], [3], 0),                                # a row of some fifty pieces
    (5, 1, 2, 4, 4, [3000], [900, 1, 450, 30, 2], 1000),
])
def test_against_the_definition(B, G, Tq, H, Hkv, pl, sl, window):
    q, kp, vp, ks, vs = _inputs(B + Tq + H, B, G, Tq, H, Hkv, max(pl) + 5, max(sl) + 3)
    got, lse = _run(q, kp, vp, pl, ks, vs, sl, window)
    _check(got, lse, q, kp, vp, pl, ks, vs, sl, window, D ** -0.5)


@pytest.mark.parametrize("side", ["prefix", "suffix"])
def test_one_side_alone(side):
    import torch
    q, kp, vp, ks, vs = _inputs(11, 3, 1, 2, 4, 2, 200, 200)
    qd, out, lse = _dev(q), torch.empty(3, 2, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, 4, device="cuda")
    if side == "prefix":
        nc.nc_prefix_attention(qd, _dev(kp), _dev(vp), _i32([190]), None, None, None, out, out_lse=lse)
        args = (kp, vp, [190], ks, vs, [0, 0, 0])
    else:
        nc.nc_prefix_attention(qd, None, None, None, _dev(ks), _dev(vs), _i32([200, 2, 71]), out, out_lse=lse)
        args = (kp, vp, [0], ks, vs, [200, 2, 71])
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    _check(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), q, *args, 0, D ** -0.5)


def test_one_tile_of_own_keys():
    """Rows of at most one key tile, no prefix: each row is one piece."""
    import torch
    q, _, _, ks, vs = _inputs(12, 3, 1, 1, 2, 1, 1, 60)
    out, lse = torch.empty(3, 1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 1, 2, device="cuda")
    nc.nc_prefix_attention(_dev(q), None, None, None, _dev(ks), _dev(vs), _i32([60, 0, 9]), out, out_lse=lse)
    torch.cuda.synchronize()
    assert nc.nc_last_launch_count() == 2 and nc.nc_get_status()[0] == 0
    e = np.zeros((1, 1, 1, D), np.float32)
    _check(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), q, e, e, [0], ks, vs, [60, 0, 9], 0, D ** -0.5)


@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_flat_and_sharp_scores(sharp):
    """All scores equal, and scores of size 30: a running maximum that moves by more than 2^8 from tile to tile."""
    pl, sl = [700], [100, 3]
    q, kp, vp, ks, vs = _inputs(13, 2, 1, 1, 2, 2, 700, 100, sharp)
    got, lse = _run(q, kp, vp, pl, ks, vs, sl)
    _check(got, lse, q, kp, vp, pl, ks, vs, sl, 0, D ** -0.5)


def test_rising_scores_rescale_every_tile():
    """Keys along q with growing length: every tile raises the maximum of every row."""
    rng = np.random.default_rng(14)
    q, kp, vp, ks, vs = _inputs(14, 2, 1, 1, 2, 2, 640, 64)
    u = rng.standard_normal(D)
    u /= np.linalg.norm(u)
    q[:] = synth.round_bf16((u * 11).astype(np.float32))
    kp[0] = synth.round_bf16((u[None, None] * np.linspace(-300, 300, 640)[:, None, None]).astype(np.float32))
    got, lse = _run(q, kp, vp, [640], ks, vs, [64, 0])
    _check(got, lse, q, kp, vp, [640], ks, vs, [64, 0], 0, D ** -0.5)


def test_strided_operands():
    """q a slice of a packed projection; caches with gaps between keys and between sequences."""
    import torch
    B, H, Hkv, P, S = 4, 4, 2, 150, 90
    q, kp, vp, ks, vs = _inputs(15, B, 2, 1, H, Hkv, P, S)
    pl, sl = [150, 33], [90, 0, 17, 64]
    packed = torch.full((B, 1, H + 3, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    packed[:, :, :H] = _dev(q)

    def spread(a):
        t = torch.full((a.shape[0] + 1, a.shape[1] + 2, Hkv + 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[:-1, :-2, :Hkv] = _dev(a)
        return t[:-1, :-2, :Hkv]

    out, lse = torch.empty(B, 1, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, H, device="cuda")
    nc.nc_prefix_attention(packed[:, :, :H], spread(kp), spread(vp), _i32(pl), spread(ks), spread(vs), _i32(sl), out, out_lse=lse)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    _check(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), q, kp, vp, pl, ks, vs, sl, 0, D ** -0.5)
    with pytest.raises(nc.NcError):                       # k and v laid out differently
        nc.nc_prefix_attention(packed[:, :, :H], spread(kp), _dev(vp), _i32(pl), None, None, None, out)


def test_values_before_every_window_may_be_anything():
    """Keys that left the window may be overwritten (NaN here), in the prefix and among the row's own keys."""
    import torch
    q, kp, vp, ks, vs = _inputs(16, 2, 1, 1, 2, 2, 200, 150)
    pl, sl, w = [200], [100, 150], 120
    t = [_dev(x) for x in (kp, vp, ks, vs)]
    for c in t[:2]:
        c[0, :200 + 100 - w] = float("nan")               # before both rows' windows
    for c in t[2:]:
        c[1, :150 - w] = float("nan")
        c[0, 100:] = float("inf")
    out, lse = torch.empty(2, 1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, 2, device="cuda")
    nc.nc_prefix_attention(_dev(q), t[0], t[1], _i32(pl), t[2], t[3], _i32(sl), out, out_lse=lse, window=w)
    torch.cuda.synchronize()
    _check(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), q, kp, vp, pl, ks, vs, sl, w, D ** -0.5)


@pytest.mark.parametrize("B,H,P", [(3, 2, 300), (1, 12, 9000), (400, 8, 70)])  # the three ways pieces are joined
def test_not_a_number_stays_in_its_row(B, H, P):
    """A query that is not a number gives a row of NaN, not an empty one; a key
    that is not one gives NaN in the rows that see it.  The others keep their bits."""
    import torch
    q, kp, vp, ks, vs = _inputs(31, B, 1, 1, H, 1, P, 8)
    sl = [i % 9 for i in range(B)]
    t, lens = [_dev(x) for x in (kp, vp, ks, vs)], (_i32([P]), _i32(sl))

    def run(qd):
        out, lse = torch.empty_like(qd), torch.empty(B, 1, H, device="cuda")
        nc.nc_prefix_attention(qd, t[0], t[1], lens[0], t[2], t[3], lens[1], out, out_lse=lse)
        torch.cuda.synchronize()
        assert nc.nc_get_status()[0] == 0
        return out, lse

    o0, l0 = run(_dev(q))
    bad = _dev(q)
    bad[B // 2, 0, 1] = float("nan")
    hit = torch.zeros(B, 1, H, dtype=torch.bool, device="cuda")
    hit[B // 2, 0, 1] = True
    o1, l1 = run(bad)
    assert torch.isnan(o1[hit]).all() and torch.isnan(l1[hit]).all()
    assert torch.equal(o1[~hit], o0[~hit]) and torch.equal(l1[~hit], l0[~hit])
    if B > 1:
        row = next(b for b in range(B) if sl[b] > 0)
        t[2][row, 0] = float("nan")
        hit.zero_()
        hit[row] = True
        o2, l2 = run(_dev(q))
        assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
        assert torch.equal(o2[~hit], o0[~hit]) and torch.equal(l2[~hit], l0[~hit])


def test_lengths_out_of_range_are_clamped_and_flagged():
    import torch
    q, kp, vp, ks, vs = _inputs(17, 2, 1, 1, 2, 2, 70, 30)
    out, lse = torch.empty(2, 1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, 2, device="cuda")
    for pl, sl, cp, cs in (([71], [30, 0], [70], [30, 0]), ([70], [-1, 31], [70], [0, 30]), ([-5], [3, 4], [0], [3, 4])):
        nc.nc_prefix_attention(_dev(q), _dev(kp), _dev(vp), _i32(pl), _dev(ks), _dev(vs), _i32(sl), out, out_lse=lse)
        torch.cuda.synchronize()
        rc, bits = nc.nc_get_status()
        assert rc == nc.STATUS_CODES["NC_ERR_DATA"] and bits == 1 << rc
        _check(out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), q, kp, vp, cp, ks, vs, cs, 0, D ** -0.5)


@pytest.mark.parametrize("T,P,H,Hkv,w", [(300, 200, 4, 4, 96), (900, 260, 4, 2, 900), (900, 10, 6, 2, 333)])
def test_agrees_with_the_attention_layer(T, P, H, Hkv, w):
    """A prompt and its continuation, token by token in the cache, against nc_attention on the joined sequence: both
    round their weights and outputs to bf16, 2^-8 each, of sums of |v| that stay below 5."""
    import torch
    rng = np.random.default_rng(18)
    q, k, v = (_dev(_bf(rng, 1, T, h, D)) for h in (H, Hkv, Hkv))
    ref = torch.empty_like(q)
    nc.nc_attention(q, k, v, ref, w, rope_qknorm=0)
    out = torch.empty(1, T - P, H, D, dtype=q.dtype, device="cuda")
    nc.nc_prefix_attention(q[:, P:], k[:, :P], v[:, :P], _i32([P]), k[:, P:], v[:, P:], _i32([T - P]), out, window=w)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    assert float((out.float() - ref[:, P:].float()).abs().max()) <= 4 * 2.0 ** -8 * 5


def test_same_result_twice_on_two_streams_and_replayed_with_new_lengths():
    import torch
    B, P, S = 6, 900, 80
    q, kp, vp, ks, vs = _inputs(19, B, 2, 1, 4, 2, P, S)
    t = [_dev(x) for x in (q, kp, vp, ks, vs)]
    pl, sl = _i32([900, 123]), _i32([1, 0, 80, 40, 64, 65])
    wsb = nc.nc_prefix_attention_workspace_bytes(B, 2, 1, 4, 2, P, S)

    def call(out, lse, ws=None):
        nc.nc_prefix_attention(t[0], t[1], t[2], pl, t[3], t[4], sl, out, out_lse=lse, workspace=ws)

    new = lambda: (torch.empty_like(t[0]), torch.empty(B, 1, 4, device="cuda"))
    first = new()
    call(*first)
    torch.cuda.synchronize()
    streams, outs, spaces = [torch.cuda.Stream() for _ in range(2)], [new(), new()], [torch.empty(wsb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, ws in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                call(*o, ws)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])
    # captured once, replayed while the rows grow
    graph, got = torch.cuda.CUDAGraph(), new()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(*got, spaces[0])
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = new()
        call(*want, spaces[1])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        sl += 1
        sl.clamp_(max=S)
        pl -= 7
    assert nc.nc_get_status()[0] == 0


@pytest.mark.parametrize("B,G,window", [(1100, 1100, 0), (1100, 550, 40), (1030, 1, 0), (1030, 2, 100)])
def test_more_rows_than_the_tables_hold(B, G, window):
    """Over 512 groups or rows: the tables of starts hold several of them per entry."""
    rng = np.random.default_rng(B + G)
    q, kp, vp, ks, vs = _inputs(B + G, B, G, 1, 2, 1, 70 if G > 2 else 300, 66)
    pl, sl = rng.integers(0, kp.shape[1] + 1, G), rng.integers(0, 67, B)
    pl[::5], sl[::3] = 0, 0
    got, lse = _run(q, kp, vp, pl, ks, vs, sl, window)
    _check(got, lse, q, kp, vp, pl, ks, vs, sl, window, D ** -0.5)


def test_cache_beyond_two_to_the_31_elements():
    """Row offsets of a long cache pass 32 bits: 140 sequences of 30000 keys of 4 heads hold 2.15e9 elements."""
    import torch
    B, S, Hkv = 140, 30000, 4
    assert B * S * Hkv * D > 2 ** 31
    ks = torch.zeros(B, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vs = torch.zeros_like(ks)
    rng = np.random.default_rng(20)
    n = 70
    k, v, q = _bf(rng, 1, n, Hkv, D), _bf(rng, 1, n, Hkv, D), _bf(rng, B, 1, Hkv, D)
    ks[B - 1, S - n:], vs[B - 1, S - n:] = _dev(k)[0], _dev(v)[0]
    sl = [0] * (B - 1) + [S]
    out, lse = torch.empty(B, 1, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, Hkv, device="cuda")
    nc.nc_prefix_attention(_dev(q), None, None, None, ks, vs, _i32(sl), out, out_lse=lse, window=n)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    assert bool((out[:-1] == 0).all()) and bool((lse[:-1] == -float("inf")).all())
    e = np.zeros((1, 1, Hkv, D), np.float32)
    _check(out[-1:].float().cpu().numpy().astype(np.float64), lse[-1:].cpu().numpy().astype(np.float64), q[-1:], e, e, [0], k, v, [n], n, D ** -0.5)
