"""nc_prefix_attention with lengths far below the caches' capacity: a single
long row among empty ones is cut over all CTAs of its heads, however many pieces
that gives.  Tolerance as in test_gpu_prefix_attention.py."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import nc
from test_gpu_prefix_attention import D, _bf, _check, _dev, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,S,n,at", [
    (500, 12800, 12800, 499),       # one warp joins a row: 66 pieces of three tiles
    (500, 12800, 12737, 250),
    (200, 32768, 32768, 3),         # four warps: 171 pieces
    (100, 32768, 30001, 99),        # the same, with few rows and a small estimate
])
def test_one_long_row_among_empty_ones(B, S, n, at):
    import torch
    ks = torch.zeros(B, S, 1, D, dtype=torch.bfloat16, device="cuda")
    vs = torch.full_like(ks, float("nan"))                   # no other row's value is read as one
    rng = np.random.default_rng(B + n)
    k, v, q = _bf(rng, 1, n, 1, D), _bf(rng, 1, n, 1, D), _bf(rng, B, 1, 1, D)
    ks[at, :n], vs[at, :n] = _dev(k)[0], _dev(v)[0]
    sl = [0] * B
    sl[at] = n
    qd = _dev(q)
    out, lse = torch.full_like(qd, float("nan")), torch.full((B, 1, 1), float("nan"), device="cuda")
    nc.nc_prefix_attention(qd, None, None, None, ks, vs, _i32(sl), out, out_lse=lse)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    rest = torch.arange(B, device="cuda") != at
    assert bool((out[rest] == 0).all()) and bool((lse[rest] == -float("inf")).all())
    e = np.zeros((1, 1, 1, D), np.float32)
    host = lambda t: t[at:at + 1].float().cpu().numpy().astype(np.float64)
    _check(host(out), host(lse), q[at:at + 1], e, e, [0], k, v, [n], 0, D ** -0.5)
