"""Workspaces of the calls: where the caller's starts, and what happens to the
one that the binding makes."""
import pytest

from decoder_only_transformer_fwd_b200 import nc

pytestmark = pytest.mark.gpu
D = 128


def _attention_case(seed, B=5, G=1, Tq=1, H=6, Hkv=2, P=300, S=90):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t = [bf(B, Tq, H, D), bf(G, P, Hkv, D), bf(G, P, Hkv, D), i32([P - 7] * G), bf(B, S, Hkv, D), bf(B, S, Hkv, D),
         i32([(37 * b) % (S + 1) for b in range(B)])]
    return t, nc.nc_prefix_attention_workspace_bytes(B, G, Tq, H, Hkv, P, S, 0)


@pytest.mark.parametrize("start", [0, 16, 32, 48, 240])
def test_prefix_attention_in_an_arena(start):
    """A workspace of exactly the size asked for, at every kind of 16-byte boundary, with nothing written around it."""
    import torch
    t, need = _attention_case(1)
    want, got = torch.empty_like(t[0]), torch.empty_like(t[0])
    nc.nc_prefix_attention(*t, want)
    arena = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    lo = -arena.data_ptr() % 256 + 256 + start
    nc.nc_prefix_attention(*t, got, workspace=arena[lo:lo + need])
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0 and torch.equal(got, want)
    assert bool((arena[:lo] == 0xA5).all()) and bool((arena[lo + need:] == 0xA5).all())


@pytest.mark.parametrize("start", [0, 16])
def test_policy_loss_in_an_arena(start):
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn(2, 30, 700, device="cuda", generator=g)
    y = torch.randint(0, 700, (2, 30), device="cuda", generator=g).int()
    adv, need = torch.randn(2, device="cuda", generator=g), nc.nc_policy_loss_workspace_bytes()
    outs = [(torch.empty(3, device="cuda"), torch.empty(2, 30, device="cuda"), torch.empty_like(z)) for _ in range(2)]
    nc.nc_policy_loss(z, y, adv, *outs[0])
    arena = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    lo = -arena.data_ptr() % 256 + 256 + start
    nc.nc_policy_loss(z, y, adv, *outs[1], workspace=arena[lo:lo + need])
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0 and all(torch.equal(a, b) for a, b in zip(*outs))
    assert bool((arena[:lo] == 0xA5).all()) and bool((arena[lo + need:] == 0xA5).all())
