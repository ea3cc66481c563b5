"""Workspaces of the calls: where the caller's starts, and what happens to the
one that the binding makes."""
import pytest

from decoder_only_transformer_fwd_b200 import nc
from nc_cases import make_case

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


def _queued_reader_of_a_freed_block(current, nbytes):
    """On the stream `current`: a block of this size full of sevens, freed while its reader still waits behind a delay.
    It is all that the stream's pool holds, so it is what the next allocation there gets.  Returns what the reader will
    have read."""
    import torch
    seen = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(current):
        block = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(100_000_000)                   # some 50 ms
        seen.copy_(block)
        at = block.data_ptr()
        del block
        assert torch.empty(nbytes, dtype=torch.uint8, device="cuda").data_ptr() == at
    return seen


def _policy_case(seed, B, T, V):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B, T, V, device="cuda", generator=g)
    y = torch.randint(0, V, (B, T), device="cuda", generator=g).int()
    return z, y, torch.randn(B, device="cuda", generator=g), torch.empty(3, device="cuda"), torch.empty(B, T, device="cuda"), torch.empty_like(z)


def test_scratch_of_a_call_on_a_side_stream_leaves_the_current_stream_alone():
    """Without a workspace and without any order between the streams: the scratch must not be a block that the current
    stream still has to read."""
    import torch
    current, side = torch.cuda.Stream(), torch.cuda.Stream()
    t, need = _attention_case(3)
    want, got = torch.empty_like(t[0]), torch.empty_like(t[0])
    nc.nc_prefix_attention(*t, want)
    seen = _queued_reader_of_a_freed_block(current, need)
    with torch.cuda.stream(current):
        nc.nc_prefix_attention(*t, got, stream=side)
    torch.cuda.synchronize()
    assert bool((seen == 7).all()) and torch.equal(got, want)
    p = _policy_case(4, 2, 50, 900)
    nc.nc_policy_loss(*p)
    want, p2 = [x.clone() for x in p[3:]], [*p[:3], *(torch.empty_like(x) for x in p[3:])]
    seen = _queued_reader_of_a_freed_block(current, nc.nc_policy_loss_workspace_bytes())
    with torch.cuda.stream(current):
        nc.nc_policy_loss(*p2, stream=side)
    torch.cuda.synchronize()
    assert bool((seen == 7).all()) and all(torch.equal(a, b) for a, b in zip(p2[3:], want))
    assert nc.nc_get_status()[0] == 0


def test_two_calls_at_once_have_scratch_of_their_own():
    """A call on the current stream, still waiting behind a delay, and one on a side stream right after it."""
    import torch
    side = torch.cuda.Stream()
    a, _ = _attention_case(5)
    b, _ = _attention_case(6)
    pa, pb = _policy_case(7, 3, 40, 1200), _policy_case(8, 3, 40, 1200)
    want = []
    for t in (a, b):
        out = torch.empty_like(t[0])
        nc.nc_prefix_attention(*t, out)
        want.append(out)
    for p in (pa, pb):
        nc.nc_policy_loss(*p)
        want += [x.clone() for x in p[3:]]
        for x in p[3:]:
            x.fill_(float("nan"))
    outs = [torch.empty_like(t[0]) for t in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(2_000_000)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        nc.nc_prefix_attention(*a, outs[0])
        nc.nc_prefix_attention(*b, outs[1], stream=side)
        nc.nc_policy_loss(*pa)
        nc.nc_policy_loss(*pb, stream=side)
        torch.cuda.synchronize()
        got = [*outs, *pa[3:], *pb[3:]]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert nc.nc_get_status()[0] == 0


@pytest.mark.parametrize("which", ["default", "side"])
def test_scratch_is_made_on_the_stream_that_is_asked_for(which):
    """The default stream as an argument while a side stream is current, and the other way round."""
    import torch
    t, _ = _attention_case(9)
    want, got = torch.empty_like(t[0]), torch.empty_like(t[0])
    nc.nc_prefix_attention(*t, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    current, asked = (side, torch.cuda.default_stream()) if which == "default" else (torch.cuda.default_stream(), side)
    with torch.cuda.stream(current):
        nc.nc_prefix_attention(*t, got, stream=asked)
        assert torch.cuda.current_stream() == current
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0 and torch.equal(got, want)


def test_other_calls_on_a_side_stream_leave_the_current_stream_alone():
    """The same for what nc_routing_attention, nc_prefix_ce and NcModel allocate."""
    import torch
    current, side = torch.cuda.Stream(), torch.cuda.Stream()

    def check(call, nbytes):
        want = [x.clone() for x in call(None)]
        seen = _queued_reader_of_a_freed_block(current, nbytes)
        with torch.cuda.stream(current):
            got = call(side)
        torch.cuda.synchronize()
        assert bool((seen == 7).all()) and all(torch.equal(a, b) for a, b in zip(got, want))
        assert nc.nc_get_status()[0] == 0

    B, T, H, M = 2, 200, 2, 128
    g = torch.Generator(device="cuda").manual_seed(10)
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    r = [bf(B, T, H, D) for _ in range(5)]
    out = torch.empty_like(r[0])

    def routing(stream):
        nc.nc_routing_attention(*r, out, 64, 0.3, stream=stream)
        return [out]

    check(routing, int(nc.lib().nc_routing_attention_workspace_bytes(B, T, H, D)))
    x, w_u = torch.randn(M, 768, device="cuda", generator=g), 0.05 * bf(256, 768)
    y = torch.randint(0, 250, (M,), device="cuda", generator=g).int()
    loss = torch.empty(2, M, device="cuda")

    def prefix_ce(stream):
        nc.nc_prefix_ce(x, w_u, y, loss, 250, [256, 512], stream=stream)
        return [loss]

    check(prefix_ce, int(nc.lib().nc_prefix_ce_workspace_bytes(M, 768, 256)))
    cfg, _, p, tok, tgt = make_case(1, 2, 48, 48, "fp32", 78)
    model = nc.NcModel(cfg, p, tok.size)
    tt, yy, u = torch.from_numpy(tok).cuda(), torch.from_numpy(tgt).cuda(), torch.rand(2, device="cuda", generator=g)
    check(lambda s: [model.forward(tt, yy, stream=s)[0]], 4 * tok.size)
    check(lambda s: list(model.generate_next(tt, u, stream=s)), 4 * 2 * cfg.vocab)
