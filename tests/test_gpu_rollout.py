"""The sampling operators together, as a reinforcement-learning step uses them:
several samples of each prompt grow token by token (nc_qk_norm_rope into the
caches, nc_prefix_attention over the shared prompt and the samples' own keys,
one captured graph replayed per token), then the model's logits of the finished
rows go through nc_policy_loss.

The attention of every new token is held against nc_attention on the whole
sequences (RoPE and QK-norm inside).  Both round qhat, khat, the weights and the
output to bf16: a rounding of qhat or khat by 2^-8 of its elements moves a score
scale qhat.khat (at most alpha^2 sqrt(D) = 15) by at most 2 * 2^-8 * 15 if all
elements err alike, 2 * 2^-8 * 15 / sqrt(D) = 0.011 as independent ones; with
weights and outputs rounded on both sides (2^-8 each) and |v| < 5 the outputs
differ by less than 5 (2 * 0.011 + 4 * 2^-8) = 0.19."""
import numpy as np
import pytest

from decoder_only_transformer_fwd_b200 import nc
from nc_cases import make_case
from oracle import policy_loss as PL

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("G,n,H,Hkv,window", [(1, 5, 4, 4, 0), (2, 3, 6, 2, 100)])
def test_samples_of_shared_prompts_grow_token_by_token(G, n, H, Hkv, window):
    import torch
    B, P_max, S_max, steps = G * n, 150, 40, 33
    plen = [150, 77][:G]
    g = torch.Generator(device="cuda").manual_seed(G * 100 + H)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    prompt = [normal(p, H + 2 * Hkv, D) for p in plen]                     # packed projections
    new = normal(steps, B, H + 2 * Hkv, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # prefill: each prompt's keys and values, once for all of its samples
    kp, vp = (torch.full((G, P_max, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, x in enumerate(prompt):
        q_hat = torch.empty(plen[i], H, D, dtype=torch.bfloat16, device="cuda")
        nc.nc_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], torch.arange(plen[i], dtype=torch.int32, device="cuda"), q_hat, kp[i],
                           v=x[:, H + Hkv:], v_out=vp[i])
    ks, vs = (torch.full((B, S_max, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pl, sl = i32(plen), torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = pl.repeat_interleave(n).clone()
    slots = torch.arange(B, dtype=torch.int32, device="cuda") * S_max
    x = torch.empty_like(new[0])
    q_hat, out = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(nc.nc_prefix_attention_workspace_bytes(B, G, 1, H, Hkv, P_max, S_max, window), dtype=torch.uint8, device="cuda")

    def step():
        nc.nc_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], pos, q_hat, ks.view(B * S_max, Hkv, D), v=x[:, H + Hkv:],
                           v_out=vs.view(B * S_max, Hkv, D), slots=slots)
        sl.add_(1)
        nc.nc_prefix_attention(q_hat.view(B, 1, H, D), kp, vp, pl, ks, vs, sl, out, window=window, workspace=ws)
        pos.add_(1)
        slots.add_(1)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    got = []
    for t in range(steps):
        x.copy_(new[t])
        graph.replay()
        got.append(out.clone())
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    got = torch.cat(got, 1).float()                                        # [B, steps, H, D]
    for b in range(B):
        full = torch.cat([prompt[b // n], new[:, b]])[None]
        T = full.shape[1]
        q, k, v = (full[:, :, lo:hi].contiguous() for lo, hi in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
        ref = torch.empty_like(q)
        aws = torch.empty(nc.nc_attention_workspace_bytes(1, T, H, Hkv, D), dtype=torch.uint8, device="cuda")
        nc.nc_attention(q, k, v, ref, window if window else T, workspace=aws)
        torch.cuda.synchronize()
        diff = (got[b] - ref[0, -steps:].float()).abs()
        assert float(diff.max()) <= 0.19 and float(diff.square().mean().sqrt()) <= 0.19 / 8


def test_logits_of_the_model_through_the_policy_loss():
    """The log-probabilities are the negated losses of nc_forward on the same tokens (fp32 mode: both within 1e-4 of
    the same value, its stated tolerance), and with A = 1 on fresh samples the gradient is that of the mean CE."""
    import torch
    cfg, _, p, tok, tgt = make_case(1, 2, 48, 48, "fp32", 77)
    B, T = tok.shape
    tgt = tgt.copy()
    tgt[1, 30:] = -1
    model = nc.NcModel(cfg, p, B * T)
    tt, yy = torch.from_numpy(tok).cuda(), torch.from_numpy(tgt).cuda()
    loss, logits = model.forward(tt, yy, want_logits=True)
    z = logits.view(B, T, -1)
    stats, logp, dz = torch.empty(3, device="cuda"), torch.empty(B, T, device="cuda"), torch.empty_like(z)
    nc.nc_policy_loss(z, yy, torch.ones(B, device="cuda"), stats, logp, dz)
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0
    assert float((logp.view(-1) + loss).abs().max()) <= 2e-4
    want = PL.policy_loss(z.cpu().numpy(), tgt, np.ones(B, np.float32))
    assert abs(float(stats[0]) + 1.0) <= 2.0 ** -16                        # -mean(r A) = -1
    size = want["size"][..., None] * (want["p"] + want["hot"])
    assert np.all(np.abs(dz.double().cpu().numpy() - want["dz"]) <= 2.0 ** -24 * np.abs(want["dz"]) + 2.0 ** -15 * size + 2.0 ** -126)
    # a second step on the same samples: the old log-probabilities are these, the reference a little off
    ref = logp - 0.25
    nc.nc_policy_loss(z, yy, torch.tensor([1.0, -1.0], device="cuda"), stats, logp.clone(), z, old_logp=logp, ref_logp=ref, kl_beta=0.1)
    torch.cuda.synchronize()
    valid = tgt >= 0
    share = valid[0].sum() / valid.sum()
    kl = np.exp(-0.25) + 0.25 - 1
    assert abs(float(stats[1]) - kl) <= 1e-5 and abs(float(stats[0]) - (-(share - (1 - share)) + 0.1 * kl)) <= 1e-5


def test_binding_refuses_layouts_it_cannot_pass_on():
    import torch
    bf = torch.bfloat16
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device="cuda")
    pos = z(8, dtype=torch.int32)
    wide = z(4, 4, 256)[:, :, ::2]                                     # elements apart
    heads = z(4, 8, D)[:, ::2]                                         # heads apart
    q, k = z(4, 4, D), z(4, 2, D)
    cache, lens, sl = z(2, 6, 2, D), z(2, dtype=torch.int32), z(4, dtype=torch.int32)
    q4 = z(4, 3, 4, D)
    logits, y, adv = z(2, 5, 16), z(2, 5, dtype=torch.int32), z(2, dtype=torch.float32)
    stats, logp = z(3, dtype=torch.float32), z(2, 5, dtype=torch.float32)
    bad = [
        lambda: nc.nc_qk_norm_rope(wide, k, pos[:4], q, k),
        lambda: nc.nc_qk_norm_rope(heads, k, pos[:4], q, k),
        lambda: nc.nc_qk_norm_rope(q, k, pos[::2], q, k),
        lambda: nc.nc_qk_norm_rope(z(4, 4, 64), z(4, 2, 64), pos[:4], z(4, 4, 64), z(4, 2, 64)),
        lambda: nc.nc_qk_norm_rope(q, k, pos[:4], q, z(3, 2, D)),         # fewer rows than tokens, no slots
        lambda: nc.nc_qk_norm_rope(q, k, pos[:4], q, k, alpha=0.0),
        lambda: nc.nc_qk_norm_rope_backward(q, k, pos[:4], q, k, heads, k),
        lambda: nc.nc_prefix_attention(q4.transpose(0, 1), cache, cache, lens, None, None, None, q4.transpose(0, 1)),
        lambda: nc.nc_prefix_attention(z(4, 6, 4, D)[:, ::2][:, :, :, :], cache, cache, lens, None, None, None, z(4, 3, 4, D)[:, :2]),
        lambda: nc.nc_prefix_attention(q4, cache[:, :, :, ::1].transpose(1, 2), cache.transpose(1, 2), lens, None, None, None, q4),
        lambda: nc.nc_prefix_attention(q4, cache, cache, lens, z(4, 6, 2, D), z(4, 8, 2, D)[:, :6], sl, q4.clone()),
        lambda: nc.nc_prefix_attention(q4, cache, cache, lens, None, None, None, q4.clone(), workspace=z(16, dtype=torch.uint8)),
        lambda: nc.nc_prefix_attention(q4, cache, cache, lens, None, None, None, q4.clone(), softmax_scale=-1.0),
        lambda: nc.nc_policy_loss(z(2, 6, 16)[:, :5], y, adv, stats, logp),  # rows not evenly spaced
        lambda: nc.nc_policy_loss(logits.transpose(1, 2), z(2, 16, dtype=torch.int32), adv, stats, z(2, 16, dtype=torch.float32)),
        lambda: nc.nc_policy_loss(logits, y, adv, stats, logp, norm=2),
        lambda: nc.nc_policy_loss(logits, y, adv, stats, logp, workspace=z(16, dtype=torch.uint8)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(nc.NcError):
            f()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert nc.nc_get_status()[0] == 0


def test_calls_on_a_stream_of_their_own_keep_their_scratch():
    """The stream argument without a workspace: the scratch made for the call is not handed out again while that
    stream still uses it."""
    import torch
    B, S, H = 6, 700, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(B, 1, H, D, device="cuda", generator=g).bfloat16()
    ks, vs = (torch.randn(B, S, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    sl = torch.tensor([700, 3, 64, 65, 500, 0], dtype=torch.int32, device="cuda")
    want, side = torch.empty_like(q), torch.cuda.Stream()
    nc.nc_prefix_attention(q, None, None, None, ks, vs, sl, want)
    torch.cuda.synchronize()
    nbytes = nc.nc_prefix_attention_workspace_bytes(B, 1, 1, H, H, 0, S, 0)
    for _ in range(20):
        out = torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)                                  # the stream is behind when the call returns
        nc.nc_prefix_attention(q, None, None, None, ks, vs, sl, out, stream=side)
        junk = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk
