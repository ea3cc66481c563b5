"""Cases and plain forms of the operators around sampling many completions of a prompt and learning from them:

- "qknorm" / "qknorm_bwd": QK-norm with RoPE at given positions, written into a cache, and its gradient;
- "prefix": attention of a batch whose rows share a long prefix, over the shared and the rows' own keys;
- "policy": the clipped policy loss with a KL term, from logits to the loss and the logits' gradient.

With `own` false every operator is computed by elementary torch operations in fp32 (fp64 for angles and long sums);
with `own` true by the library's calls.  Head dimension 128, RoPE base 100000, alpha 1.15 and eps 1e-6 throughout, as in
the model's configuration.
"""
import math

import numpy as np
import torch

own = False

D = 128
ALPHA, BASE, EPS = 1.15, 100000.0, 1e-6
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one generation step of 16 rows: each new token's k and v go to their row's next cache slot
        {"name": "qknorm step 16", "op": "qknorm", "N": 16, "H": 12, "Hkv": 12, "dtype": "bf16", "cache": 256},
        # prefill of four rows of 2048 at the depth-24 widths, into a cache
        {"name": "qknorm prefill 8192", "op": "qknorm", "N": 8192, "H": 12, "Hkv": 12, "dtype": "bf16", "cache": 2048},
        # the gradient of the same pass
        {"name": "qknorm bwd 8192", "op": "qknorm_bwd", "N": 8192, "H": 12, "Hkv": 12, "dtype": "bf16"},
        # fp32 mode, an odd number of tokens, grouped heads
        {"name": "qknorm bwd fp32 777", "op": "qknorm_bwd", "N": 777, "H": 12, "Hkv": 4, "dtype": "fp32"},
        # a few samples of a short prompt, first tokens: latency
        {"name": "prefix 4x512", "op": "prefix", "G": 1, "n": 4, "Tq": 1, "H": 12, "Hkv": 12, "P": 512, "S": 64, "window": 0},
        # 16 samples of a 2048-token prompt, a sliding-window layer
        {"name": "prefix 16x2048 w1024", "op": "prefix", "G": 1, "n": 16, "Tq": 1, "H": 12, "Hkv": 12, "P": 2048, "S": 512, "window": 1024},
        # three prompts of ragged length, grouped heads, chunks of five tokens
        {"name": "prefix 3x20 tq5 gqa", "op": "prefix", "G": 3, "n": 20, "Tq": 5, "H": 12, "Hkv": 4, "P": 5000, "S": 333, "window": 0},
        # 64 samples of a long document
        {"name": "prefix 64x32768", "op": "prefix", "G": 1, "n": 64, "Tq": 1, "H": 12, "Hkv": 12, "P": 32768, "S": 1024, "window": 0},
        # one row of completions: 64 tokens at the model's vocabulary
        {"name": "policy 64", "op": "policy", "B": 1, "T": 64, "V": 32768, "dtype": "fp32", "per_token": False, "norm": 0, "kl": 0.05, "on_policy": False},
        # 8 completions, bf16 logits of an odd vocabulary, every sequence weighing the same
        {"name": "policy 8x250 bf16", "op": "policy", "B": 8, "T": 250, "V": 40009, "dtype": "bf16", "per_token": True, "norm": 1, "kl": 0.0, "on_policy": False},
        # a full batch: 16 completions of 512 tokens
        {"name": "policy 16x512", "op": "policy", "B": 16, "T": 512, "V": 32768, "dtype": "fp32", "per_token": False, "norm": 0, "kl": 0.05, "on_policy": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qknorm", "qknorm_bwd", "prefix", "prefix", "policy"])
    H = rng.choice([4, 6, 8, 12, 16])
    Hkv = rng.choice([h for h in (1, 2, 3, 4, 6, 8, 12, 16) if H % h == 0])
    if op.startswith("qknorm"):
        c = {"op": op, "N": _log(rng, 1, 16384), "H": H, "Hkv": Hkv, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        if op == "qknorm":
            c["cache"] = rng.choice([256, 500, 2048])
        return c
    if op == "prefix":
        while True:
            c = {"op": op, "G": rng.choice([1, 1, 2, 3]), "n": _log(rng, 1, 96), "Tq": rng.choice([1, 1, 1, 2, 7]), "H": H, "Hkv": Hkv,
                 "P": _log(rng, 16, 32768), "S": _log(rng, 1, 1500), "window": rng.choice([0, 0, 128, 1000, 1024])}
            w = work(c)
            if w["bytes"] <= 4.5e8 and w["flops"] <= 3e11 and c["G"] * c["n"] * c["Tq"] * H * (c["P"] + c["S"]) <= 26e6:
                return c
    V = _log(rng, 500, 60000)
    M = _log(rng, 1, max(2, min(16384, 8192 * 32768 // V)))
    B = max(1, min(M, rng.choice([1, 2, 5, 8, 16, 32])))
    return {"op": op, "B": B, "T": max(1, M // B), "V": V, "dtype": rng.choice(["fp32", "fp32", "bf16"]), "per_token": rng.random() < 0.3,
            "norm": rng.choice([0, 1]), "kl": rng.choice([0.0, 0.05]), "on_policy": rng.random() < 0.25}


def _lengths(case):
    """Prefix length of every group and suffix length of every row, ragged, a row in seven without keys of its own."""
    P, S, B = case["P"], case["S"], case["G"] * case["n"]
    pl = [P - (g * 397) % max(1, P // 3) for g in range(case["G"])]
    sl = [0 if b % 7 == 3 else 1 + ((b * 2654435761 + 97531) % (1 << 32)) * S // (1 << 32) for b in range(B)]
    return pl, sl


def work(case):
    if case["op"].startswith("qknorm"):
        N, H, Hkv, e = case["N"], case["H"], case["Hkv"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "qknorm":
            return {"bytes": N * (H + 2 * Hkv) * D * e * 2 + N * 8, "flops": N * (H + Hkv) * D * 8}
        return {"bytes": N * (H + Hkv) * D * e * 3 + N * 4, "flops": N * (H + Hkv) * D * 16}
    if case["op"] == "prefix":
        H, Hkv, Tq, n = case["H"], case["Hkv"], case["Tq"], case["n"]
        pl, sl = _lengths(case)
        w = case["window"] or 1 << 60
        keys = pairs = 0
        for g, P in enumerate(pl):
            low = P  # the first prefix position that a row of the group sees
            for b in range(g * n, (g + 1) * n):
                first = P + sl[b] - Tq  # position of the row's first query
                keys += sl[b] - max(0, min(sl[b], first - w + 1 - P))
                for i in range(Tq):
                    lo, hi = max(0, first + i - w + 1), first + i
                    pairs += max(0, hi - lo + 1)
                    low = min(low, lo)
            keys += P - max(0, low)
        rows = len(sl) * Tq * H
        return {"bytes": keys * Hkv * D * 4 + rows * D * 4 + rows * 4, "flops": 4 * D * H * pairs}
    M, V, e = case["B"] * case["T"], case["V"], 2 if case["dtype"] == "bf16" else 4
    return {"bytes": M * V * e * 2 + M * 24, "flops": M * V * 6}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def normal(*shape, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype).normal_(generator=g)

    if case["op"].startswith("qknorm"):
        N, H, Hkv, dt = case["N"], case["H"], case["Hkv"], _dt(case)
        qkv = normal(N, H + 2 * Hkv, D, dtype=dt)  # one projection's output: q, k and v are views of its rows
        s = {"case": case, "q": qkv[:, :H], "k": qkv[:, H:H + Hkv], "v": qkv[:, H + Hkv:]}
        if case["op"] == "qknorm_bwd":
            s["positions"] = (torch.arange(N, device=dev) % 2048).int()
            s["dq_hat"], s["dk_hat"] = normal(N, H, D, dtype=dt), normal(N, Hkv, D, dtype=dt)
            return s
        R = case["cache"]
        if N < R:  # a generation step: token n goes to some slot of row n's cache, far into its sequence
            slots = torch.arange(N, device=dev) * R + torch.randint(0, R, (N,), device=dev, generator=g)
            s["positions"] = torch.randint(0, 1 << 17, (N,), device=dev, generator=g).int()
            s["slots"], rows = slots.int(), N * R
        else:  # rows of R tokens; one token in 61 is padding and is not kept
            n = torch.arange(N, device=dev)
            s["positions"], s["slots"], rows = (n % R).int(), torch.where(n % 61 == 60, -1, n).int(), N
        rows = min(rows, 1 << 18)
        s["slots"] = torch.where(s["slots"] < rows, s["slots"], -1).int()
        s["k_cache"] = torch.zeros(rows, Hkv, D, device=dev, dtype=dt)
        s["v_cache"] = torch.zeros(rows, Hkv, D, device=dev, dtype=dt)
        return s
    if case["op"] == "prefix":
        G, n, Tq, H, Hkv, P, S = (case[x] for x in ("G", "n", "Tq", "H", "Hkv", "P", "S"))
        bf = torch.bfloat16

        def unit(*shape):  # what QK-norm gives: vectors of norm alpha sqrt(D)
            x = normal(*shape, dtype=bf)
            return x.mul_(ALPHA * math.sqrt(D) / x.float().square().sum(-1, keepdim=True).sqrt())

        pl, sl = _lengths(case)
        return {"case": case, "q": unit(G * n, Tq, H, D), "kp": unit(G, P, Hkv, D), "vp": normal(G, P, Hkv, D, dtype=bf),
                "ks": unit(G * n, S, Hkv, D), "vs": normal(G * n, S, Hkv, D, dtype=bf),
                "pl": torch.tensor(pl, dtype=torch.int32, device=dev), "sl": torch.tensor(sl, dtype=torch.int32, device=dev)}
    B, T, V = case["B"], case["T"], case["V"]
    z = torch.empty(B, T, V, device=dev, dtype=_dt(case)).normal_(0.0, 2.0, generator=g)
    y = torch.randint(0, V, (B, T), device=dev, generator=g)
    # completions end at different places; behind the end there is padding
    last = torch.randint(max(1, T // 2), T + 1, (B, 1), device=dev, generator=g)
    valid = torch.arange(T, device=dev)[None] < last
    # a sampled token is one that the policy finds likely; the old and reference policies are near it
    z.scatter_add_(2, y[..., None], torch.empty(B, T, 1, device=dev, dtype=z.dtype).uniform_(4.0, 10.0, generator=g))
    lp = z.gather(2, y[..., None])[..., 0].float() - z.logsumexp(-1).float()
    s = {"case": case, "z": z, "y": torch.where(valid, y, -1).int(), "old": None if case["on_policy"] else lp + 0.2 * normal(B, T),
         "ref": lp + 0.2 * normal(B, T) if case["kl"] else None, "adv": normal(B, T) if case["per_token"] else normal(B)}
    return s


# ---------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------

def _cos_sin(positions):
    f = BASE ** (-torch.arange(D // 2, device=positions.device, dtype=torch.float64) / (D // 2))
    a = positions.double()[:, None] * f
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin):
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_qknorm(s):
    cos, sin = _cos_sin(s["positions"])

    def norm(x):
        r = _rotate(x.float(), cos, sin)
        return (ALPHA * r / (r.square().mean(-1, keepdim=True) + EPS).sqrt()).to(x.dtype)

    q_hat, k_hat = norm(s["q"]), norm(s["k"])
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    s["k_cache"][at] = k_hat[keep]
    s["v_cache"][at] = s["v"][keep]
    return [q_hat, s["k_cache"], s["v_cache"]]


def _plain_qknorm_bwd(s):
    cos, sin = _cos_sin(s["positions"])

    def grad(x, dy):
        x32, back = x.float(), _rotate(dy.float(), cos, -sin)
        inv = 1.0 / (x32.square().mean(-1, keepdim=True) + EPS).sqrt()
        return (ALPHA * inv * (back - x32 * inv * inv * (x32 * back).mean(-1, keepdim=True))).to(x.dtype)

    return [grad(s["q"], s["dq_hat"]), grad(s["k"], s["dk_hat"])]


def _plain_prefix(s):
    c = s["case"]
    G, n, Tq, H, Hkv, P, S = (c[x] for x in ("G", "n", "Tq", "H", "Hkv", "P", "S"))
    B, R, dev = G * n, H // Hkv, s["q"].device
    q = s["q"].float().view(B, Tq, Hkv, R, D) / math.sqrt(D)
    qg = q.view(G, n * Tq, Hkv, R, D).permute(0, 2, 1, 3, 4).reshape(G, Hkv, n * Tq * R, D)
    qb = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tq * R, D)
    kp, vp, ks, vs = (s[x].float().transpose(1, 2) for x in ("kp", "vp", "ks", "vs"))
    sp = (qg @ kp.transpose(-1, -2)).view(G, Hkv, n, Tq, R, P).transpose(1, 2).reshape(B, Hkv, Tq, R, P)
    ss = (qb @ ks.transpose(-1, -2)).view(B, Hkv, Tq, R, S)
    pl = s["pl"].long().repeat_interleave(n)
    sl = s["sl"].long()
    pos = (pl + sl - Tq)[:, None] + torch.arange(Tq, device=dev)
    jp, js = torch.arange(P, device=dev), torch.arange(S, device=dev)
    w = c["window"] or 1 << 60
    ap, as_ = jp.expand(B, 1, P), (pl[:, None] + js)[:, None]
    seen_p = (jp < pl[:, None])[:, None] & (ap <= pos[..., None]) & (pos[..., None] - ap < w)
    seen_s = (js < sl[:, None])[:, None] & (as_ <= pos[..., None]) & (pos[..., None] - as_ < w)
    seen = torch.cat([seen_p, seen_s], -1)[:, None, :, None]
    x = torch.cat([sp, ss], -1).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m.clamp_min(-1e30)).exp()
    l = e.sum(-1, keepdim=True)
    ep = e[..., :P].reshape(G, n, Hkv, Tq * R, P).transpose(1, 2).reshape(G, Hkv, n * Tq * R, P)
    op = (ep @ vp).view(G, Hkv, n, Tq, R, D).transpose(1, 2).reshape(B, Hkv, Tq, R, D)
    os_ = (e[..., P:].reshape(B, Hkv, Tq * R, S) @ vs).view(B, Hkv, Tq, R, D)
    o = torch.where(l > 0, (op + os_) / l.clamp_min(1e-30), 0.0)
    lse = (m + l.log())[..., 0]
    return [o.transpose(1, 2).reshape(B, Tq, H, D).to(s["q"].dtype), lse.transpose(1, 2).reshape(B, Tq, H)]


def _weights(y, norm):
    valid = y >= 0
    if norm == 0:
        return valid.double() / valid.sum().clamp_min(1)
    per = valid.sum(1, keepdim=True)
    return valid.double() / per.clamp_min(1) / (per > 0).sum().clamp_min(1)


def _plain_policy(s):
    c = s["case"]
    z, y = s["z"].float(), s["y"]
    at = y.clamp_min(0).long()[..., None]
    m = z.amax(-1, keepdim=True)
    e = (z - m).exp()
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    lp = (z.gather(2, at).double() - m - total.log())[..., 0]
    w = _weights(y, c["norm"])
    A = s["adv"].double() if c["per_token"] else s["adv"].double()[:, None]
    r = (lp - (lp if s["old"] is None else s["old"].double())).exp()
    free, cut = r * A, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A
    loss = -torch.minimum(free, cut)
    slope = torch.where(free <= cut, -r * A, 0.0)
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        d = s["ref"].double() - lp
        kl = d.exp() - d - 1
        loss = loss + c["kl"] * kl
        slope = slope + c["kl"] * (1 - d.exp())
    stats = torch.stack([(w * loss).sum(), (w * kl).sum(), (w * (free > cut)).sum()]).float()
    gz = (w * slope).float()[..., None]
    dz = -gz * (e * total.reciprocal().float())
    dz.scatter_add_(2, at, gz)
    return [stats, torch.where(y >= 0, lp, 0.0).float(), dz.to(s["z"].dtype)]


# ---------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------

def _own(s):
    from decoder_only_transformer_fwd_b200 import nc
    c = s["case"]
    if c["op"] == "qknorm":
        q_hat = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
        nc.nc_qk_norm_rope(s["q"], s["k"], s["positions"], q_hat, s["k_cache"], v=s["v"], v_out=s["v_cache"], slots=s["slots"],
                           alpha=ALPHA, rope_base=BASE, eps=EPS, reverse=True)
        return [q_hat, s["k_cache"], s["v_cache"]]
    if c["op"] == "qknorm_bwd":
        dq, dk = torch.empty_like(s["dq_hat"]), torch.empty_like(s["dk_hat"])
        nc.nc_qk_norm_rope_backward(s["q"], s["k"], s["positions"], s["dq_hat"], s["dk_hat"], dq, dk, alpha=ALPHA, rope_base=BASE, eps=EPS, reverse=True)
        return [dq, dk]
    if c["op"] == "prefix":
        out = torch.empty_like(s["q"])
        lse = torch.empty(s["q"].shape[:3], device=out.device)
        nc.nc_prefix_attention(s["q"], s["kp"], s["vp"], s["pl"], s["ks"], s["vs"], s["sl"], out, out_lse=lse, window=c["window"])
        return [out, lse]
    stats = torch.empty(3, device=s["z"].device)
    logp = torch.empty(s["y"].shape, device=s["z"].device)
    dz = torch.empty_like(s["z"])
    nc.nc_policy_loss(s["z"], s["y"], s["adv"], stats, logp, dz, old_logp=s["old"], ref_logp=s["ref"], clip_low=CLIP_LOW,
                      clip_high=CLIP_HIGH, kl_beta=c["kl"], norm=c["norm"])
    return [stats, logp, dz]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"qknorm": _plain_qknorm, "qknorm_bwd": _plain_qknorm_bwd, "prefix": _plain_prefix, "policy": _plain_policy}[op](state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _turn(x, positions, sign):
    """x's pairs (i, i + D/2) as complex numbers, turned by the position's angles."""
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    angle = sign * positions.double()[:, None, None] * torch.exp(-2.0 * i / D * math.log(BASE))
    t = torch.complex(x[..., :D // 2], x[..., D // 2:]) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([t.real, t.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qknorm":
        outs = []
        for x in (s["q"].double(), s["k"].double()):
            outs.append(ALPHA * _turn(x, s["positions"], 1.0) * (x.pow(2).sum(-1, keepdim=True) / D + EPS).rsqrt())
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        slots = s["slots"].long()
        rows = torch.nonzero(slots >= 0)[:, 0]
        kc.index_copy_(0, slots[rows], outs[1][rows])
        vc.index_copy_(0, slots[rows], s["v"].double()[rows])
        return [outs[0], kc, vc]
    if case["op"] == "qknorm_bwd":
        outs = []
        for x, dy in ((s["q"], s["dq_hat"]), (s["k"], s["dk_hat"])):
            x = x.double().requires_grad_()
            y = ALPHA * _turn(x, s["positions"], 1.0) * (x.pow(2).sum(-1, keepdim=True) / D + EPS).rsqrt()
            outs.append(torch.autograd.grad(y, x, dy.double())[0])
        return outs
    if case["op"] == "prefix":
        n, Tq, H, Hkv = (case[x] for x in ("n", "Tq", "H", "Hkv"))
        pl, sl = _lengths(case)
        w = case["window"] or 1 << 60
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        for b in range(case["G"] * n):
            P, S = pl[b // n], sl[b]
            last = P + S - 1
            lo = max(0, last - Tq + 1 - w + 1)  # no query of the row sees a key before this one
            if last < lo:
                continue
            k = torch.cat([s["kp"][b // n, min(lo, P):P], s["ks"][b, max(0, lo - P):S]]).double().repeat_interleave(H // Hkv, 1)
            v = torch.cat([s["vp"][b // n, min(lo, P):P], s["vs"][b, max(0, lo - P):S]]).double().repeat_interleave(H // Hkv, 1)
            for i in range(Tq):
                at = P + S - Tq + i
                first = max(0, at - w + 1)
                if at < first:
                    continue
                x = torch.einsum("hd,jhd->hj", s["q"][b, i].double(), k[first - lo:at + 1 - lo]) / math.sqrt(D)
                lse[b, i] = torch.logsumexp(x, 1)
                o[b, i] = torch.einsum("hj,jhd->hd", torch.exp(x - lse[b, i][:, None]), v[first - lo:at + 1 - lo])
        return [o, lse]
    B, T = case["B"], case["T"]
    count = [int(v) for v in (s["y"] >= 0).sum(1).tolist()]
    total = np.zeros(3)
    lps, dz = [], torch.empty(s["z"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        z, y = s["z"][b].double(), s["y"][b].long()
        logp = torch.log_softmax(z, -1)
        hot = torch.zeros_like(z).scatter_(1, y.clamp_min(0)[:, None], 1.0) * (y >= 0)[:, None]
        lp = (logp.masked_fill(hot == 0, 0.0)).sum(-1)
        if case["norm"] == 0:
            wt = 1.0 / max(1, sum(count))
        else:
            wt = 1.0 / max(1, count[b]) / max(1, sum(v > 0 for v in count))
        wt = wt * (y >= 0).double()
        A = s["adv"][b].double()
        old = lp if s["old"] is None else s["old"][b].double()
        r = torch.exp(lp - old)
        # the clipped branch is the smaller one only above the upper border (A > 0) or below the lower one (A < 0)
        out = ((A > 0) & (r > 1 + CLIP_HIGH)) | ((A < 0) & (r < 1 - CLIP_LOW))
        bound = torch.where(r > 1, torch.full_like(r, 1 + CLIP_HIGH), torch.full_like(r, 1 - CLIP_LOW))
        loss = -torch.where(out, bound, r) * A
        slope = torch.where(out, torch.zeros_like(r), -r * A)
        kl = torch.zeros_like(r)
        if s["ref"] is not None:
            ratio = torch.exp(s["ref"][b].double() - lp)
            kl = ratio - 1 - torch.log(ratio)
            loss, slope = loss + case["kl"] * kl, slope + case["kl"] * (1 - ratio)
        total += np.array([float((wt * x).sum()) for x in (loss, kl, out.double())])
        lps.append(lp)
        dz[b] = (wt * slope)[:, None] * (hot - torch.exp(logp))
    return [torch.tensor(total), torch.stack(lps), dz]
