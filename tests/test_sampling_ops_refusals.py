"""What nc_qk_norm_rope, nc_qk_norm_rope_backward, nc_prefix_attention and
nc_policy_loss refuse, without a GPU: the C checks (made before any launch)
and those of the Python binding."""
import ctypes as C

import pytest
import torch

from decoder_only_transformer_fwd_b200 import nc

_BUF = (C.c_byte * 8192)()
A16 = (C.addressof(_BUF) + 15) & ~15
P = C.c_void_p(A16)
OFF4, OFF2 = C.c_void_p(A16 + 4), C.c_void_p(A16 + 2)
S = nc.STATUS_CODES
NAN, INF = float("nan"), float("inf")


def _call(fn, names, defaults, **kw):
    a = dict(defaults, **kw)
    return getattr(nc.lib(), fn)(*[a[n] for n in names])


QK_NAMES = "q ldq k ldk v ldv pos slots N H Hkv D qo ldqo ko ldko vo ldvo rows alpha base reverse eps dtype stream".split()
QK_BASE = dict(q=P, ldq=512, k=P, ldk=256, v=P, ldv=256, pos=P, slots=None, N=4, H=4, Hkv=2, D=128, qo=P, ldqo=512, ko=P,
               ldko=256, vo=P, ldvo=256, rows=4, alpha=1.15, base=1e5, reverse=0, eps=1e-6, dtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "ARG"), (dict(k=None), "ARG"), (dict(pos=None), "ARG"), (dict(qo=None), "ARG"), (dict(ko=None), "ARG"),
    (dict(v=None), "ARG"), (dict(vo=None), "ARG"), (dict(alpha=0.0), "ARG"), (dict(alpha=NAN), "ARG"), (dict(alpha=INF), "ARG"),
    (dict(base=0.5), "ARG"), (dict(base=NAN), "ARG"), (dict(reverse=2), "ARG"), (dict(eps=-1.0), "ARG"), (dict(eps=NAN), "ARG"), (dict(dtype=2), "ARG"),
    (dict(N=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(Hkv=3), "SHAPE"), (dict(D=64), "SHAPE"),
    (dict(rows=3), "SHAPE"), (dict(rows=-1, slots=P), "SHAPE"), (dict(ldq=504), "SHAPE"), (dict(ldk=248), "SHAPE"),
    (dict(ldv=248), "SHAPE"), (dict(ldqo=504), "SHAPE"), (dict(ldko=248), "SHAPE"), (dict(ldvo=0), "SHAPE"),
    (dict(q=OFF4), "ALIGN"), (dict(v=OFF4), "ALIGN"), (dict(ko=OFF4), "ALIGN"), (dict(pos=OFF2), "ALIGN"),
    (dict(slots=OFF2), "ALIGN"), (dict(ldq=516), "ALIGN"), (dict(ldvo=260), "ALIGN"), (dict(ldk=258, dtype=1), "ALIGN")])
def test_qk_norm_rope_refuses(kw, status):
    assert _call("nc_qk_norm_rope", QK_NAMES, QK_BASE, **kw) == S["NC_ERR_" + status]


def test_qk_norm_rope_of_no_tokens_is_nothing():
    assert _call("nc_qk_norm_rope", QK_NAMES, QK_BASE, N=0) == 0
    assert nc.nc_last_launch_count() == 0


QB_NAMES = "q ldq k ldk pos gq ldgq gk ldgk N H Hkv D dq lddq dk lddk alpha base reverse eps dtype stream".split()
QB_BASE = dict(q=P, ldq=512, k=P, ldk=256, pos=P, gq=P, ldgq=512, gk=P, ldgk=256, N=4, H=4, Hkv=2, D=128, dq=P, lddq=512, dk=P,
               lddk=256, alpha=1.15, base=1e5, reverse=1, eps=1e-6, dtype=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "ARG"), (dict(gq=None), "ARG"), (dict(gk=None), "ARG"), (dict(dq=None), "ARG"), (dict(dk=None), "ARG"),
    (dict(pos=None), "ARG"), (dict(alpha=-1.0), "ARG"), (dict(base=0.0), "ARG"), (dict(dtype=-1), "ARG"), (dict(D=127), "SHAPE"),
    (dict(H=5), "SHAPE"), (dict(N=-2), "SHAPE"), (dict(ldgq=508), "SHAPE"), (dict(lddk=252), "SHAPE"), (dict(dq=OFF4), "ALIGN"),
    (dict(ldgk=257), "ALIGN"), (dict(pos=OFF2), "ALIGN")])
def test_qk_norm_rope_backward_refuses(kw, status):
    assert _call("nc_qk_norm_rope_backward", QB_NAMES, QB_BASE, **kw) == S["NC_ERR_" + status]


PA_NAMES = ("q ldq kp vp ldp lsp pl ks vs lds lss sl out lse B G Tq H Hkv D P_max S_max window scale ws wsb stream").split()
PA_BASE = dict(q=P, ldq=512, kp=P, vp=P, ldp=256, lsp=2560, pl=P, ks=P, vs=P, lds=256, lss=1280, sl=P, out=P, lse=P, B=4, G=2,
               Tq=1, H=4, Hkv=2, D=128, P_max=10, S_max=5, window=0, scale=0.1, ws=P, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "ARG"), (dict(out=None), "ARG"), (dict(kp=None), "ARG"), (dict(vp=None), "ARG"), (dict(pl=None), "ARG"),
    (dict(ks=None), "ARG"), (dict(vs=None), "ARG"), (dict(sl=None), "ARG"), (dict(scale=0.0), "ARG"), (dict(scale=NAN), "ARG"),
    (dict(scale=INF), "ARG"), (dict(scale=-1.0), "ARG"),
    (dict(D=64), "SHAPE"), (dict(B=0), "SHAPE"), (dict(G=0), "SHAPE"), (dict(G=3), "SHAPE"), (dict(Tq=0), "SHAPE"),
    (dict(Hkv=3), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(P_max=-1), "SHAPE"), (dict(P_max=0, S_max=0), "SHAPE"),
    (dict(P_max=1 << 30, S_max=1), "SHAPE"), (dict(H=258, Hkv=2, ldq=258 * 128), "SHAPE"), (dict(B=1 << 20, G=1, Tq=1 << 12), "SHAPE"),
    (dict(ldq=504), "SHAPE"), (dict(ldp=248), "SHAPE"), (dict(lds=248), "SHAPE"), (dict(lsp=2552), "SHAPE"),
    (dict(lss=1272), "SHAPE"), (dict(ldp=1 << 37), "SHAPE"), (dict(lss=1 << 39), "SHAPE"), (dict(ldq=1 << 39), "SHAPE"),
    (dict(q=OFF4), "ALIGN"), (dict(vp=OFF4), "ALIGN"), (dict(ks=OFF4), "ALIGN"), (dict(out=OFF4), "ALIGN"), (dict(ldq=516), "ALIGN"),
    (dict(ldp=260, lsp=2600), "ALIGN"), (dict(lds=260, lss=1300), "ALIGN"), (dict(lsp=2564), "ALIGN"), (dict(pl=OFF2), "ALIGN"),
    (dict(sl=OFF2), "ALIGN"), (dict(ws=OFF4), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(wsb=15), "WORKSPACE")])
def test_prefix_attention_refuses(kw, status):
    assert _call("nc_prefix_attention", PA_NAMES, PA_BASE, **kw) == S["NC_ERR_" + status]


def test_prefix_attention_workspace():
    need = nc.nc_prefix_attention_workspace_bytes
    # either side holds 512 + 4 bytes per query row at least
    assert need(4, 2, 1, 4, 2, 10, 5, 0) >= 2 * 4 * 4 * 516
    assert need(4, 2, 1, 4, 2, 10, 0, 0) < need(4, 2, 1, 4, 2, 10, 5, 0)
    assert need(4, 3, 1, 4, 2, 10, 5, 0) == 0 and need(4, 2, 1, 4, 3, 10, 5, 0) == 0
    assert _call("nc_prefix_attention", PA_NAMES, PA_BASE, wsb=need(4, 2, 1, 4, 2, 10, 5, 0) - 1) == S["NC_ERR_WORKSPACE"]


PL_NAMES = ("z ldl y adv per old ref B T V lo hi beta norm stats logp dz lddl dtype ws wsb stream").split()
PL_BASE = dict(z=P, ldl=16, y=P, adv=P, per=0, old=None, ref=None, B=2, T=3, V=16, lo=0.2, hi=0.2, beta=0.0, norm=0, stats=P,
               logp=P, dz=P, lddl=16, dtype=1, ws=P, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), "ARG"), (dict(y=None), "ARG"), (dict(adv=None), "ARG"), (dict(stats=None), "ARG"), (dict(logp=None), "ARG"),
    (dict(lo=-0.1), "ARG"), (dict(lo=1.0), "ARG"), (dict(lo=NAN), "ARG"), (dict(hi=-0.1), "ARG"), (dict(hi=INF), "ARG"),
    (dict(beta=-1.0), "ARG"), (dict(beta=NAN), "ARG"), (dict(norm=2), "ARG"), (dict(per=2), "ARG"), (dict(dtype=3), "ARG"),
    (dict(B=0), "SHAPE"), (dict(T=0), "SHAPE"), (dict(V=0), "SHAPE"), (dict(ldl=15), "SHAPE"), (dict(lddl=15), "SHAPE"),
    (dict(B=1 << 16, T=1 << 16), "SHAPE"), (dict(B=1 << 15, T=(1 << 15) + 1), "SHAPE"), (dict(z=OFF2), "ALIGN"), (dict(dz=OFF2), "ALIGN"), (dict(y=OFF2), "ALIGN"),
    (dict(adv=OFF2), "ALIGN"), (dict(old=OFF2), "ALIGN"), (dict(ref=OFF2), "ALIGN"), (dict(stats=OFF2), "ALIGN"),
    (dict(logp=OFF2), "ALIGN"), (dict(ws=OFF4), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(wsb=100), "WORKSPACE")])
def test_policy_loss_refuses(kw, status):
    assert _call("nc_policy_loss", PL_NAMES, PL_BASE, **kw) == S["NC_ERR_" + status]


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_wrong_tensors():
    i32 = torch.int32
    q, k, pos = _t(4, 4, 128), _t(4, 2, 128), _t(4, dtype=i32)
    bad = [
        lambda: nc.nc_qk_norm_rope(q, k, pos, q.clone(), k.clone()),                            # on the CPU
        lambda: nc.nc_qk_norm_rope(q.half(), k, pos, q, k),
        lambda: nc.nc_qk_norm_rope(q, k.float(), pos, q, k),
        lambda: nc.nc_qk_norm_rope(q, k, pos.long(), q, k),
        lambda: nc.nc_qk_norm_rope(q, k, pos[:3], q, k),
        lambda: nc.nc_qk_norm_rope(q, k, pos, q[:, :3], k),
        lambda: nc.nc_qk_norm_rope(q, k, pos, q, k, v=k),
        lambda: nc.nc_qk_norm_rope(q[0], k, pos, q, k),
        lambda: nc.nc_qk_norm_rope_backward(q, k, pos, q, k[:3], q, k),
        lambda: nc.nc_qk_norm_rope_backward(q, k, pos, q.float(), k, q, k),
    ]
    q4, kp, ks, lens = _t(4, 1, 4, 128), _t(2, 10, 2, 128), _t(4, 5, 2, 128), _t(2, dtype=i32)
    sl = _t(4, dtype=i32)
    bad += [
        lambda: nc.nc_prefix_attention(q4, kp, kp, lens, ks, ks, sl, q4.clone()),               # on the CPU
        lambda: nc.nc_prefix_attention(q4, kp, kp, lens, ks[:3], ks[:3], sl[:3], q4),
        lambda: nc.nc_prefix_attention(q4, kp, None, lens, ks, ks, sl, q4),
        lambda: nc.nc_prefix_attention(q4, None, None, None, None, None, None, q4),
        lambda: nc.nc_prefix_attention(q4, kp, kp, sl, ks, ks, sl, q4),
        lambda: nc.nc_prefix_attention(q4, kp, kp, lens.long(), ks, ks, sl, q4),
        lambda: nc.nc_prefix_attention(q4.float(), kp, kp, lens, ks, ks, sl, q4),
        lambda: nc.nc_prefix_attention(q4, kp, kp[:, :, :1], lens, ks, ks, sl, q4),
    ]
    z, y, adv, out, lp = _t(2, 3, 16), _t(2, 3, dtype=i32), _t(2, dtype=torch.float32), _t(3, dtype=torch.float32), _t(2, 3, dtype=torch.float32)
    bad += [
        lambda: nc.nc_policy_loss(z, y, adv, out, lp),                                          # on the CPU
        lambda: nc.nc_policy_loss(z.double(), y, adv, out, lp),
        lambda: nc.nc_policy_loss(z, y.long(), adv, out, lp),
        lambda: nc.nc_policy_loss(z, y, adv[:1], out, lp),
        lambda: nc.nc_policy_loss(z, y, adv, out[:2], lp),
        lambda: nc.nc_policy_loss(z, y, adv, out, lp, z.float()),
        lambda: nc.nc_policy_loss(z[0], y, adv, out, lp),
    ]
    for f in bad:
        with pytest.raises(nc.NcError):
            f()
