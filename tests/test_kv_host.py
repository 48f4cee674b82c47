"""Refusals of the cache, attention and norm entry points: host checks, made
before any device call (no GPU needed)."""
import ctypes

import pytest
import torch

from nvfp4_mixture_experts_top_gb300 import binding as B

P16, P8, P2 = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8), ctypes.c_void_p(4096 + 2)
OK, INVAL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


def _plan(B_=4, S=16, ld=8, M=8, nf=9, T=4, **over):
    a = dict(ctx=P16, new=P16, table=P16, free=P16, count=P16, start=P16, kv=P16, slots=P16, left=P8, st=None)
    a.update(over)
    return B.load().kv_plan(a["ctx"], a["new"], B_, S, a["table"], ld, M, a["free"], nf, a["count"], T, a["start"], a["kv"],
                            a["slots"], a["left"], a["st"], None)


@pytest.mark.parametrize("want,over", [
    (INVAL, dict(B_=-1)), (INVAL, dict(T=-1)), (INVAL, dict(nf=-1)), (SHAPE, dict(S=48)), (SHAPE, dict(S=0)),
    (SHAPE, dict(B_=8193)), (SHAPE, dict(M=0)), (SHAPE, dict(ld=7)), (INVAL, dict(count=None)), (INVAL, dict(left=P16)),
    (INVAL, dict(ctx=None)), (INVAL, dict(slots=None)), (INVAL, dict(free=None)), (ALIGN, dict(table=P2))])
def test_plan_refusals(want, over):
    assert _plan(**over) == want


def _append(dt=0, ld_k=256, ld_v=256, T=4, Hkv=2, D=128, P=10, S=64, **over):
    a = dict(k=P16, v=P16, slots=P16, kc=P16, ke=P16, vc=P16, ve=P16, st=None)
    a.update(over)
    return B.load().kv_append(a["k"], a["v"], dt, ld_k, ld_v, a["slots"], T, Hkv, D, P, S, a["kc"], a["ke"], a["vc"],
                              a["ve"], a["st"], None)


@pytest.mark.parametrize("want,over", [
    (INVAL, dict(T=-1)), (INVAL, dict(Hkv=0)), (INVAL, dict(dt=3)), (SHAPE, dict(D=96)), (SHAPE, dict(S=24)),
    (SHAPE, dict(ld_k=255)), (SHAPE, dict(ld_v=260)), (SHAPE, dict(dt=1, ld_v=257)), (SHAPE, dict(P=1 << 26)),
    (OK, dict(T=0, k=None)), (INVAL, dict(k=None)), (INVAL, dict(ve=None)), (ALIGN, dict(k=P8)), (ALIGN, dict(vc=P8)),
    (ALIGN, dict(slots=P2))])
def test_append_refusals(want, over):
    assert _append(**over) == want


def _attn(ld_q=512, ld_t=8, M=8, T=4, B_=2, Hq=4, Hkv=2, D=128, P=10, S=64, n=2, nbytes=None, **over):
    a = dict(q=P16, kc=P16, ke=P16, vc=P16, ve=P16, table=P16, kv=P16, start=P16, out=P16, lse=P16, st=None, ws=P16)
    a.update(over)
    L = B.load()
    if nbytes is None:
        nbytes = L.kv_attention_workspace_bytes(T, B_, Hq, Hkv, D)
    return L.kv_attention(a["q"], ld_q, a["kc"], a["ke"], a["vc"], a["ve"], a["table"], ld_t, M, a["kv"], a["start"], T,
                          B_, Hq, Hkv, D, P, S, n, 0.1, a["out"], a["lse"], a["st"], a["ws"], nbytes, None)


@pytest.mark.parametrize("want,over", [
    (INVAL, dict(T=-1)), (INVAL, dict(B_=-1)), (INVAL, dict(Hkv=0)), (INVAL, dict(n=-1)), (SHAPE, dict(D=32)),
    (SHAPE, dict(S=65)), (SHAPE, dict(Hq=5)), (SHAPE, dict(ld_q=511)), (SHAPE, dict(ld_q=516)), (SHAPE, dict(ld_t=7)),
    (SHAPE, dict(M=0)), (SHAPE, dict(B_=8193)), (OK, dict(T=0, q=None)), (OK, dict(B_=0, q=None)), (INVAL, dict(q=None)),
    (INVAL, dict(out=None)), (INVAL, dict(table=None)), (ALIGN, dict(q=P8)), (ALIGN, dict(kc=P8)), (ALIGN, dict(lse=P2)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(nbytes=0)), (ALIGN, dict(ws=P8))])
def test_attention_refusals(want, over):
    assert _attn(**over) == want


def test_attention_workspace_is_small():
    L = B.load()
    for T, n, Hq, Hkv, D in ((1, 1, 1, 1, 64), (512, 512, 48, 8, 128), (8192, 4, 128, 1, 128), (8192, 8192, 64, 8, 128)):
        assert 0 < L.kv_attention_workspace_bytes(T, n, Hq, Hkv, D) <= 64 << 20
    assert L.kv_attention_workspace_bytes(-1, 1, 1, 1, 64) == 0


def _norm(ld_x=64, dt=0, ld_a=64, g_t=0, g_c=1, T=3, H=64, **over):
    a = dict(x=P16, a=P16, gate=None, post=P16, pre=P16, y=P16, h=P16)
    a.update(over)
    return B.load().block_norm(a["x"], ld_x, a["a"], dt, ld_a, a["gate"], g_t, g_c, a["post"], a["pre"], 1.0, 1e-6, T, H,
                               a["y"], a["h"], None)


@pytest.mark.parametrize("want,over", [
    (INVAL, dict(T=-1)), (INVAL, dict(H=0)), (INVAL, dict(dt=2)), (SHAPE, dict(H=60)), (SHAPE, dict(H=16392, ld_x=16392)),
    (SHAPE, dict(ld_x=56)), (SHAPE, dict(ld_x=65)), (SHAPE, dict(ld_a=68)), (SHAPE, dict(dt=1, ld_a=66)),
    (SHAPE, dict(gate=P16, g_c=2)), (SHAPE, dict(gate=P16, g_t=65)), (SHAPE, dict(gate=P16, g_t=32)),
    (OK, dict(T=0, x=None)), (INVAL, dict(x=None)), (INVAL, dict(a=None, pre=None)), (INVAL, dict(y=None)),
    (INVAL, dict(h=None)), (ALIGN, dict(x=P8)), (ALIGN, dict(gate=P8)), (ALIGN, dict(pre=P8))])
def test_norm_refusals(want, over):
    assert _norm(**over) == want


def test_binding_refuses_wrong_tensors():
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    kc, ke = torch.zeros(4, 2, 16, 64, dtype=u8), torch.zeros(4, 2, dtype=u8)
    table, one = torch.zeros(1, 4, dtype=i32), torch.zeros(1, dtype=i32)
    k = torch.zeros(1, 2, 64, dtype=bf)
    with pytest.raises(ValueError):
        B.kv_append(k, k, one, kc, ke, kc[:3], ke)               # halves of different size
    with pytest.raises(ValueError):
        B.kv_append(k, k.float(), one, kc, ke, kc, ke)           # two types
    with pytest.raises(ValueError):
        B.kv_append(k[:, :1], k[:, :1], one, kc, ke, kc, ke)     # heads missing
    with pytest.raises(ValueError):
        B.kv_append(k, k, one.long(), kc, ke, kc, ke)            # slot type
    with pytest.raises(ValueError):
        B.kv_attention(k.half(), kc, ke, kc, ke, table, one, torch.zeros(2, dtype=i32), 1)
    with pytest.raises(ValueError):
        B.kv_attention(k, kc, ke, kc, ke, table, one, one, 1)    # query_start has B + 1 entries
    with pytest.raises(ValueError):
        B.kv_attention(k, kc, ke, kc, ke, table.t(), one, torch.zeros(2, dtype=i32), 1)
    with pytest.raises(ValueError):
        B.kv_plan(one, one, table, one, torch.zeros(2, dtype=i32), 16, 1)
    x = torch.zeros(2, 64, dtype=bf)
    with pytest.raises(ValueError):
        B.block_norm(x.float())
    with pytest.raises(ValueError):
        B.block_norm(x, gate=x)                                  # a gate without a block output
    with pytest.raises(ValueError):
        B.block_norm(x, x, w_pre=torch.zeros(32, dtype=bf))
    with pytest.raises(ValueError):
        B.block_norm(x, x, gate=torch.zeros(3, 64, dtype=bf))
    with pytest.raises(ValueError):
        B.block_norm(x, x.t())
