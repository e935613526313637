"""Refusals of the products with 4-bit weights and of a router's training terms,
without a GPU: the C ABI's status codes (no call here passes every check) and
the binding's layout checks on CPU tensors."""
import ctypes

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B

FAKE = 0x7F0000000000
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _experts(x=FAKE, xs=None, w=FAKE, ws=None, sc=FAKE, ss=None, group=16, wg=None, bias=None, bs=0,
             cnt=FAKE, e=4, rows=32, H=64, N=32, act=0, out=FAKE, os=None, dt=0):
    nw = 2 * N if act == 3 else N
    return B.load().moe_ep_expert_matmul_w4(
        x, rows * H if xs is None else xs, w, nw * H // 2 if ws is None else ws, sc,
        nw * 16 if ss is None else ss, group, wg, bias, bs, cnt, e, rows, H, N, act, out,
        rows * N if os is None else os, dt, None)


def test_expert_matmul_w4_refusals():
    for kw in (dict(e=0), dict(e=1025), dict(rows=-1), dict(rows=1 << 31), dict(H=0), dict(N=0),
               dict(rows=(1 << 31) - 255), dict(H=(1 << 20) + 32), dict(N=(1 << 20) + 8),
               dict(act=4), dict(act=-1), dict(x=None), dict(w=None), dict(sc=None),
               dict(out=None), dict(cnt=None), dict(xs=32 * 64 - 8), dict(ws=32 * 32 - 16),
               dict(ss=32 * 16 - 16), dict(os=32 * 32 - 8), dict(xs=-8), dict(ws=-16),
               dict(bias=FAKE, bs=28), dict(N=1 << 15, H=1 << 15), dict(xs=1 << 62),
               dict(ss=(1 << 63) - 16), dict(rows=1 << 30, N=1 << 10, e=1024), dict(group=8),
               dict(group=0), dict(group=64), dict(group=-16), dict(H=512, group=16)):
        assert _experts(**kw) == B.EINVAL, kw
    for kw in (dict(H=48), dict(N=36), dict(x=FAKE + 8), dict(w=FAKE + 4), dict(sc=FAKE + 8),
               dict(out=FAKE + 4), dict(xs=32 * 64 + 4), dict(ws=32 * 32 + 8),
               dict(ss=32 * 16 + 8), dict(os=32 * 32 + 4), dict(bias=FAKE + 4, bs=32),
               dict(bias=FAKE, bs=34), dict(wg=FAKE + 2), dict(N=4, ws=4 * 32, dt=0)):
        assert _experts(**kw) == B.EALIGN, kw
    assert _experts(dt=2) == B.EDTYPE and _experts(dt=7) == B.EDTYPE
    assert _experts(rows=0) == B.OK and _experts(rows=0, x=None, w=None, sc=None) == B.OK


def _mm(x=FAKE, xs=64, w=FAKE, ws=32, sc=FAKE, ss=16, group=16, wg=None, bias=None, T=8, H=64, N=32,
        act=0, res=None, rs=32, out=FAKE, os=32, dt=0):
    return B.load().moe_ep_matmul_w4(x, xs, w, ws, sc, ss, group, wg, bias, T, H, N, act, res, rs,
                                     out, os, dt, None)


def test_matmul_w4_refusals():
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(N=0), dict(xs=56), dict(ws=16),
               dict(ws=0), dict(ws=-32), dict(ss=0), dict(ss=-16), dict(ss=1 << 30),
               dict(ws=1 << 30), dict(os=24), dict(res=FAKE, rs=24), dict(act=9), dict(x=None),
               dict(w=None), dict(sc=None), dict(out=None), dict(xs=1 << 22),
               dict(N=1 << 20, ws=1 << 12), dict(N=1 << 20, ss=1 << 12),
               dict(res=FAKE, rs=40), dict(os=1 << 62), dict(group=17), dict(H=512, ws=256, xs=512),
               dict(H=1 << 20, N=1 << 16, xs=1 << 20, ws=1 << 19, ss=1 << 16)):
        assert _mm(**kw) == B.EINVAL, kw
    for kw in (dict(H=48), dict(N=28), dict(xs=68), dict(ws=40), dict(ss=24), dict(os=36),
               dict(res=FAKE + 64, rs=36), dict(x=FAKE + 2), dict(w=FAKE + 8), dict(sc=FAKE + 4),
               dict(out=FAKE + 8), dict(bias=FAKE + 4), dict(res=FAKE + 8), dict(wg=FAKE + 1)):
        assert _mm(**kw) == B.EALIGN, kw
    assert _mm(dt=2) == B.EDTYPE
    assert _mm(T=0) == B.OK


def _balance(x=FAKE, stride=64, dtype=1, ids=FAKE, T=4, E=64, K=4, score=0, start=None, S=1,
             counts=FAKE, tokens=FAKE, mean=FAKE, loss=FAKE, ws=FAKE, size=1 << 40):
    return B.load().moe_ep_balance_loss(x, stride, dtype, ids, T, E, K, score, start, S, counts,
                                        tokens, mean, loss, ws, size, None)


def test_balance_loss_refusals():
    for kw in (dict(E=0), dict(E=1025, stride=2000), dict(K=0), dict(K=65), dict(T=-1),
               dict(score=2), dict(score=-1), dict(S=0), dict(S=-1), dict(S=2), dict(stride=63),
               dict(x=None), dict(ids=None), dict(counts=None), dict(tokens=None),
               dict(mean=None), dict(loss=None), dict(T=(1 << 29) + 1), dict(stride=1 << 62),
               dict(S=1 << 30, start=FAKE), dict(T=1 << 31, K=1)):
        assert _balance(**kw) == B.EINVAL, kw
    assert _balance(dtype=2) == B.EDTYPE
    for kw in (dict(x=FAKE + 2), dict(x=FAKE + 1, dtype=0), dict(ids=FAKE + 2),
               dict(start=FAKE + 1), dict(counts=FAKE + 2), dict(tokens=FAKE + 2),
               dict(mean=FAKE + 3), dict(loss=FAKE + 2), dict(T=5000, ws=FAKE + 8)):
        assert _balance(**kw) == B.EALIGN, kw
    need = B.moe_ep_balance_workspace_bytes(5000, 64, 1)
    assert need > 0 and need % 16 == 0
    assert _balance(T=5000, ws=None) == B.EWORKSPACE
    assert _balance(T=5000, size=need - 1) == B.EWORKSPACE


def test_balance_workspace():
    assert B.moe_ep_balance_workspace_bytes(0, 8) == 0
    assert B.moe_ep_balance_workspace_bytes(1, 256, 9) == 0
    few, many = (B.moe_ep_balance_workspace_bytes(65536, 256, s) for s in (1, 64))
    assert 0 < few < many < 4 << 20
    for bad in ((-1, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (1 << 31, 8, 1),
                (4, 1024, 1 << 21)):
        with pytest.raises(B.MoeEpError) as e:
            B.moe_ep_balance_workspace_bytes(*bad)
        assert e.value.status == B.EINVAL
    assert B.load().moe_ep_balance_workspace_bytes(4, 8, 1, None) == B.EINVAL
    n = ctypes.c_size_t()
    # the largest that is allowed: no product overflows
    assert B.load().moe_ep_balance_workspace_bytes((1 << 31) - 1, 1024, 1 << 19,
                                                   ctypes.byref(n)) == B.OK
    assert n.value > 0


def _grad(x=FAKE, stride=64, dtype=1, ids=FAKE, T=4, E=64, K=4, score=0, gw=FAKE, start=None, S=1,
          counts=FAKE, tokens=FAKE, gl=FAKE, out=FAKE + 64, gs=64, gd=1):
    return B.load().moe_ep_route_backward(x, stride, dtype, ids, T, E, K, score, 1, 1.0, gw, start,
                                          S, counts, tokens, gl, out, gs, gd, None)


def test_route_backward_refusals():
    for kw in (dict(E=0), dict(E=1025, stride=2000, gs=2000), dict(K=0), dict(K=65), dict(T=-1),
               dict(score=2), dict(stride=63), dict(gs=63), dict(x=None), dict(ids=None),
               dict(out=None), dict(T=(1 << 29) + 1), dict(stride=1 << 62), dict(gs=1 << 62),
               dict(gw=None, gl=None), dict(counts=None), dict(tokens=None), dict(S=0),
               dict(S=2), dict(S=1 << 30, start=FAKE), dict(out=FAKE, gs=72),
               dict(out=FAKE, gd=0)):
        assert _grad(**kw) == B.EINVAL, kw
    assert _grad(dtype=2) == B.EDTYPE and _grad(gd=2) == B.EDTYPE
    for kw in (dict(x=FAKE + 2), dict(x=FAKE + 1, dtype=0), dict(ids=FAKE + 2), dict(gw=FAKE + 2),
               dict(gl=FAKE + 2), dict(out=FAKE + 2), dict(out=FAKE + 1, gd=0),
               dict(start=FAKE + 2), dict(counts=FAKE + 1), dict(tokens=FAKE + 1)):
        assert _grad(**kw) == B.EALIGN, kw
    assert _grad(T=0) == B.OK and _grad(T=0, gl=None, counts=None, tokens=None) == B.OK


# -- the binding's layout checks ---------------------------------------------

def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def _refused(bad, match=None):
    for i, f in enumerate(bad):
        with pytest.raises(ValueError, match=match):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_wrong_w4_layouts():
    x, w, s, o = z(2, 16, 64), z(2, 32, 32, dtype=U8), z(2, 32, 16, dtype=U8), z(2, 16, 32)
    cnt = z(2, dtype=I32)
    E = B.prepare_expert_matmul_w4
    _refused([
        lambda: E(x[0], w, s, cnt, o),
        lambda: E(x, w[:, :24], s, cnt, o),
        lambda: E(x, w, s, cnt, o, 16, "silu_gated"),
        lambda: E(x, w, s, cnt, o, 16, "tanh"),
        lambda: E(x, w, s, cnt, o, 24),
        lambda: E(x.float(), w, s, cnt, o),
        lambda: E(x, w.to(torch.int8), s, cnt, o),
        lambda: E(x, w, s[:, :, :4], cnt, o),
        lambda: E(x, w, s.view(torch.float8_e8m0fnu), cnt, o, 16),
        lambda: E(x, w, s.view(torch.float8_e4m3fn), cnt, o, 32),
        lambda: E(x, w, s.view(torch.int8), cnt, o),
        lambda: E(x, w, s[:, :16], cnt, o),
        lambda: E(x, w, s[0], cnt, o),
        lambda: E(x, w, s, cnt, o.half()),
        lambda: E(x, w, s, cnt[:1], o),
        lambda: E(x, w, s, cnt.long(), o),
        lambda: E(x, w, s, cnt, o, bias=z(2, 24, dtype=F32)),
        lambda: E(x, w, s, cnt, o, w_global=z(2, dtype=F32)),
        lambda: E(x, w, s, cnt, o, w_global=z(2, 2, dtype=F32)),
        lambda: E(x, w, s, cnt, o, w_global=z(2, 1)),
        lambda: E(z(2, 16, 48), z(2, 32, 24, dtype=U8), s, cnt, o),
        lambda: E(z(1, 16, 64).expand(2, 16, 64), w, s, cnt, o),
        lambda: E(x, z(1, 32, 32, dtype=U8).expand(2, 32, 32), s, cnt, o),
    ])
    M = B.prepare_matmul_w4
    _refused([
        lambda: M(x, w, s, o),
        lambda: M(x[0], w[0], s[0], o[0], residual=o[1].float()),
        lambda: M(x[0], w[0], s[0], o[0], residual=o[1][:8]),
        lambda: M(x[0], w[0], s[0], o[0], bias=z(33, dtype=F32)),
        lambda: M(x[0], w[0], s[0][:, :3], o[0]),
        lambda: M(x[0], w[0], z(33, 16, dtype=U8), o[0]),
        lambda: M(x[0], w[0], s, o[0]),
        lambda: M(x[0], z(32, 32, dtype=U8).t(), s[0], o[0]),
        lambda: M(x[0], w[0], s[0], o[0], w_global=z(2, dtype=F32)),
        lambda: M(z(1, 64).expand(16, 64), w[0], s[0], o[0]),
    ])
    _refused([lambda: M(x[0], w[0], s[0], o[0]), lambda: E(x, w, s, cnt, o)], "one GPU")


def test_binding_refuses_wrong_routing_layouts():
    x, ids = z(6, 8, dtype=F32), z(6, 2, dtype=I32)
    c, t, m, l = z(1, 8, dtype=I32), z(1, dtype=I32), z(1, 8, dtype=F32), z(1, dtype=F32)
    L = B.prepare_balance_loss
    _refused([
        lambda: L(x.half(), ids, c, t, m, l),
        lambda: L(x[0], ids, c, t, m, l),
        lambda: L(x, ids.long(), c, t, m, l),
        lambda: L(x, ids[:5], c, t, m, l),
        lambda: L(x, z(2, 6, dtype=I32).t(), c, t, m, l),
        lambda: L(z(8, 6, dtype=F32).t(), ids, c, t, m, l),
        lambda: L(x, ids, c[:, :7], t, m, l),
        lambda: L(x, ids, c.float(), t, m, l),
        lambda: L(x, ids, c, t.long(), m, l),
        lambda: L(x, ids, c, t, m.double(), l),
        lambda: L(x, ids, c, t, m, l[0]),
        lambda: L(x, ids, c, t, m, l, score="max"),
        lambda: L(x, ids, c, t, m, l, seq_start=z(1, dtype=I32)),
        lambda: L(x, ids, c, t, m, l, seq_start=z(2, dtype=torch.int64)),
        lambda: L(x, ids, z(2, 8, dtype=I32), z(2, dtype=I32), z(2, 8, dtype=F32), z(2, dtype=F32)),
        lambda: L(x, ids, z(8, 2, dtype=I32).t()[:1], t, z(8, 3, dtype=F32).t()[:1], l,
                  workspace=z(4, 6)[:, ::2]),
    ])
    G = B.prepare_route_backward
    gw, gl, out = z(6, 2, dtype=F32), z(1, dtype=F32), z(6, 8)
    _refused([
        lambda: G(x, ids, out),
        lambda: G(x, ids, out.half(), grad_weights=gw),
        lambda: G(x, ids, out[:5], grad_weights=gw),
        lambda: G(x, ids, z(8, 6).t(), grad_weights=gw),
        lambda: G(x, ids, out, grad_weights=gw[:, :1]),
        lambda: G(x, ids, out, grad_weights=gw.double()),
        lambda: G(x, ids, out, grad_weights=z(2, 6, dtype=F32).t()),
        lambda: G(x, ids, out, grad_loss=gl),
        lambda: G(x, ids, out, grad_loss=gl, counts=c),
        lambda: G(x, ids, out, grad_loss=gl, counts=c, tokens=z(2, dtype=I32)),
        lambda: G(x, ids, out, grad_weights=gw, counts=c, tokens=t),
        lambda: G(x, ids, out, grad_weights=gw, seq_start=z(2, dtype=I32)),
        lambda: G(x, ids, out, grad_loss=z(2, dtype=F32), counts=z(2, 8, dtype=I32),
                  tokens=z(2, dtype=I32)),
        lambda: G(x, ids, out, "top", grad_weights=gw),
    ])
    _refused([lambda: L(x, ids, c, t, m, l), lambda: G(x, ids, out, grad_weights=gw)], "one GPU")
