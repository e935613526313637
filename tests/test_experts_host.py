"""Refusals of the router's choice and of the products, without a GPU: the C
ABI's status codes (no call here passes every check) and the binding's
layout checks on CPU tensors."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B

FAKE = 0x7F0000000000
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _route(x=FAKE, stride=64, dtype=1, bias=None, T=4, E=64, K=4, score=0, ng=1, tg=1, ids=FAKE,
           w=FAKE):
    return B.load().moe_ep_route_topk(x, stride, dtype, bias, T, E, K, score, ng, tg, 1, 1.0, ids,
                                      w, None)


def test_route_refusals():
    for kw in (dict(E=0), dict(E=1025, stride=2000), dict(K=0), dict(K=65, E=128, stride=128),
               dict(K=65), dict(T=-1), dict(score=2), dict(ng=0), dict(ng=3), dict(ng=4, tg=5),
               dict(ng=4, tg=0), dict(ng=16, tg=1, K=5), dict(stride=63), dict(x=None),
               dict(ids=None), dict(w=None), dict(T=(1 << 29) + 1), dict(ng=128, E=128, stride=128),
               dict(stride=1 << 62)):
        assert _route(**kw) == B.EINVAL, kw
    assert _route(dtype=2) == B.EDTYPE
    assert _route(x=FAKE + 2) == B.EALIGN
    assert _route(x=FAKE + 1, dtype=0) == B.EALIGN
    assert _route(ids=FAKE + 2) == B.EALIGN and _route(w=FAKE + 2) == B.EALIGN
    assert _route(bias=FAKE + 1) == B.EALIGN
    assert _route(T=0) == B.OK                      # nothing to do, nothing enqueued


def _experts(x=FAKE, xs=None, w=FAKE, ws=None, bias=None, bs=0, cnt=FAKE, e=4, rows=32, H=64, N=32,
             act=0, out=FAKE, os=None, dt=0):
    nw = 2 * N if act == 3 else N
    return B.load().moe_ep_expert_matmul(
        x, rows * H if xs is None else xs, w, nw * H if ws is None else ws, bias, bs, cnt, e, rows,
        H, N, act, out, rows * N if os is None else os, dt, None)


def test_expert_matmul_refusals():
    for kw in (dict(e=0), dict(e=1025), dict(rows=-1), dict(rows=1 << 31), dict(H=0), dict(N=0),
               dict(H=(1 << 20) + 8), dict(N=(1 << 20) + 8), dict(act=4), dict(act=-1),
               dict(x=None), dict(w=None), dict(out=None), dict(cnt=None), dict(xs=32 * 64 - 8),
               dict(ws=32 * 64 - 8), dict(os=32 * 32 - 8), dict(xs=-8), dict(bias=FAKE, bs=28),
               dict(N=1 << 15, H=1 << 15), dict(N=1 << 14, H=1 << 15, act=3),
               dict(xs=1 << 62), dict(rows=1 << 30, N=1 << 10, e=1024)):
        assert _experts(**kw) == B.EINVAL, kw
    for kw in (dict(H=60), dict(N=36), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(out=FAKE + 4),
               dict(xs=32 * 64 + 4), dict(ws=32 * 64 + 4), dict(os=32 * 32 + 4),
               dict(bias=FAKE + 4, bs=32), dict(bias=FAKE, bs=34)):
        assert _experts(**kw) == B.EALIGN, kw
    assert _experts(dt=2) == B.EDTYPE and _experts(dt=7) == B.EDTYPE
    assert _experts(rows=0) == B.OK


def _fp8(x=FAKE, xs=FAKE, xss=None, w=FAKE, ws=FAKE, wss=None, e=2, rows=16, H=256, N=128, act=0,
         dt=0, osc=None, oss=None, cnt=FAKE):
    nw = 2 * N if act == 3 else N
    blocks = -(-N // 128) * (2 if act == 3 else 1) if N > 0 else 1
    return B.load().moe_ep_expert_matmul_fp8(
        x, rows * H, xs, rows * 4 if xss is None else xss, w, nw * H, ws,
        blocks * (H // 128) if wss is None else wss, None, 0, cnt, e, rows, H, N, act, FAKE,
        rows * N, dt, osc, rows * 4 if oss is None else oss, None)


def test_expert_matmul_fp8_refusals():
    for kw in (dict(H=192), dict(xs=None), dict(ws=None), dict(xss=60), dict(wss=1),
               dict(act=3, wss=2), dict(dt=2), dict(osc=FAKE), dict(dt=1, osc=FAKE),
               dict(dt=2, osc=FAKE, N=144), dict(dt=2, osc=FAKE, oss=60), dict(cnt=None)):
        assert _fp8(**kw) == B.EINVAL, kw
    for kw in (dict(xs=FAKE + 4), dict(xss=66), dict(ws=FAKE + 8), dict(x=FAKE + 8),
               dict(dt=2, osc=FAKE + 4), dict(dt=2, osc=FAKE, oss=66)):
        assert _fp8(**kw) == B.EALIGN, kw
    assert _fp8(dt=3) == B.EDTYPE
    assert _fp8(rows=0) == B.OK


def _mm(x=FAKE, xs=64, w=FAKE, ws=64, bias=None, T=8, H=64, N=32, act=0, res=None, rs=32, out=FAKE,
        os=32, dt=0):
    return B.load().moe_ep_matmul(x, xs, w, ws, bias, T, H, N, act, res, rs, out, os, dt, None)


def test_matmul_refusals():
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(N=0), dict(xs=56), dict(ws=56),
               dict(ws=0), dict(os=24), dict(res=FAKE, rs=24), dict(act=9), dict(x=None),
               dict(w=None), dict(out=None), dict(xs=1 << 22), dict(N=1 << 20, ws=1 << 12),
               dict(res=FAKE, rs=40), dict(os=1 << 62)):
        assert _mm(**kw) == B.EINVAL, kw
    for kw in (dict(H=60), dict(N=28), dict(xs=68), dict(ws=68), dict(os=36),
               dict(res=FAKE + 64, rs=36), dict(x=FAKE + 2), dict(w=FAKE + 8), dict(out=FAKE + 8),
               dict(bias=FAKE + 4), dict(res=FAKE + 8)):
        assert _mm(**kw) == B.EALIGN, kw
    assert _mm(dt=2) == B.EDTYPE
    assert _mm(T=0) == B.OK


# -- the binding's layout checks ---------------------------------------------

def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_wrong_layouts():
    i32 = torch.int32
    x, w, o = z(2, 16, 64), z(2, 32, 64), z(2, 16, 32)
    cnt = z(2, dtype=i32)
    bad = [
        lambda: B.prepare_expert_matmul(x[0], w, cnt, o),
        lambda: B.prepare_expert_matmul(x, w[:, :24], cnt, o),
        lambda: B.prepare_expert_matmul(x, w, cnt, o, "silu_gated"),
        lambda: B.prepare_expert_matmul(x, w, cnt, o, "tanh"),
        lambda: B.prepare_expert_matmul(x.float(), w, cnt, o),
        lambda: B.prepare_expert_matmul(x, w.half(), cnt, o),
        lambda: B.prepare_expert_matmul(x, w, cnt, o.half()),
        lambda: B.prepare_expert_matmul(x, w, cnt[:1], o),
        lambda: B.prepare_expert_matmul(x, w, cnt.long(), o),
        lambda: B.prepare_expert_matmul(x, w, cnt, o, bias=z(2, 32)),
        lambda: B.prepare_expert_matmul(x, w, cnt, o, bias=z(2, 24, dtype=F32)),
        lambda: B.prepare_expert_matmul(z(2, 64, 16).transpose(1, 2), w, cnt, o),
        lambda: B.prepare_expert_matmul(z(1, 16, 64).expand(2, 16, 64), w, cnt, o),
        lambda: B.prepare_expert_matmul(x, w, cnt, z(2, 8, 32)),
        lambda: B.prepare_matmul(x, w[0], o[0]),
        lambda: B.prepare_matmul(x[0], w[0], o[0], residual=o[1].float()),
        lambda: B.prepare_matmul(x[0], w[0], o[0], residual=o[1][:8]),
        lambda: B.prepare_matmul(x[0], w[0], o[0], bias=z(33, dtype=F32)),
        lambda: B.prepare_matmul(x[0], z(64, 32).t(), o[0]),
        lambda: B.prepare_matmul(z(1, 64).expand(16, 64), w[0], o[0]),
        lambda: B.prepare_route_topk(z(4, 8).half(), z(4, 2, dtype=i32), z(4, 2, dtype=F32)),
        lambda: B.prepare_route_topk(z(4, 8), z(4, 2, dtype=torch.int64), z(4, 2, dtype=F32)),
        lambda: B.prepare_route_topk(z(4, 8), z(4, 2, dtype=i32), z(4, 3, dtype=F32)),
        lambda: B.prepare_route_topk(z(4, 8), z(3, 2, dtype=i32), z(3, 2, dtype=F32)),
        lambda: B.prepare_route_topk(z(8, 4).t(), z(4, 2, dtype=i32), z(4, 2, dtype=F32)),
        lambda: B.prepare_route_topk(z(4, 8), z(4, 2, dtype=i32), z(4, 2, dtype=F32), "max"),
        lambda: B.prepare_route_topk(z(4, 8), z(4, 2, dtype=i32), z(4, 2, dtype=F32),
                                     bias=z(9, dtype=F32)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_wrong_fp8_layouts():
    cnt = z(2, dtype=torch.int32)
    x, w = z(2, 16, 256, dtype=F8), z(2, 128, 256, dtype=F8)
    xs, ws = z(2, 16, 4, dtype=F32), z(2, 1, 2, dtype=F32)
    o, c, s = z(2, 16, 128), z(2, 16, 128, dtype=F8), z(2, 16, 4, dtype=F32)
    bad = [
        lambda: B.prepare_expert_matmul_fp8(x, xs[:, :, :2], w, ws, cnt, o),
        lambda: B.prepare_expert_matmul_fp8(x, xs, w, z(2, 2, 2, dtype=F32), cnt, o),
        lambda: B.prepare_expert_matmul_fp8(x, xs, w, ws, cnt, c),
        lambda: B.prepare_expert_matmul_fp8(x, xs, w, ws, cnt, o, out_scale=s),
        lambda: B.prepare_expert_matmul_fp8(x, xs, w, ws, cnt, c, out_scale=s[:, :, :1]),
        lambda: B.prepare_expert_matmul_fp8(x.float().to(BF16), xs, w, ws, cnt, o),
        lambda: B.prepare_expert_matmul_fp8(x[:, :, :192].contiguous(), xs,
                                            w[:, :, :192].contiguous(), ws, cnt, o),
        lambda: B.prepare_expert_matmul_fp8(x, xs.double(), w, ws, cnt, o),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="one GPU"):
        B.prepare_matmul(z(4, 64), z(32, 64), z(4, 32))
