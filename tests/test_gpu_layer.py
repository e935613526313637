"""GPU: a whole MoE layer as LogicalEP.step() runs it (router, pack, expert
batch, the experts' two products, reduce, unpack, the expert of all tokens),
against its 64-bit evaluation token by token; eager, over two lanes, and as
replayed graphs."""
import pytest
import torch

import workloads as wl
from combine_topk_ids_dest_amd import binding as B
from combine_topk_ids_dest_amd.emulate import LogicalEP
from parity import say
from products import U, product64, route64

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H8 = 2.0 ** -8                  # half a step of bf16, relative
H4 = 2.0 ** -4                  # and of e4m3


def weights(E, H, I, S, fp8, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, k: torch.randn(*s, generator=g) / k ** 0.5
    d = dict(gate=n(E, H, k=H).to(BF16), shared13=n(2 * S, H, k=H).to(BF16),
             shared2=n(H, S, k=S).to(BF16))
    w13, w2 = n(E, 2 * I, H, k=H), n(E, H, I, k=I)
    if not fp8:
        return dict(d, w13=w13.to(BF16), w2=w2.to(BF16)), w13.to(BF16).double(), w2.to(BF16).double()
    out = []
    for w, halves in ((w13, 2), (w2, 1)):
        rows, cols = w.shape[1] // halves, w.shape[2]
        s = (torch.rand(E, halves * -(-rows // 128), cols // 128, generator=g) + 0.5) * 2.0 ** -8
        row = torch.arange(halves * rows)
        row = row // rows * -(-rows // 128) + row % rows // 128
        full = s.double()[:, row].repeat_interleave(128, dim=2)
        q = (w / full).float().to(F8)
        out.append((q, s, q.double() * full))
    (q13, s13, f13), (q2, s2, f2) = out
    return dict(d, w13=q13, w2=q2, w13_scale=s13, w2_scale=s2), f13, f2


ROUTE = dict(score="sigmoid", n_group=4, topk_group=3, renormalize=True, scale=1.5)


def build(W, E, K, T, H, I, S, fp8, lanes=1, dtype=BF16, bias=None):
    w = wl.WORKLOADS[1].scaled(W=W, E=E, K=K, T=T, cap=T, H=H, pad_frac=0.0)
    mode = dict(quant_group=128) if fp8 else {}
    ep = LogicalEP(T, H, E, K, W, T, [2 * H], dtype, "cuda", fill=0xFF, lanes=lanes, **mode)
    xs = [wl.hidden_bf16(w, s, 3) for s in range(W)]
    for s in range(W):
        ids, wts = wl.routing(w, s, 3)
        ep.set_source(s, ids, wts, [xs[s].view("uint8").reshape(T, 2 * H)])
    d, f13, f2 = weights(E, H, I, S, fp8)
    dev = {k: v.cuda() for k, v in d.items()}
    ep.set_layer(route=dict(ROUTE, bias=None if bias is None else bias.cuda()), **dev)
    return ep, xs, d, f13, f2


def quantised(x):
    """The pack's fp8 rows: exact values (float64)."""
    v = x.float().view(x.shape[0], -1, 128)
    amax = v.abs().amax(dim=2)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (v / s[:, :, None]).to(F8)
    return (q.double() * s.double()[:, :, None]).view(x.shape)


def check(ep, xs, d, f13, f2, fp8, bias=None):
    W, E, K, T, H = ep.W, ep.E, ep.K, ep.T, ep.H
    I = f2.shape[2]
    half = torch.finfo(ep.dtype).eps / 2
    assert int(ep.err.item()) == 0
    for s in range(W):
        x = torch.from_numpy(wl.bf16_bits_to_f32(xs[s]))
        logits = ep._layer["logits"][s].cpu()
        v, e = product64(x.double(), d["gate"].double(), None, "none", E)
        assert bool(((logits.double() - v).abs() <= e + v.abs() * 2.0 ** -24).all())
        ids, wts = route64(logits, bias, K, **{k: ROUTE[k] for k in
                                               ("score", "n_group", "topk_group",
                                                "renormalize", "scale")})
        assert torch.equal(ep.ids[s].cpu(), ids)
        rows = quantised(x) if fp8 else x.double()
        out = torch.zeros(T, H, dtype=torch.float64)
        err = torch.zeros(T, H, dtype=torch.float64)
        per_dest = torch.zeros(W, T, H, dtype=torch.float64)
        dest_err = torch.zeros(W, T, H, dtype=torch.float64)
        for g in range(E):
            hit = (ids == g).any(dim=1)
            if not bool(hit.any()):
                continue
            h, eh = product64(rows[hit], f13[g], None, "silu_gated", I, extra=4)
            # the rows between the products: bf16, or e4m3 with a scale of
            # their amax / 448 (its subnormals' half step 2^-10)
            if fp8:
                sc = (h.abs() + eh).view(-1, I // 128, 128).amax(dim=2) / 448
                eh = eh + (h.abs() + eh) * H4 + sc.repeat_interleave(128, 1) * 2.0 ** -10
            else:
                eh = eh + (h.abs() + eh) * H8
            w2 = f2[g]
            y = h @ w2.t()
            ey = eh @ w2.abs().t() + (I + 4) * U * ((h.abs() + eh) @ w2.abs().t())
            ey = ey + (y.abs() + ey) * half
            wt = (wts * (ids == g)).sum(dim=1)[hit, None]
            r = g // ep.e_local
            per_dest[r, hit] += wt * y
            dest_err[r, hit] += wt * (ey + 4 * U * y.abs())
        dest_err += (per_dest.abs() + dest_err) * half
        out, err = per_dest.sum(0), dest_err.sum(0)
        err = err + (W + 1) * U * per_dest.abs().sum(0) + (out.abs() + err) * half
        h, eh = product64(x.double(), d["shared13"].double(), None, "silu_gated",
                          d["shared2"].shape[1])
        eh = eh + (h.abs() + eh) * H8
        w2 = d["shared2"].double()
        y = h @ w2.t()
        ey = eh @ w2.abs().t() + h.shape[1] * U * ((h.abs() + eh) @ w2.abs().t())
        out, err = out + y, err + ey + U * (out + y).abs()
        err = err + (out.abs() + err) * half
        got = ep.out[s].double().cpu()
        assert bool(((got - out).abs() <= err).all()), (s, float(((got - out).abs() / err).max()))
        # and far inside of the bound on the whole
        assert float((got - out).norm() / out.norm()) < (0.06 if fp8 else 0.02)


@pytest.mark.gpu
@pytest.mark.parametrize("W,E,K,T,H,I,S,fp8,dtype", [
    (4, 16, 3, 60, 256, 128, 64, False, BF16),
    (2, 8, 2, 150, 128, 72, 40, False, F32),
    (4, 16, 4, 90, 256, 256, 64, True, BF16),
    (1, 4, 2, 33, 128, 128, 8, True, F32),
])
def test_layer_step_matches_64_bits(W, E, K, T, H, I, S, fp8, dtype):
    say(f"[layer] W={W} E={E} K={K} T={T} H={H} I={I} fp8={fp8} {dtype}")
    bias = torch.linspace(-0.2, 0.2, E)
    ep, *rest = build(W, E, K, T, H, I, S, fp8, dtype=dtype, bias=bias)
    ep.step()
    torch.cuda.synchronize()
    check(ep, *rest, fp8, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_over_lanes_and_graphs_gives_the_same_bytes(fp8):
    say(f"[layer] lanes and graphs, fp8={fp8}")
    ep, *rest = build(4, 16, 3, 70, 256, 128, 64, fp8, lanes=2)
    ep.step()
    torch.cuda.synchronize()
    check(ep, *rest, fp8)
    want = ep.out.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ep.out.fill_(0)
    ep.step(streams=streams)
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), ep.out.view(torch.int16))
    ep.capture_lane_graphs()
    for _ in range(3):
        ep.out.fill_(0)
        ep.ids.fill_(-5)
        torch.cuda.synchronize()
        ep.step_graphs(streams)
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), ep.out.view(torch.int16))


def test_set_layer_refusals():
    """Without a GPU: the checks come before any buffer is made."""
    ep = object.__new__(LogicalEP)
    ep.E, ep.H, ep.T, ep.W = 8, 64, 4, 2
    ep.quant_group, ep.quant_fp4, ep.row_bytes = None, False, [128]
    w13, w2 = torch.zeros(8, 64, 64), torch.zeros(8, 64, 32)
    for kw, change in ((dict(w13=w13[:4], w2=w2), {}), (dict(w13=w13, w2=w2[:, :32]), {}),
                       (dict(w13=w13[:, :63], w2=w2), {}),
                       (dict(w13=w13, w2=w2, w13_scale=w13), {}),
                       (dict(w13=w13, w2=w2, shared13=w13[0]), {}),
                       (dict(w13=w13, w2=w2), dict(quant_fp4=True)),
                       (dict(w13=w13, w2=w2), dict(quant_group=64)),
                       (dict(w13=w13, w2=w2), dict(quant_group=128)),
                       (dict(w13=w13, w2=w2), dict(row_bytes=[64]))):
        was = {k: getattr(ep, k) for k in change}
        for k, v in change.items():
            setattr(ep, k, v)
        with pytest.raises(ValueError):
            ep.set_layer(**kw)
        for k, v in was.items():
            setattr(ep, k, v)
