"""A layer with 4-bit experts and a router in training, as LogicalEP.step() runs
it: its outputs against their 64-bit evaluation token by token, the balance
terms of each rank and the router's gradient; eager, over lanes and as replayed
graphs. The refusals of set_layer run without a GPU."""
import pytest
import torch

import workloads as wl
from combine_topk_ids_dest_amd.emulate import LogicalEP
from products import U, allowed, product64, route64
from routing import balance64, grad64
from w4 import pitch, random_w4, value64

BF16, F32 = torch.bfloat16, torch.float32
H8 = 2.0 ** -8                  # half a step of bf16, relative
ROUTE = dict(score="sigmoid", n_group=4, topk_group=3, renormalize=True, scale=1.5)


def weights(E, H, I, group, seed=1):
    g = torch.Generator().manual_seed(seed)
    w13, s13 = random_w4((E,), 2 * I, H, group, g)
    w2, s2 = random_w4((E,), H, I, group, g)
    f13, f2 = torch.rand(E, 2, generator=g) + 0.5, torch.rand(E, 1, generator=g) + 0.5
    d = dict(w13=w13, w2=w2, w13_scale=s13, w2_scale=s2, w13_global=f13, w2_global=f2,
             gate=(torch.randn(E, H, generator=g) / H ** 0.5).to(BF16))
    full13 = value64(w13, s13, group) * f13.double().repeat_interleave(I, 1)[:, :, None]
    return d, full13, value64(w2, s2, group) * f2.double()[:, :, None]


def build(W, E, K, T, H, I, group, lanes=1, device="cuda"):
    w = wl.WORKLOADS[1].scaled(W=W, E=E, K=K, T=T, cap=T, H=H, pad_frac=0.0)
    ep = LogicalEP(T, H, E, K, W, T, [2 * H], BF16, device, lanes=lanes)
    xs = [wl.hidden_bf16(w, s, 3) for s in range(W)]
    for s in range(W):
        ids, wts = wl.routing(w, s, 3)
        ep.set_source(s, ids, wts, [xs[s].view("uint8").reshape(T, 2 * H)])
    d, f13, f2 = weights(E, H, I, group)
    ep.set_layer(route=ROUTE, w4_group=group, balance=True,
                 **{k: v.to(device) for k, v in d.items()})
    return ep, xs, f13, f2


def check(ep, xs, f13, f2):
    W, E, K, T, H = ep.W, ep.E, ep.K, ep.T, ep.H
    assert int(ep.err.item()) == 0
    for s in range(W):
        x = torch.from_numpy(wl.bf16_bits_to_f32(xs[s])).double()
        logits = ep._layer["logits"][s].cpu()
        ids, wts = route64(logits, None, K, **ROUTE)
        assert torch.equal(ep.ids[s].cpu(), ids)
        per_dest, dest_err = torch.zeros(W, T, H).double(), torch.zeros(W, T, H).double()
        for e in range(E):
            hit = (ids == e).any(dim=1)
            if not bool(hit.any()):
                continue
            h, eh = product64(x[hit], f13[e], None, "silu_gated", f13.shape[1] // 2, extra=2)
            eh = eh + (h.abs() + eh) * H8                # rows between the products
            y = h @ f2[e].t()
            ey = eh @ f2[e].abs().t() + (h.shape[1] + 2) * U * ((h.abs() + eh) @ f2[e].abs().t())
            ey = ey + (y.abs() + ey) * H8
            wt = (wts * (ids == e)).sum(dim=1)[hit, None]
            r = e // ep.e_local
            per_dest[r, hit] += wt * y
            dest_err[r, hit] += wt * (ey + 4 * U * y.abs())
        dest_err += (per_dest.abs() + dest_err) * H8
        out, err = per_dest.sum(0), dest_err.sum(0)
        err = err + (W + 1) * U * per_dest.abs().sum(0) + (out.abs() + err) * H8
        off = (ep.out[s].double().cpu() - out).abs()
        assert bool((off <= err).all()), (s, float((off / err).max()))
        t = {k: v.cpu() for k, v in ep.balance_terms(s).items()}
        counts, tokens, mean, loss, emean, eloss = balance64(logits, ids, "sigmoid", [0, T])
        assert torch.equal(t["counts"].long(), counts) and torch.equal(t["tokens"].long(), tokens)
        assert bool(((t["mean_score"].double() - mean).abs() <= allowed(mean, emean, F32)).all())
        assert bool(((t["loss"].double() - loss).abs() <= allowed(loss, eloss, F32)).all())
        g = torch.Generator().manual_seed(s)
        gw, gl = torch.randn(T, K, generator=g), torch.tensor([0.3])
        grad = torch.empty(T, E, device=ep.device)
        ep.router_grad(s, grad, gw.to(ep.device), gl.to(ep.device))
        torch.cuda.synchronize()
        want, e = grad64(logits, ids, "sigmoid", True, 1.5, gw, [0, T], counts, tokens, gl)
        assert bool(((grad.cpu().double() - want).abs() <= allowed(want, e, F32)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("group,W,E,K,T,H,I", [(16, 4, 16, 3, 60, 256, 96), (32, 2, 8, 2, 300, 128, 160)])
def test_step_with_4_bit_experts_and_balance(group, W, E, K, T, H, I):
    ep, *rest = build(W, E, K, T, H, I, group)
    ep.step()
    torch.cuda.synchronize()
    check(ep, *rest)
    assert ep._layer["w13_scale"].shape[-1] == pitch(H, group)


@pytest.mark.gpu
def test_lanes_and_graphs_give_the_same_layer():
    ep, *rest = build(4, 16, 3, 70, 256, 96, 16, lanes=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ep.step(streams=streams)
    torch.cuda.synchronize()
    check(ep, *rest)
    eager = ep.out.clone()
    ep.capture_lane_graphs()
    for _ in range(3):
        ep.out.fill_(0)
        for v in ep._layer["balance"].values():
            v.fill_(0)
        torch.cuda.synchronize()
        ep.step_graphs(streams)
        torch.cuda.synchronize()
        assert torch.equal(ep.out, eager)
        check(ep, *rest)


def test_set_layer_refuses_what_does_not_fit():
    E, H, I = 8, 64, 32
    ep = lambda **kw: LogicalEP(T=4, H=H, E=E, K=2, W=2, cap=4, row_bytes=[2 * H], device="cpu", **kw)
    d, _, _ = weights(E, H, I, 16)
    ok = dict(d, w4_group=16)
    ep().set_layer(**ok)
    ep().set_layer(**ok, balance=True)
    bad = [
        dict(ok, w4_group=8), dict(ok, w4_group=None), dict(ok, w13_scale=None),
        dict(ok, w2_scale=None), dict(ok, w2_scale=d["w2_scale"][:, :, :8]),
        dict(ok, w13=d["w13"][:, :, :16]), dict(ok, w2=d["w2"][:, :32]),
        dict(ok, w13_global=d["w2_global"]), dict(ok, w2_global=d["w13_global"]),
        dict(ok, gate=None, balance=True),
        dict(w13=torch.zeros(E, 2 * I, H).to(BF16), w2=torch.zeros(E, H, I).to(BF16),
             w13_global=d["w13_global"]),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            ep().set_layer(**kw)
            pytest.fail(str({k for k in kw}))
    with pytest.raises(ValueError, match="bf16 rows"):
        q = LogicalEP(T=4, H=128, E=E, K=2, W=2, cap=4, row_bytes=[256], device="cpu",
                      quant_group=128)
        q.set_layer(**dict(weights(E, 128, I, 16)[0], w4_group=16))
    e = ep()
    e.set_layer(**ok)
    with pytest.raises(ValueError, match="balance"):
        e.balance_terms(0)
    with pytest.raises(ValueError, match="balance"):
        e.router_grad(0, torch.zeros(4, E), grad_loss=torch.zeros(1))
    with pytest.raises(ValueError, match="router"):
        ep().router_grad(0, torch.zeros(4, E))
