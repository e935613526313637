"""GPU: the gradient through the weights of a plain softmax (no renormalising)
where its terms cancel: w g - p sum(w g) of tokens whose picks have almost all
of the scores. Bounds are relative to what is left, not to the terms.

With d the error of a softmax's sum relative to it, every score p is off by the
factor 1 +- d and nothing else of its own (the picks' exponentials are fp64), so
an expert's p (G - M), G the gradients of its picks and M = sum p G, is off by
p d (|M| + |G - M|), and by some 2^-46 of p (|G| + sum p |G|) for the fp64
steps. d is what the experts not picked add: u (|x - m| + E / 64 + 24) of their
scores (fp32 exponentials), and 2^-46. The result is rounded to fp32 twice."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import allowed
from routing import U

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32 = torch.float32


def exact(x, ids, scale, gw):
    """(gradient, bound) in float64; the difference G - M is formed from the
    scores of the others, so nothing cancels here either."""
    T, E = x.shape
    x = x.double()
    live = x > -math.inf
    m = torch.where(live, x, -math.inf).amax(dim=1, keepdim=True)
    ex = torch.where(live, torch.exp(x - m), 0.0)
    got = (ids >= 0) & (ids < E)
    at = torch.where(got, ids, 0).long()
    got = got & live.gather(1, at)
    G = torch.zeros(T, E).double().scatter_add(1, at, torch.where(got, gw.double(), 0.0))
    picked = torch.zeros(T, E).double().scatter_add(1, at, got.double()) > 0
    total = ex.sum(dim=1, keepdim=True)
    p = ex / total
    M = (p * G).sum(dim=1, keepdim=True)
    # G_e - M = sum_j p_j (G_e - G_j), G_j = 0 for experts not picked
    diff = torch.zeros(T, E + 1).double()
    for k in range(ids.shape[1]):
        mine = (p * (G.gather(1, at[:, k:k + 1]) - G)).sum(dim=1, keepdim=True)
        diff.scatter_(1, torch.where(got, at, E)[:, k:k + 1], mine)
    diff = diff[:, :E]
    want = scale * p * torch.where(picked, diff, -M.expand(T, E))
    size = torch.where(live, (x - m).abs(), 0.0)
    rest = torch.where(picked, 0.0, ex)
    own = U * (size + E / 64 + 24)
    d = (rest * own).sum(dim=1, keepdim=True) / total + E * 2.0 ** -126 + 2.0 ** -46
    slop = 2.0 ** -46 * ((p * G.abs()).sum(dim=1, keepdim=True) + G.abs())
    e = p * (d * (M.abs() + diff.abs()) + slop)
    e = torch.where(picked, e, p * (d * M.abs() + slop) + (own + 8 * U) * p * M.abs())
    return want, abs(scale) * e + 2 * U * want.abs() + 2.0 ** -120


def run(x, ids, scale, gw):
    grad = torch.full(x.shape, float("nan"), device=DEV)
    B.moe_ep_route_backward(x.to(DEV), ids.to(DEV), grad, "softmax", False, scale, gw.to(DEV))
    torch.cuda.synchronize()
    return grad.cpu()


def check(x, ids, scale, gw):
    want, e = exact(x, ids, scale, gw)
    off, tol = (run(x, ids, scale, gw).double() - want).abs(), allowed(want, e, F32)
    bad = ~(off <= tol)
    at = (off / tol).nan_to_num(9e9).flatten().argmax()
    assert not bool(bad.any()), (int(bad.sum()), float(off.flatten()[at]),
                                 float(want.flatten()[at]), float(tol.flatten()[at]))


# T chooses how many tokens a wave has and in how many lanes its picks lie
@pytest.mark.parametrize("T", [61, 17001])
@pytest.mark.parametrize("E,K", [(8, 1), (64, 2), (256, 8), (160, 12), (513, 3)])
def test_confident_tokens(T, E, K):
    """Gaps of 5 to 35 between the picks' logits and the others'."""
    say(f"[route grad] confident T={T} E={E} K={K}")
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, E, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(97)])
    ids = ids[torch.arange(T) % 97].to(torch.int32)
    gap = 5.0 + 30.0 * torch.rand(T, 1, generator=g)
    near = torch.rand(T, K, generator=g) * torch.tensor([0.0, 0.3, 4.0])[torch.arange(T) % 3, None]
    x.scatter_(1, ids.long(), 3.0 + gap - near)
    gw = torch.randn(T, K, generator=g)
    gw[::4] = gw[::4, :1]                        # picks alike: only the others' share is left
    check(x, ids, 1.7, gw)


@pytest.mark.parametrize("T", [61, 17001])
@pytest.mark.parametrize("E,K", [(8, 2), (256, 8), (160, 12)])
def test_the_same_expert_twice(T, E, K):
    say(f"[route grad] confident, repeats T={T} E={E} K={K}")
    g = torch.Generator().manual_seed(T + E + 1)
    x = torch.randn(T, E, generator=g)
    ids = torch.randint(0, max(2, K // 2), (T, K), generator=g, dtype=torch.int32)
    ids[::5] = ids[::5, :1]                      # one expert for all
    ids[1::7, K - 1] = -1
    ids[2::11] = -1
    x[:, :max(2, K // 2)] += 12.0 + 12.0 * torch.rand(T, 1, generator=g)
    x[3::13, 0] = -math.inf
    gw = torch.randn(T, K, generator=g)
    gw[ids < 0] = float("nan")
    check(x, ids, -0.6, gw)


@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 17.0, 20.0, 25.0])
def test_one_pick_far_above_the_others(gap):
    """One pick, 8 experts: p (1 - p) g, which fp32 differences have to a few
    parts in ten at a gap of 17."""
    say(f"[route grad] gap {gap}")
    x = torch.zeros(3, 8)
    x[:, 2] = gap
    ids = torch.full((3, 1), 2, dtype=torch.int32)
    gw = torch.tensor([[1.0], [-0.7], [3.3]])
    got = run(x, ids, 1.0, gw)[:, 2].double()
    rest = 7.0 * math.exp(-gap)
    want = gw[:, 0].double() * rest / (1.0 + rest) ** 2
    # the exponential's argument and two places of its own, the sum, 2^-46 of p in fp64
    assert bool(((got - want).abs() <= want.abs() * U * (gap + 30) + 2.0 ** -46).all()), (got, want)
