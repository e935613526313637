"""GPU: a router's training terms (counts, mean scores, balance loss, the
logits' gradient) against their plain 64-bit forms, autograd and differences."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import allowed
from routing import U, balance64, definition64, grad64

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(T, E, K, dtype, masked, g, padding=0.1):
    x = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = -math.inf
    x = x.to(dtype)
    top = x.float().topk(K, dim=1)
    ids = torch.where(top.values > -math.inf, top.indices, -1).to(torch.int32)
    ids[torch.rand(T, generator=g) < padding] = -1
    return x, ids


def cut(T, S, seed):
    """Ragged sequences in [0, T]: empty ones, tokens before the first and
    behind the last."""
    if S == 1:
        return [0, T]
    r = torch.randint(0, T + 1, (S + 1,), generator=gen(seed)).tolist()
    return sorted(r)


def balance(x, ids, score, bounds, stream=None, ws=None):
    """The four outputs, in buffers of marks."""
    T, E = x.shape
    S = len(bounds) - 1
    start = None if bounds == [0, T] else torch.tensor(bounds, dtype=torch.int32, device=DEV)
    counts = torch.full((S, E), -7, dtype=torch.int32, device=DEV)
    tokens = torch.full((S,), -7, dtype=torch.int32, device=DEV)
    mean = torch.full((S, E), float("nan"), device=DEV)
    loss = torch.full((S,), float("nan"), device=DEV)
    n = B.moe_ep_balance_workspace_bytes(T, E, S)
    if ws is None:
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if n else None
    B.moe_ep_balance_loss(x, ids, counts, tokens, mean, loss, ws, score, start, stream)
    return counts, tokens, mean, loss


def check_balance(x, ids, score, bounds, got):
    counts, tokens, mean, loss, emean, eloss = balance64(x, ids, score, bounds)
    gc, gt, gm, gl = (t.cpu() for t in got)
    assert torch.equal(gc.long(), counts) and torch.equal(gt.long(), tokens)
    for have, want, e in ((gm, mean, emean), (gl, loss, eloss)):
        off, tol = (have.double() - want).abs(), allowed(want, e, F32)
        assert bool((off <= tol).all()), float((off / tol).max())


BALANCE = [
    # T, E, K, S, score, dtype, masked
    (1, 1, 1, 1, "softmax", F32, 0.0),
    (1, 256, 8, 1, "sigmoid", F32, 0.0),
    (2, 8, 2, 5, "softmax", BF16, 0.0),
    (63, 60, 4, 3, "sigmoid", BF16, 0.3),
    (128, 256, 8, 1, "sigmoid", F32, 0.0),
    (255, 65, 6, 4, "softmax", F32, 0.5),
    (256, 160, 6, 300, "softmax", F32, 0.1),
    (257, 256, 8, 1, "softmax", F32, 0.05),
    (300, 512, 10, 7, "sigmoid", BF16, 0.2),
    (1000, 1000, 64, 3, "softmax", BF16, 0.1),
    (1111, 1024, 16, 40, "sigmoid", F32, 0.3),
    (2047, 384, 7, 1, "sigmoid", BF16, 0.0),
    (3000, 128, 2, 2000, "softmax", F32, 0.0),
    (9001, 64, 1, 6, "softmax", BF16, 0.02),
    (20000, 16, 4, 1, "sigmoid", F32, 0.0),
]


@pytest.mark.parametrize("T,E,K,S,score,dtype,masked", BALANCE)
def test_balance_matches_64_bits(T, E, K, S, score, dtype, masked):
    say(f"[balance] T={T} E={E} K={K} S={S} {score} {dtype} masked={masked}")
    x, ids = inputs(T, E, K, dtype, masked, gen(T + E))
    if T > 2:
        x[1] = -math.inf                         # picks of an expert with no score
        x[2, : max(1, E // 2)] = float("nan")
    bounds = cut(T, S, T)
    got = balance(x.to(DEV), ids.to(DEV), score, bounds)
    torch.cuda.synchronize()
    check_balance(x, ids, score, bounds, got)


def test_balance_extremes():
    """Infinities, far logits, one expert for all, ids that are no picks, no
    tokens at all."""
    say("[balance] extremes")
    E, K = 96, 4
    x = torch.zeros(9, E)
    x[1, 5] = math.inf
    x[2, 7] = x[2, 90] = math.inf
    x[3] = -3.0e38
    x[4, 1:] = -1000.0
    x[5] = torch.linspace(-800, 800, E)
    x[6] = -500.0 + torch.arange(E) / 8
    x[7] = float("nan")
    ids = torch.tensor([[0, 0, 0, 0]] * 8 + [[E, -5, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        for bounds in ([0, 9], [0, 4, 4, 9], [8, 9], [0, 0, 9, 9]):
            check_balance(x, ids, score, bounds, balance(x.to(DEV), ids.to(DEV), score, bounds))
    none = balance(torch.zeros(0, E, device=DEV), torch.zeros(0, K, dtype=torch.int32, device=DEV),
                   "softmax", [0, 0])
    torch.cuda.synchronize()
    assert all(bool((t == 0).all()) for t in none)


def test_balance_even_and_one_sided():
    """1 where all experts are picked alike and score alike; E where one
    expert has everything."""
    say("[balance] even, one-sided")
    T, E, K = 640, 32, 2
    ids = (torch.arange(T * K, dtype=torch.int32) % E).view(T, K)
    _, _, _, loss = balance(torch.zeros(T, E, device=DEV), ids.to(DEV), "softmax", [0, T])
    one = torch.full((T, E), -math.inf)
    one[:, 3] = 0.0
    _, _, mean, most = balance(one.to(DEV), torch.full((T, 1), 3, dtype=torch.int32, device=DEV),
                               "softmax", [0, T])
    torch.cuda.synchronize()
    assert abs(float(loss) - 1.0) <= 64 * U and float(most) == E and float(mean[0, 3]) == 1.0


def test_seq_start_is_clamped():
    say("[balance] clamped bounds")
    T, E, K = 400, 64, 4
    x, ids = inputs(T, E, K, F32, 0.0, gen(4))
    wild = balance(x.to(DEV), ids.to(DEV), "softmax", [-9, 100, 100, 2 ** 31 - 1])
    torch.cuda.synchronize()
    check_balance(x, ids, "softmax", [0, 100, 100, T], wild)
    grad = torch.empty(T, E, device=DEV)
    gl = torch.tensor([1.0, -2.0, 0.5])
    B.moe_ep_route_backward(x.to(DEV), ids.to(DEV), grad, grad_loss=gl.to(DEV), counts=wild[0],
                            tokens=wild[1],
                            seq_start=torch.tensor([-9, 100, 100, 2 ** 31 - 1], dtype=torch.int32,
                                                   device=DEV))
    torch.cuda.synchronize()
    want, e = grad64(x, ids, "softmax", True, 1.0, None, [0, 100, 100, T], wild[0].cpu(),
                     wild[1].cpu(), gl)
    assert bool(((grad.cpu().double() - want).abs() <= allowed(want, e, F32)).all())


GRAD = [
    # T, E, K, S, score, renormalize, dtype, grad dtype, masked, through
    (1, 1, 1, 1, "softmax", True, F32, F32, 0.0, "both"),
    (1, 256, 8, 1, "sigmoid", True, F32, F32, 0.0, "both"),
    (5, 8, 2, 2, "softmax", False, BF16, F32, 0.3, "both"),
    (64, 60, 60, 3, "softmax", True, F32, BF16, 0.1, "weights"),
    (128, 256, 8, 1, "sigmoid", False, F32, F32, 0.0, "weights"),
    (129, 256, 8, 1, "softmax", False, BF16, BF16, 0.05, "both"),
    (500, 160, 6, 9, "sigmoid", True, BF16, BF16, 0.3, "both"),
    (777, 1024, 64, 4, "softmax", False, F32, F32, 0.2, "both"),
    (1000, 513, 10, 500, "sigmoid", True, F32, F32, 0.5, "loss"),
    (4099, 128, 4, 3, "softmax", True, F32, F32, 0.0, "both"),
    (9001, 65, 1, 1, "softmax", False, F32, BF16, 0.0, "loss"),
    (20000, 16, 3, 30, "sigmoid", False, BF16, F32, 0.1, "both"),
]


def grad_inputs(T, E, K, S, score, dtype, masked, through, seed):
    g = gen(seed)
    x, ids = inputs(T, E, K, dtype, masked, g)
    bounds = cut(T, S, seed + 1)
    counts, tokens = balance64(x, ids, score, bounds)[:2]
    gw = torch.randn(T, K, generator=g) if through != "loss" else None
    gl = (torch.rand(S, generator=g) + 0.5) * T ** 0.5 if through != "weights" else None
    return x, ids, bounds, counts.int(), tokens.int(), gw, gl


def run_grad(x, ids, bounds, counts, tokens, gw, gl, score, renorm, scale, out_dtype, stream=None):
    T, E = x.shape
    grad = torch.full((T, E), float("nan"), dtype=out_dtype, device=DEV)
    kw = {}
    if gl is not None:
        kw = dict(grad_loss=gl.to(DEV), counts=counts.to(DEV), tokens=tokens.to(DEV),
                  seq_start=None if bounds == [0, T] else
                  torch.tensor(bounds, dtype=torch.int32, device=DEV))
    B.moe_ep_route_backward(x.to(DEV), ids.to(DEV), grad, score, renorm, scale,
                            None if gw is None else gw.to(DEV), stream=stream, **kw)
    torch.cuda.synchronize()
    return grad


def check_grad(grad, x, ids, bounds, counts, tokens, gw, gl, score, renorm, scale):
    want, e = grad64(x, ids, score, renorm, scale, gw, bounds, counts, tokens, gl)
    off, tol = (grad.cpu().double() - want).abs(), allowed(want, e, grad.dtype)
    assert bool((off <= tol).all()), float((off / tol).nan_to_num(9e9).max())


@pytest.mark.parametrize("T,E,K,S,score,renorm,dtype,gdtype,masked,through", GRAD)
def test_route_backward_matches_64_bits(T, E, K, S, score, renorm, dtype, gdtype, masked, through):
    say(f"[route grad] T={T} E={E} K={K} S={S} {score} renorm={renorm} {dtype} {gdtype} {through}")
    args = grad_inputs(T, E, K, S, score, dtype, masked, through, T + E)
    x = args[0]
    if T > 4:
        x[1] = -math.inf
        x[2, : max(1, E // 2)] = float("nan")
        if args[5] is not None:
            args[5][args[1] < 0] = float("nan")          # what no pick may read into the sums
    grad = run_grad(*args, score, renorm, 1.7, gdtype)
    check_grad(grad, *args, score, renorm, 1.7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_extremes_and_repeats(score, renorm):
    """Infinities, far logits, the same expert picked twice, ids that are no
    picks, a scale of 0 and a negative one."""
    say(f"[route grad] extremes {score} renorm={renorm}")
    E, K = 96, 4
    x = torch.zeros(9, E)
    x[1, 5] = math.inf
    x[2, 7] = x[2, 90] = math.inf
    x[3] = -3.0e38
    x[4, 1:] = -700.0
    x[5] = torch.linspace(-30, 30, E)
    x[6] = -500.0 + torch.arange(E) / 8
    ids = torch.tensor([[0, 0, 1, 0], [5, 6, 5, 7], [7, 90, 1, -1], [3, 4, 5, 6], [0, 1, 2, 3],
                        [95, 94, 0, 95], [95, 94, 93, 0], [1, 2, 1, 2],
                        [E, -5, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    gw = torch.randn(9, K, generator=gen(1))
    gl = torch.tensor([3.0])
    counts, tokens = (t.int() for t in balance64(x, ids, score, [0, 9])[:2])
    for scale in (1.0, 0.0, -2.5):
        args = (x, ids, [0, 9], counts, tokens, gw, gl)
        check_grad(run_grad(*args, score, renorm, scale, F32), *args, score, renorm, scale)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
def test_route_backward_against_autograd_and_differences(score, renorm):
    say(f"[route grad] autograd, differences {score} renorm={renorm}")
    T, E, K, S = 40, 48, 5, 3
    x, ids, bounds, counts, tokens, gw, gl = grad_inputs(T, E, K, S, score, F32, 0.0, "both", 77)
    ids[3, 1] = ids[3, 0]
    counts, tokens = (t.int() for t in balance64(x, ids, score, bounds)[:2])
    grad = run_grad(x, ids, bounds, counts, tokens, gw, gl, score, renorm, 1.3, F32).cpu().double()
    f = lambda v: definition64(v, ids, score, renorm, 1.3, gw, bounds, counts, tokens, gl)
    v = x.double().requires_grad_(True)
    f(v).backward()
    _, e = grad64(x, ids, score, renorm, 1.3, gw, bounds, counts, tokens, gl)
    assert bool(((grad - v.grad).abs() <= allowed(v.grad, e, F32) + 1e-12).all())
    h = 1e-5
    for t, k in ((0, 0), (3, 1), (17, 2), (39, 4)):
        for col in (int(ids[t, k]) if ids[t, k] >= 0 else 0, (t * 7) % E):
            up, down = x.double().clone(), x.double().clone()
            up[t, col] += h
            down[t, col] -= h
            slope = float(f(up) - f(down)) / (2 * h)
            # h^2 times a third derivative of order one, and 1e-16 / h of rounding
            assert abs(slope - float(grad[t, col])) <= 1e-8 + float(allowed(
                grad[t, col], e[t, col], F32))


def test_strided_logits_in_place_gradient_and_other_columns():
    """Logits as columns of a wider product; the gradient in their place."""
    say("[route grad] strided, in place")
    T, E, K = 70, 72, 4
    x, ids, bounds, counts, tokens, gw, gl = grad_inputs(T, E, K, 1, "softmax", BF16, 0.0, "both", 5)
    wide = torch.full((T, 130), float("nan"), dtype=BF16, device=DEV)
    wide[:, 33:33 + E] = x.to(DEV)
    view = wide[:, 33:33 + E]
    got = balance(view, ids.to(DEV), "softmax", bounds)
    torch.cuda.synchronize()
    check_balance(x, ids, "softmax", bounds, got)
    B.moe_ep_route_backward(view, ids.to(DEV), view, grad_weights=gw.to(DEV),
                            grad_loss=gl.to(DEV), counts=got[0], tokens=got[1])
    torch.cuda.synchronize()
    check_grad(view, x, ids, bounds, counts, tokens, gw, gl, "softmax", True, 1.0)
    assert bool(torch.isnan(wide[:, :33]).all()) and bool(torch.isnan(wide[:, 33 + E:]).all())


@pytest.mark.parametrize("T,S", [(100, 3), (5000, 6)])
def test_balance_streams_graphs_and_two_at_once(T, S):
    """The eager bytes from another stream, from replays of a graph (on new
    logits too), and from two calls at once with workspaces of their own."""
    say(f"[balance] graph and streams T={T}")
    E, K = 256, 8
    sets = []
    for seed in (1, 2):
        x, ids, bounds, _, _, gw, gl = grad_inputs(T, E, K, S, "sigmoid", F32, 0.0, "both", seed)
        d = dict(x=x.to(DEV), ids=ids.to(DEV), gw=gw.to(DEV), gl=gl.to(DEV),
                 start=torch.tensor(bounds, dtype=torch.int32, device=DEV),
                 counts=torch.zeros(S, E, dtype=torch.int32, device=DEV),
                 tokens=torch.zeros(S, dtype=torch.int32, device=DEV),
                 mean=torch.zeros(S, E, device=DEV), loss=torch.zeros(S, device=DEV),
                 grad=torch.zeros(T, E, device=DEV),
                 ws=torch.empty(max(16, B.moe_ep_balance_workspace_bytes(T, E, S)),
                                dtype=torch.uint8, device=DEV))
        sets.append(d)

    def go(d, stream=None):
        B.moe_ep_balance_loss(d["x"], d["ids"], d["counts"], d["tokens"], d["mean"], d["loss"],
                              d["ws"], "sigmoid", d["start"], stream)
        B.moe_ep_route_backward(d["x"], d["ids"], d["grad"], "sigmoid", True, 2.0, d["gw"],
                                d["gl"], d["counts"], d["tokens"], d["start"], stream)

    names = ("counts", "tokens", "mean", "loss", "grad")
    take = lambda d: [d[n].clone() for n in names]
    same = lambda a, d: all(torch.equal(u, d[n]) for u, n in zip(a, names))
    eager = []
    for d in sets:
        go(d)
        torch.cuda.synchronize()
        eager.append(take(d))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for d, st in zip(sets, streams):
            go(d, st)
        torch.cuda.synchronize()
        assert all(same(a, d) for a, d in zip(eager, sets))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(sets[0])
    kept = sets[0]["x"].clone()
    for rep in range(4):
        sets[0]["x"].copy_(kept if rep % 2 == 0 else sets[1]["x"])
        for n in names:
            sets[0][n].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        if rep % 2 == 0:
            assert same(eager[0], sets[0]), rep
        else:
            assert torch.equal(sets[0]["counts"], eager[0][0])        # the same ids
            assert not torch.equal(sets[0]["loss"], eager[0][3])


def test_common_counts_of_several_ranks():
    """Ranks that sum their counts before the backward pass get the gradient of
    the loss with the common counts and their own mean scores."""
    say("[balance] common counts")
    T, E, K = 90, 64, 4
    g = gen(12)
    ranks = [inputs(T, E, K, F32, 0.0, g) for _ in range(2)]
    outs = [balance(x.to(DEV), ids.to(DEV), "softmax", [0, T]) for x, ids in ranks]
    common = outs[0][0] + outs[1][0]
    gl = torch.tensor([0.7])
    for (x, ids), o in zip(ranks, outs):
        grad = torch.empty(T, E, device=DEV)
        B.moe_ep_route_backward(x.to(DEV), ids.to(DEV), grad, grad_loss=gl.to(DEV), counts=common,
                                tokens=o[1])
        torch.cuda.synchronize()
        check_grad(grad, x, ids, [0, T], common.cpu(), o[1].cpu(), None, gl, "softmax", True, 1.0)


@pytest.mark.parametrize("T", [100, 200, 70000])
def test_more_sequences_than_a_grid_has_rows(T):
    """Sequences of one token each, most of them empty or not, past 2^16 of
    them."""
    S, E, K = 66000, 8, 2
    say(f"[balance] S={S} T={T}")
    x, ids = inputs(T, E, K, F32, 0.0, gen(T))
    bounds = [min(T, i) for i in range(S + 1)]
    got = balance(x.to(DEV), ids.to(DEV), "softmax", bounds)
    torch.cuda.synchronize()
    n = min(S, T)
    picked = torch.zeros(S, E, dtype=torch.int32)
    for k in range(K):
        real = ids[:n, k] >= 0
        picked[:n][real, ids[:n, k][real].long()] += 1
    assert torch.equal(got[0].cpu(), picked)
    real = (ids[:n] >= 0).any(dim=1)
    assert torch.equal(got[1].cpu()[:n], real.int()) and not bool(got[1][n:].any())
    q = torch.softmax(x[:n].double(), dim=1) * real[:, None]
    # one token: its scores, the largest off by their sum's and exponentials' places
    assert bool(((got[2].cpu()[:n].double() - q).abs() <= 64 * U * q).all())
    loss = E * (picked[:n].double() / K * q).sum(dim=1)
    assert bool(((got[3].cpu()[:n].double() - loss).abs() <= 64 * U * loss).all())
    assert not bool(got[2][n:].any()) and not bool(got[3][n:].any())
