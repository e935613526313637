"""GPU: the router's gradient of so many tokens that a wave has several (picks in 8 or 16
lanes each; one a wave for many experts), in every width of its experts, and both
training terms with more sequences than a grid has blocks."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import allowed
from routing import balance64, grad64
from test_gpu_balance import check_grad, grad_inputs, run_grad

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32

WAVES = [
    # T, E, K, S, dtype, grad dtype, masked, through
    (8191, 64, 6, 2, F32, F32, 0.0, "both"),
    (8192, 128, 6, 2, F32, F32, 0.0, "both"),
    (16385, 8, 2, 1, F32, F32, 0.0, "both"),
    (16391, 60, 8, 40, BF16, F32, 0.2, "both"),
    (17001, 64, 9, 3, F32, BF16, 0.0, "both"),
    (17001, 100, 1, 2, F32, F32, 0.1, "both"),
    (16386, 128, 16, 5, BF16, BF16, 0.3, "both"),
    (17003, 256, 8, 7, BF16, BF16, 0.05, "both"),
    (16390, 256, 8, 1, F32, F32, 0.0, "weights"),
    (16401, 256, 12, 9, F32, F32, 0.1, "both"),
    (16400, 256, 6, 4, F32, F32, 0.0, "loss"),
    (16421, 384, 7, 11, F32, F32, 0.1, "both"),
    (16393, 512, 10, 2, BF16, F32, 0.0, "both"),
    (16389, 1000, 8, 3, F32, F32, 0.4, "both"),
    (16387, 1024, 16, 30, F32, BF16, 0.0, "both"),
    (16385, 160, 17, 2, F32, F32, 0.0, "both"),      # too many picks: one token a wave
    (70001, 64, 4, 300, BF16, F32, 0.0, "both"),     # 32 tokens a block and more
]


@pytest.mark.parametrize("T,E,K,S,dtype,gdtype,masked,through", WAVES)
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True),
                                          ("sigmoid", False), ("sigmoid", True)])
def test_several_tokens_of_a_wave(T, E, K, S, dtype, gdtype, masked, through, score, renorm):
    say(f"[route grad] T={T} E={E} K={K} S={S} {score} renorm={renorm} {through}")
    args = grad_inputs(T, E, K, S, score, dtype, masked, through, T + E + K)
    x, ids, gw = args[0], args[1], args[5]
    x[1] = -math.inf
    x[T - 2, : max(1, E // 2)] = float("nan")
    if gw is not None:
        gw[ids < 0] = float("nan")               # what no pick may read into the sums
    check_grad(run_grad(*args, score, renorm, 1.7, gdtype), *args, score, renorm, 1.7)


@pytest.mark.parametrize("K", [4, 11])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True),
                                          ("sigmoid", False), ("sigmoid", True)])
def test_repeated_picks_and_the_gradient_in_place(K, score, renorm):
    say(f"[route grad] repeats, in place K={K} {score} renorm={renorm}")
    T, E = 16400, 96
    x, ids, bounds, _, _, gw, gl = grad_inputs(T, E, K, 5, score, F32, 0.0, "both", K)
    ids[::3, 1] = ids[::3, 0]
    ids[1::5] = ids[1::5, :1]
    ids[2::7, 0] = E                             # no pick
    counts, tokens = (t.int() for t in balance64(x, ids, score, bounds)[:2])
    wide = torch.full((T, 130), float("nan"), device=DEV)
    view = wide[:, 17:17 + E]
    view.copy_(x)
    B.moe_ep_route_backward(view, ids.to(DEV), view, score, renorm, 0.7, gw.to(DEV), gl.to(DEV),
                            counts.to(DEV), tokens.to(DEV),
                            torch.tensor(bounds, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    check_grad(view, x, ids, bounds, counts, tokens, gw, gl, score, renorm, 0.7)
    assert bool(torch.isnan(wide[:, :17]).all()) and bool(torch.isnan(wide[:, 17 + E:]).all())


@pytest.mark.parametrize("T,E", [(100, 4), (300, 65)])
def test_more_sequences_than_blocks(T, E):
    """Past 2^20 sequences (in a block each, or in a block per 64 experts each), almost
    all of them empty: at the first, at the last and around 2^20."""
    S, K = (1 << 20) + 3, 2
    say(f"[balance] S={S} T={T} E={E}")
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, E, generator=g)
    ids = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32)
    full = [0, 7, 1 << 19, (1 << 20) - 1, 1 << 20, (1 << 20) + 2]
    cuts = sorted(torch.randint(1, T, (len(full) - 1,), generator=g).tolist()) + [T]
    start = torch.zeros(S + 1, dtype=torch.int32)
    for s, end in zip(full, cuts):
        start[s + 1:] = end
    start = start.to(DEV)
    bounds = [0] + cuts
    counts = torch.full((S, E), -7, dtype=torch.int32, device=DEV)
    tokens = torch.full((S,), -7, dtype=torch.int32, device=DEV)
    mean = torch.full((S, E), float("nan"), device=DEV)
    loss = torch.full((S,), float("nan"), device=DEV)
    n = B.moe_ep_balance_workspace_bytes(T, E, S)
    ws = torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device=DEV)
    B.moe_ep_balance_loss(x.to(DEV), ids.to(DEV), counts, tokens, mean, loss, ws, "softmax", start)
    gl = torch.rand(S, generator=g) + 0.5
    grad = torch.full((T, E), float("nan"), device=DEV)
    B.moe_ep_route_backward(x.to(DEV), ids.to(DEV), grad, grad_loss=gl.to(DEV), counts=counts,
                            tokens=tokens, seq_start=start)
    torch.cuda.synchronize()
    c, t, m, l, em, el = balance64(x, ids, "softmax", bounds)
    at = torch.tensor(full, device=DEV)
    assert torch.equal(counts[at].cpu().long(), c) and torch.equal(tokens[at].cpu().long(), t)
    assert bool(((mean[at].cpu().double() - m).abs() <= allowed(m, em, F32)).all())
    assert bool(((loss[at].cpu().double() - l).abs() <= allowed(l, el, F32)).all())
    empty = torch.ones(S, dtype=torch.bool, device=DEV)
    empty[at] = False
    assert not any(bool(v[empty].any()) for v in (counts, tokens, mean, loss))
    want, e = grad64(x, ids, "softmax", True, 1.0, None, bounds, c, t, gl[full])
    assert bool(((grad.cpu().double() - want).abs() <= allowed(want, e, F32)).all())
