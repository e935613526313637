"""GPU: the balance loss of many tokens. A wave adds at most 256 tokens' scores
in fp32, a block its 16 waves' and fp64 takes over from there, so a mean score is
off by (256 + 24) roundings and its scores' own errors, however many tokens."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from routing import U

pytestmark = pytest.mark.gpu

DEV = "cuda"
ADDS = 280 * 2.0 ** -24


def run(x, ids, score, start, S):
    T, E = x.shape
    counts = torch.full((S, E), -7, dtype=torch.int32, device=DEV)
    tokens = torch.full((S,), -7, dtype=torch.int32, device=DEV)
    mean = torch.full((S, E), float("nan"), device=DEV)
    loss = torch.full((S,), float("nan"), device=DEV)
    ws = torch.full((B.moe_ep_balance_workspace_bytes(T, E, S),), 0xFF, dtype=torch.uint8,
                    device=DEV)
    B.moe_ep_balance_loss(x, ids, counts, tokens, mean, loss, ws, score, start)
    torch.cuda.synchronize()
    return counts, tokens, mean, loss


def test_scores_that_round_the_same_way():
    """2^26 tokens alike: sums that fp32 would carry from token to token drift by
    2e-4."""
    T, E = 1 << 26, 4
    say(f"[balance] {T} tokens alike")
    row = torch.tensor([0.0, 1.0, 2.0, 3.0])
    x = row.to(torch.bfloat16).to(DEV).repeat(T, 1)
    ids = torch.full((T, 1), 3, dtype=torch.int32, device=DEV)
    counts, tokens, mean, loss = run(x, ids, "softmax", None, 1)
    q = torch.softmax(row.double(), dim=0)
    assert counts.tolist() == [[0, 0, 0, T]] and tokens.tolist() == [T]
    # an exponential of 3 and its sum, as tests/routing.py has them
    tol = ADDS + U * (3 + 3 + 24)
    assert bool(((mean[0].cpu().double() - q).abs() <= tol * q).all()), mean[0].cpu().double() / q - 1
    assert abs(float(loss) - 4 * float(q[3])) <= (tol + U) * 4 * float(q[3])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_more_tiles_than_blocks_and_ragged_sequences(score):
    T, E, K = (1 << 22) + 77, 8, 2
    say(f"[balance] {T} tokens {score}")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((T, E), generator=g, device=DEV)
    ids = torch.randint(-1, E, (T, K), generator=g, device=DEV, dtype=torch.int32)
    bounds = [5, 1_000_003, 1_000_003, 1_000_090, T - 9]
    S = len(bounds) - 1
    start = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    counts, tokens, mean, loss = run(x, ids, score, start, S)
    p = torch.softmax(x.double(), dim=1) if score == "softmax" else torch.sigmoid(x.double())
    q = p / p.sum(dim=1, keepdim=True)
    real = (ids >= 0).any(dim=1)
    for s in range(S):
        at = slice(bounds[s], bounds[s + 1])
        mine = ids[at][ids[at] >= 0].long()
        want = torch.bincount(mine, minlength=E)
        n = int(real[at].sum())
        assert torch.equal(counts[s].long(), want) and int(tokens[s]) == n
        m = (q[at] * real[at][:, None]).sum(dim=0) / max(1, n)
        tol = ADDS + U * (2 * 12 + 24)           # logits of at most 6
        assert bool(((mean[s].double() - m).abs() <= tol * m).all())
        full = E * float((want.double() / max(1, int(want.sum())) * m).sum())
        assert abs(float(loss[s]) - full) <= (tol + U) * full
