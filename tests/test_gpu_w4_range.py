"""GPU: rows of x near both ends of bf16's range. Wherever no sum of products of
x with the weights leaves fp32's range, no result does, whichever tiles the rows
get and whatever the bare codes' sums would be."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import assert_close, product64
from w4 import pitch, random_w4, value64

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16
TOP = 3.3895313892515355e38                      # the largest bf16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def small_scales(N, H, group, g):
    """Codes of all kinds under scales of 2^-9 and 2^-8."""
    w, s = random_w4((), N, H, group, g)
    n = H // group
    if group == 16:
        s[:, :n] = torch.randint(1, 3, (N, n), generator=g, dtype=torch.uint8)
    else:
        s[:, :n] = torch.randint(127 - 9, 127 - 7, (N, n), generator=g, dtype=torch.uint8)
    return w, s


@pytest.mark.parametrize("group", [16, 32])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 13, 40, 150])
def test_large_rows_under_small_scales(T, group):
    say(f"[w4 range] large rows, T={T} /{group}")
    H, N = 288, 72
    g = gen(T + group)
    w, s = small_scales(N, H, group, g)
    w64 = value64(w, s, group)
    # one large value; all of them large, sums of either sign within range; and
    # a single one of the largest
    one = torch.zeros(H)
    one[41] = 1.0e38
    all_ = (torch.randint(0, 2, (H,), generator=g) * 2 - 1) * \
        (0.9 * TOP / w64.abs().sum(dim=1).max()).float().clamp(max=0.9 * TOP)
    last = torch.zeros(H)
    last[H - 1] = TOP
    x = torch.stack([(one, all_, last)[(t + T) % 3] for t in range(T)]).to(BF16)
    want, e = product64(x.double(), w64, None, "none", N)
    assert float((x.double().abs() @ w64.abs().t()).max()) < 3.1e38         # so no partial sum is past the range
    o = torch.full((T, N), 7.0, device=DEV)
    B.moe_ep_matmul_w4(x.to(DEV), w.to(DEV), s.to(DEV), o, group)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(o).all()), "a sum of bare codes left the range"
    assert_close(o, want, e, (T, group))


@pytest.mark.parametrize("group", [16, 32])
@pytest.mark.parametrize("T", [1, 3, 4, 5, 13, 40, 150])
def test_tiny_values_under_large_scales(T, group):
    """One value in a row, so that each output is a weight times a power of two,
    exactly, from x's smallest numbers on."""
    say(f"[w4 range] tiny values, T={T} /{group}")
    H, N = 288, 72
    g = gen(T * 3 + group)
    w, s = random_w4((), N, H, group, g)
    s[:, :H // group] = 0x7E if group == 16 else 127 + 9         # 448, 512
    w64 = value64(w, s, group)
    for low in (-133, -126, -119, -112):
        x = torch.zeros(T, H)
        at = torch.randint(0, H, (T,), generator=g)
        x[torch.arange(T), at] = torch.tensor([2.0 ** (low + t % 7) for t in range(T)])
        x = x.to(BF16)
        want = x.double() @ w64.t()
        o = torch.full((T, N), 7.0, device=DEV)
        B.moe_ep_matmul_w4(x.to(DEV), w.to(DEV), s.to(DEV), o, group)
        torch.cuda.synchronize()
        assert bool((o.cpu().double() == want).all()), (low, T)


@pytest.mark.parametrize("T", [1, 3, 4, 16])
def test_scales_of_one_group_with_large_rows(T):
    """Every E4M3 scale with the largest x that it leaves in range."""
    say(f"[w4 range] each scale, T={T}")
    H, N = 64, 256
    w = torch.full((N, H // 2), 0x77, dtype=torch.uint8)   # codes of 6
    s = torch.zeros((N, pitch(H, 16)), dtype=torch.uint8)
    s[:, 1] = torch.arange(N, dtype=torch.int32).to(torch.uint8)
    w64 = value64(w, s, 16)
    fine = ~torch.isnan(w64).any(dim=1)
    size = w64[:, 16].abs()
    for k in (16, 31):
        big = torch.where(size > 0, 0.9 * TOP / size, TOP).clamp(max=TOP)
        for n in range(0, N, 37):
            if not bool(fine[n]):
                continue
            x = torch.zeros(T, H)
            x[:, k] = float(big[n])
            x = x.to(BF16)
            o = torch.full((T, N), 7.0, device=DEV)
            B.moe_ep_matmul_w4(x.to(DEV), w.to(DEV), s.to(DEV), o, 16)
            torch.cuda.synchronize()
            want = x.double() @ torch.where(fine[:, None], w64, 0.0).t()
            have = o.cpu().double()[:, n]
            assert bool((have == want[:, n].float().double()).all()), (k, n, T)
