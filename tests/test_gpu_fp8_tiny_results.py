"""GPU: fp8 products whose results are so small that amax / 448 rounds to zero
in fp32, or to a number that leaves amax past the largest code: the scale is then
the number above, and the codes stand for the results. All results here are
whole multiples of 2^-149, and nothing but the scale and the codes is rounded."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say

F8 = torch.float8_e4m3fn
TINY = 2.0 ** -149


@pytest.mark.gpu
@pytest.mark.parametrize("counts,rows", [([5], 16), ([40, 0, 7], 64), ([300, 130], 304)])
@pytest.mark.parametrize("top,steps", [
    (96, 1),        # 0.2 steps of 2^-149: rounded, the scale would be 0
    (544, 2),       # 1.2: one step would leave 544
    (656, 2),       # 1.46: one would leave 656
    (1000, 3),      # 2.2: two would leave 500
    (1120, 3),      # 2.5: two (to even) would leave 560
    (6496, 15),     # 14.5: fourteen (to even) would leave 464, a tie
    (6720, 15),     # 15
])
def test_tiny_results_keep_finite_codes(counts, rows, top, steps):
    """The largest result of the first 128 columns is `top`; those of the second
    are zero."""
    say(f"[fp8 tiny] counts={counts} top={top}")
    H, N, e = 128, 256, len(counts)
    g = torch.Generator().manual_seed(rows)
    x = torch.zeros(e, rows, H)
    x[:, :, :16] = 1.0
    w = torch.zeros(e, N, H)
    w[:, :128, 0] = torch.randint(-13, 14, (e, 128), generator=g).float()
    w[:, 7] = 0
    w[:, 7, :top // 448] = 448
    w[:, 7, top // 448] = top % 448
    w[:, :, 16:] = torch.randint(-13, 14, (e, N, H - 16), generator=g).float()   # meet zeros
    assert torch.equal(w.to(F8).float(), w)
    want = (w[:, :, :16].sum(dim=2) / steps).to(F8).float()
    want[:, 128:] = 0
    osc = torch.zeros(e, rows, B.scale_pitch(N, 128), device="cuda")
    o = torch.zeros(e, rows, N, dtype=F8, device="cuda")
    xs = torch.full((e, rows, 4), TINY, device="cuda")
    B.moe_ep_expert_matmul_fp8(x.to(F8).cuda(), xs, w.to(F8).cuda(),
                               torch.ones(e, 2, 1, device="cuda"),
                               torch.tensor(counts, dtype=torch.int32, device="cuda"), o, "none",
                               None, osc)
    torch.cuda.synchronize()
    for i, c in enumerate(counts):
        assert bool((osc[i, :c, 0].cpu().double() == steps * TINY).all()), i
        assert bool((osc[i, :c, 1].cpu() == 1).all())
        assert bool((o[i, :c].float().cpu() == want[i]).all()), i
