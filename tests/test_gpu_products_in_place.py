"""GPU: the product over all tokens with its residual in place, at sizes whose
last round of tiles is cut in parts: each result holds the residual once, and
equals the result with a residual of its own bit for bit."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import assert_close, product64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# Tiles of the last round and what a part of theirs has: 84 and 96 and 112 in
# halves of 96 rows, 80 in halves of 128, 44 in quarters of 64, 19 in quarters
# of 32; the last one takes the middle tiles.
SIZES = [(513, 2048, 7168), (520, 2048, 7168), (576, 2048, 7168), (384, 4096, 12288),
         (300, 1536, 14336), (3000, 4096, 7168), (576, 4096, 25600), (100, 4096, 70400),
         (4100, 264, 1544)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,H,N", SIZES)
def test_residual_in_place_is_added_once(T, H, N, out):
    say(f"[matmul] in place T={T} H={H} N={N} {out}")
    g = torch.Generator().manual_seed(T + H + N)
    x = torch.randn(T, H, generator=g).to(BF16).cuda()
    w = (torch.randn(N, H, generator=g) / H ** 0.5).to(BF16).cuda()
    r = torch.randn(T, N, generator=g).to(out).cuda()
    apart = torch.full((T, N), float("nan"), dtype=out, device="cuda")
    B.moe_ep_matmul(x, w, apart, residual=r)
    v, e = product64(x.double(), w.double(), None, "none", N, r.double())
    assert_close(apart, v.cpu(), e.cpu(), (T, H, N))
    for rep in range(3):
        o = r.clone()
        B.moe_ep_matmul(x, w, o, residual=o)
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.uint8), apart.view(torch.uint8)), rep
