"""GPU: fp8 products whose large terms cancel within a block of 128 columns.

The codes stand for whole numbers and the scales are 1, 2 or 4, so that every
product is a whole number, and the terms' absolute values add up to less than
2^24: a sum held in fp32 (24 bits) is exact in whatever order it is taken, and
the result is the exact sum rounded once. A sum that keeps fewer bits loses the
small terms beside +-448 * 448."""
import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def whole_codes(shape, g):
    return torch.randint(-4, 5, shape, generator=g).float()


def inputs(counts, rows, H, N, gated, seed):
    """x, w with pairs of columns in each block where 448 * 448 cancels; the
    scales; a bias; the exact results in float64. Gated: the gate rows are zero
    with a bias of 64, and silu(64) is 64 in fp32."""
    g = torch.Generator().manual_seed(seed)
    e, hb = len(counts), H // 128
    x, w = whole_codes((e, rows, H), g), whole_codes((e, N, H), g)
    for blk in range(hb):
        p = 128 * blk + torch.randperm(128, generator=g)[:2]
        x[:, :, p[0]], x[:, :, p[1]] = 448.0, -448.0
        w[:, :, p[0]] = w[:, :, p[1]] = 448.0
    xs = 2.0 ** torch.randint(0, 2, (e, rows, hb), generator=g)
    ws = 2.0 ** torch.randint(0, 2, (e, -(-N // 128), hb), generator=g)
    b = torch.randint(-9, 10, (e, N), generator=g).float()
    xf = x.double() * xs.double().repeat_interleave(128, dim=2)
    wf = w.double() * ws.double().repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)
    y = xf @ wf.transpose(1, 2) + b.double()[:, None]
    assert float((xf.abs() @ wf.abs().transpose(1, 2)).max()) + 9 < 2.0 ** 24
    if gated:
        y = 64 * y
        w = torch.cat([torch.zeros_like(w), w], dim=1)
        ws = torch.cat([torch.ones_like(ws), ws], dim=1)
        b = torch.cat([torch.full_like(b, 64.0), b], dim=1)
    pad = torch.full((e, rows, B.scale_pitch(H, 128)), float("nan"))
    pad[:, :, :hb] = xs
    return x.to(F8), pad, w.to(F8), ws, b, y


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, F32, F8])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,rows,H,N", [
    ([1, 16, 0, 7], 16, 512, 128),           # 16-row tiles
    ([20, 3, 32], 32, 256, 384),
    ([64, 17, 33], 64, 640, 256),            # 64-row tiles
    ([5, 300, 129, 200], 304, 384, 384),     # every higher one
    ([256, 224, 192, 160, 96] * 14, 256, 256, 1024),
])
def test_large_terms_that_cancel_leave_the_small_ones(counts, rows, H, N, gated, out):
    say(f"[fp8 sums] counts={counts[:5]} H={H} N={N} gated={gated} {out}")
    x, xs, w, ws, b, y = (t.cuda() for t in inputs(counts, rows, H, N, gated, H + N))
    o = torch.zeros(y.shape, dtype=out, device="cuda")
    osc = torch.zeros(len(counts), rows, B.scale_pitch(N, 128), device="cuda") if out == F8 else None
    B.moe_ep_expert_matmul_fp8(x, xs, w, ws, torch.tensor(counts, dtype=torch.int32, device="cuda"),
                               o, "silu_gated" if gated else "none", b, osc)
    torch.cuda.synchronize()
    for i, c in enumerate(counts):
        want = y[i, :c].float()
        assert torch.equal(want.double(), y[i, :c])
        if out != F8:
            assert bool((o[i, :c] == want.to(out)).all()), i
            continue
        # on the CPU: torch divides by a number on the GPU as a product with its
        # reciprocal, and the scale is amax / 448 rounded once
        want = want.cpu()
        amax = want.abs().view(c, N // 128, 128).amax(dim=2)
        s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        assert torch.equal(osc[i, :c, :N // 128].cpu(), s), i
        q = (want / s.repeat_interleave(128, dim=1)).to(F8)
        assert torch.equal(o[i, :c].float().cpu(), q.float()), i
