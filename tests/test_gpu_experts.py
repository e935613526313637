"""GPU: the router's choice and the products against their plain 64-bit
forms, at the sizes, masks and layouts where they can go wrong. Buffers hold
NaN (or a marker) wherever a call must not read or write."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import U, assert_close, product64, route64

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# The router's choice
# ---------------------------------------------------------------------------

ROUTE = [
    # T, E, K, score, bias, n_group, topk_group, renormalize, dtype, masked
    (1, 1, 1, "softmax", False, 1, 1, True, F32, 0.0),
    (1, 256, 8, "sigmoid", True, 8, 4, True, F32, 0.0),
    (3, 8, 2, "softmax", False, 1, 1, False, BF16, 0.3),
    (5, 8, 8, "softmax", True, 4, 4, True, F32, 0.6),
    (129, 256, 8, "sigmoid", True, 8, 4, True, BF16, 0.05),
    (127, 60, 4, "softmax", False, 1, 1, True, F32, 0.5),
    (67, 64, 6, "sigmoid", False, 8, 3, False, F32, 0.2),
    (33, 65, 64, "softmax", True, 1, 1, True, F32, 0.1),
    (19, 160, 6, "softmax", False, 8, 3, True, BF16, 0.7),
    (7, 1024, 10, "sigmoid", True, 64, 9, True, F32, 0.9),
    (11, 1000, 16, "softmax", False, 1, 1, True, BF16, 0.0),
    (4, 64, 1, "sigmoid", True, 64, 1, True, F32, 0.5),
]


def _route(logits, bias, K, score, n_group, topk_group, renorm, scale, stream=None):
    T = logits.shape[0]
    ids = torch.full((T, K), -77, dtype=torch.int32, device=DEV)
    w = torch.full((T, K), float("nan"), device=DEV)
    B.moe_ep_route_topk(logits, ids, w, score, bias, n_group, topk_group, renorm, scale, stream)
    return ids, w


def _check_route(logits, bias, K, score, n_group, topk_group, renorm, scale=1.0):
    ids, w = _route(logits.to(DEV), None if bias is None else bias.to(DEV), K, score, n_group,
                    topk_group, renorm, scale)
    torch.cuda.synchronize()
    eid, ew = route64(logits, bias, K, score, n_group, topk_group, renorm, scale)
    assert torch.equal(ids.cpu(), eid)
    off = (w.cpu().double() - ew).abs()
    # fp64 throughout, then one rounding (half a step, 2^-24)
    assert bool((off <= ew.abs() * 2.0 ** -23 + 2.0 ** -149).all()), float(off.max())
    return ids, w


@pytest.mark.parametrize("T,E,K,score,with_bias,ng,tg,renorm,dtype,masked", ROUTE)
def test_route_matches_the_definition(T, E, K, score, with_bias, ng, tg, renorm, dtype, masked):
    say(f"[route] T={T} E={E} K={K} {score} bias={with_bias} groups={tg}/{ng} {dtype}")
    g = gen(T * 1000 + E)
    x = torch.randn(T, E, generator=g) * 2
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = -math.inf
    if T > 2:
        x[1] = -math.inf                         # no expert left
        x[2, : max(1, E // 2)] = float("nan")
    x = x.to(dtype)
    bias = torch.randn(E, generator=g) * 0.2 if with_bias else None
    _check_route(x, bias, K, score, ng, tg, renorm, 2.5)


def test_route_ties_infinities_and_extremes():
    say("[route] ties, infinities, extremes")
    E = 96
    x = torch.zeros(8, E)
    x[1] = torch.arange(E) % 3                   # many ties
    x[2, 5] = math.inf                           # one +inf
    x[3, 7] = x[3, 90] = math.inf                # two
    x[4] = -3.0e38
    x[5, 1:] = -1000.0                           # scores that underflow
    x[6, ::2] = -0.0
    x[7] = torch.linspace(-800, 800, E)
    for score in ("softmax", "sigmoid"):
        for ng, tg in ((1, 1), (8, 3)):
            _check_route(x, None, 6, score, ng, tg, True)
            _check_route(x, torch.where(torch.arange(E) == 5, -math.inf, 0.0), 6, score, ng, tg,
                         True)


def test_route_strided_logits_and_streams():
    """Logits as columns of a wider product, on another stream; the outputs
    feed the pack."""
    say("[route] strided, side stream")
    wide = torch.randn(70, 320, generator=gen(3)).to(DEV)
    x = wide[:, 32:32 + 256]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, w = _route(x, None, 8, "softmax", 1, 1, True, 1.0, side)
    side.synchronize()
    eid, ew = route64(x.cpu(), None, 8, "softmax", 1, 1, True, 1.0)
    assert torch.equal(ids.cpu(), eid)
    assert bool(((w.cpu().double() - ew).abs() <= ew * 2.0 ** -23).all())


# ---------------------------------------------------------------------------
# The product over all tokens
# ---------------------------------------------------------------------------

MATMUL = [
    # T, H, N, act, bias, residual, out
    (1, 8, 8, "none", False, False, F32),
    (1, 7168, 64, "silu_gated", False, False, BF16),
    (1, 520, 1000, "none", True, True, F32),
    (2, 64, 16, "silu", True, False, BF16),
    (15, 72, 24, "gelu", True, True, BF16),
    (16, 128, 4, "none", True, False, F32),
    (17, 1032, 40, "silu_gated", True, True, BF16),
    (33, 136, 264, "none", False, True, BF16),
    (63, 960, 72, "silu_gated", False, False, F32),
    (64, 256, 512, "none", True, False, BF16),
    (65, 1024, 136, "silu_gated", True, False, BF16),
    (100, 2048, 256, "none", False, False, F32),
    (129, 200, 1032, "gelu", False, True, F32),
    (255, 512, 392, "silu_gated", True, True, BF16),
    (257, 1160, 520, "none", True, True, BF16),
    (513, 328, 776, "silu", False, False, BF16),
    (1000, 192, 1288, "silu_gated", False, True, BF16),
]


def _mm_inputs(T, H, N, act, bias, residual, out, seed=0):
    g = gen(seed + T * 7 + H * 3 + N)
    nw = 2 * N if act == "silu_gated" else N
    x = torch.randn(T, H, generator=g).to(BF16)
    w = (torch.randn(nw, H, generator=g) / H ** 0.5).to(BF16)
    b = torch.randn(nw, generator=g) if bias else None
    r = torch.randn(T, N, generator=g).to(out) if residual else None
    return x, w, b, r


def _mm_ref(x, w, b, r, act, N):
    return product64(x.double(), w.double(), None if b is None else b.double(), act, N,
                     None if r is None else r.double())


def _to(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("T,H,N,act,bias,residual,out", MATMUL)
def test_matmul_matches_64_bits(T, H, N, act, bias, residual, out):
    say(f"[matmul] T={T} H={H} N={N} {act} bias={bias} residual={residual} {out}")
    x, w, b, r = _mm_inputs(T, H, N, act, bias, residual, out)
    o = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    B.moe_ep_matmul(_to(x), _to(w), o, act, _to(b), _to(r))
    torch.cuda.synchronize()
    assert_close(o, *_mm_ref(x, w, b, r, act, N), (T, H, N))


@pytest.mark.parametrize("T", [5, 70, 300])
def test_matmul_strided_rows_and_residual_in_place(T):
    """Every operand a column range of a wider tensor whose other columns are
    NaN; the residual is the output itself; nothing outside is written."""
    say(f"[matmul] strided, in place, T={T}")
    H, N = 264, 344
    x, w, b, r = _mm_inputs(T, H, N, "none", True, True, BF16, 5)

    def wide(t, pad):
        big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        big[:, 8:8 + t.shape[1]] = t.to(DEV)
        return big, big[:, 8:8 + t.shape[1]]

    bx, vx = wide(x, 24)
    bw, vw = wide(w, 40)
    bo, vo = wide(r, 16)
    before = bo.clone()
    B.moe_ep_matmul(vx, vw, vo, "none", _to(b), vo)
    torch.cuda.synchronize()
    assert_close(vo, *_mm_ref(x, w, b, r, "none", N), T)
    assert torch.equal(bo[:, :8].view(torch.int16), before[:, :8].view(torch.int16))
    assert torch.equal(bo[:, 8 + N:].view(torch.int16), before[:, 8 + N:].view(torch.int16))


def test_matmul_row_independence_and_nonfinite_rows():
    """A row of NaN or infinities in x spoils that row of the output only; a
    weight row, that column only."""
    say("[matmul] non-finite rows")
    T, H, N = 150, 320, 200
    x, w, _, _ = _mm_inputs(T, H, N, "none", False, False, F32, 9)
    x[149] = float("nan")
    x[3, 17] = math.inf
    w[199, 0] = float("nan")
    o = torch.zeros(T, N, device=DEV)
    B.moe_ep_matmul(_to(x), _to(w), o)
    torch.cuda.synchronize()
    o = o.cpu()
    assert bool(torch.isnan(o[149]).all()) and bool(torch.isnan(o[:, 199]).all())
    assert bool(torch.isinf(o[3, :199]).all())
    rows = [t for t in range(T) if t not in (3, 149)]
    y, e = _mm_ref(x[rows], w[:199], None, None, "none", 199)
    assert_close(o[rows][:, :199], y, e, "finite part")


# ---------------------------------------------------------------------------
# The experts' products
# ---------------------------------------------------------------------------

EXPERTS = [
    # counts, rows, H, N, act, bias, out
    ([0], 16, 64, 16, "none", False, BF16),
    ([1], 1, 8, 8, "none", True, F32),
    ([3, 0, 1, 16], 16, 136, 40, "silu_gated", True, BF16),
    ([17, 33, 0, 64, 63], 64, 520, 136, "none", True, BF16),
    ([-4, 5, 99], 40, 264, 72, "gelu", False, F32),          # clamped to [0, rows]
    ([128, 65, 0, 0, 1, 129], 160, 256, 264, "silu_gated", False, BF16),
    ([300, 0, 257, 255], 320, 328, 520, "silu_gated", True, BF16),
    ([511, 2, 256], 520, 200, 776, "none", True, F32),
    ([0] * 70 + [2] + [0] * 60 + [7], 8, 64, 24, "silu", True, BF16),
    ([40, 600, 0, 18], 640, 1160, 288, "silu_gated", False, F32),
]


def _experts(counts, rows, H, N, act, bias, seed=0):
    g = gen(seed + len(counts) * 31 + H + N)
    e = len(counts)
    nw = 2 * N if act == "silu_gated" else N
    n = [min(max(c, 0), rows) for c in counts]
    x = torch.full((e, rows, H), float("nan"), dtype=BF16)
    for i in range(e):
        x[i, :n[i]] = torch.randn(n[i], H, generator=g).to(BF16)
    w = (torch.randn(e, nw, H, generator=g) / H ** 0.5).to(BF16)
    b = torch.randn(e, nw, generator=g) if bias else None
    return n, x, w, b


def _marked(shape, dtype):
    """A buffer of a bit pattern that no result has, to see what is written."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(0xFB)
    return t


def _check_experts(n, x, w, b, act, N, out, o):
    o = o.cpu()
    for i, c in enumerate(n):
        if c:
            y, e = product64(x[i, :c].double(), w[i].double(),
                             None if b is None else b[i].double(), act, N)
            assert_close(o[i, :c], y, e, ("expert", i))
        tail = o[i, c:].contiguous().view(torch.uint8)
        assert bool((tail == 0xFB).all()), ("rows behind the count", i)


@pytest.mark.parametrize("counts,rows,H,N,act,bias,out", EXPERTS)
def test_expert_matmul_matches_64_bits(counts, rows, H, N, act, bias, out):
    say(f"[experts] counts={counts[:6]} rows={rows} H={H} N={N} {act} {out}")
    n, x, w, b = _experts(counts, rows, H, N, act, bias)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    o = _marked((len(n), rows, N), out)
    B.moe_ep_expert_matmul(_to(x), _to(w), cnt, o, act, _to(b))
    torch.cuda.synchronize()
    _check_experts(n, x, w, b, act, N, out, o)


def test_expert_matmul_strided_far_experts():
    """Experts further apart than 2^32 bytes, in x, w and out."""
    say("[experts] far strides")
    counts, rows, H, N = [70, 3, 260], 264, 136, 72
    n, x, w, b = _experts(counts, rows, H, N, "silu_gated", True, 3)
    far = (1 << 31) + 64                       # elements: over 4 GiB of bf16

    def spread(t):
        per = t.shape[1] * t.shape[2]
        big = torch.empty(far * (len(n) - 1) + per, dtype=t.dtype, device=DEV)
        v = big.as_strided(t.shape, (far, t.shape[2], 1))
        v.copy_(t)
        return v

    o = spread(torch.zeros(len(n), rows, N, dtype=BF16))
    o.copy_(_marked((len(n), rows, N), BF16))
    B.moe_ep_expert_matmul(spread(x), spread(w), torch.tensor(counts, dtype=torch.int32, device=DEV),
                           o, "silu_gated", _to(b))
    torch.cuda.synchronize()
    _check_experts(n, x, w, b, "silu_gated", N, BF16, o.contiguous())


EXPERTS8 = [
    # counts, rows, H, N, act, bias, out
    ([1], 1, 128, 16, "none", False, F32),
    ([0, 5, 16], 16, 256, 40, "none", True, BF16),
    ([17, 0, 64, 1], 64, 640, 136, "silu_gated", True, BF16),
    ([200, 3, 0, 129], 208, 384, 264, "silu_gated", False, F32),
    ([300, 257, 31], 320, 512, 384, "none", True, BF16),
    ([1, 0, 15], 16, 256, 128, "none", False, F8),
    ([33, 0, 16, 5], 40, 640, 384, "silu_gated", True, F8),
    ([300, 2, 130], 304, 384, 640, "silu_gated", False, F8),
    ([260, 0, 64], 264, 256, 256, "silu", True, F8),
]


def _experts8(counts, rows, H, N, act, bias, seed=0):
    """Codes and scales, and the exact values they stand for (float64)."""
    n, x, w, b = _experts(counts, rows, H, N, act, bias, seed + 100)
    g = gen(seed + 7)
    e, hb = len(n), H // 128
    halves = w.shape[1] // N
    per = -(-N // 128)
    gp = B.scale_pitch(H, 128)
    xq = torch.full((e, rows, H), 0x7F, dtype=torch.uint8)          # NaN codes behind the count
    xs = torch.full((e, rows, gp), float("nan"))
    x64 = torch.zeros(e, rows, H, dtype=torch.float64)
    for i, c in enumerate(n):
        v = x[i, :c].float().view(c, hb, 128)
        s = torch.rand(c, hb, generator=g) * 0.01 + 0.001
        q = (v / s[:, :, None] * 0.05).clamp(-448, 448).to(F8)
        xq[i, :c] = q.view(torch.uint8).view(c, H)
        xs[i, :c, :hb] = s
        x64[i, :c] = (q.double() * s.double()[:, :, None]).view(c, H)
    wq = (torch.randn(e, halves * N, H, generator=g) * 3).to(F8)
    ws = torch.rand(e, halves * per, hb, generator=g) + 0.5
    row = torch.arange(halves * N)
    row = row // N * per + row % N // 128
    w64 = wq.double() * ws.double()[:, row].repeat_interleave(128, dim=2)
    return n, (xq.view(F8), xs, wq, ws, b), x64, w64


@pytest.mark.parametrize("counts,rows,H,N,act,bias,out", EXPERTS8)
def test_expert_matmul_fp8_matches_64_bits(counts, rows, H, N, act, bias, out):
    say(f"[experts fp8] counts={counts} rows={rows} H={H} N={N} {act} {out}")
    n, (xq, xs, wq, ws, b), x64, w64 = _experts8(counts, rows, H, N, act, bias)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    o = _marked((len(n), rows, N), torch.uint8 if out == F8 else out)
    np_ = B.scale_pitch(N, 128)
    osc = _marked((len(n), rows, np_), F32) if out == F8 else None
    B.moe_ep_expert_matmul_fp8(_to(xq), _to(xs), _to(wq), _to(ws), cnt, o, act, _to(b), osc)
    torch.cuda.synchronize()
    if out != F8:
        o = o.cpu()
        for i, c in enumerate(n):
            # a slab's scale is itself a rounded product, and one more multiply-add
            y, e = product64(x64[i, :c], w64[i], None if b is None else b[i].double(), act, N,
                             extra=4)
            assert_close(o[i, :c], y, e, ("expert", i))
            assert bool((o[i, c:].contiguous().view(torch.uint8) == 0xFB).all())
        return
    codes, osc = o.cpu(), osc.cpu()
    for i, c in enumerate(n):
        y, e = product64(x64[i, :c], w64[i], None if b is None else b[i].double(), act, N,
                         extra=4)
        amax = y.abs().view(c, N // 128, 128).amax(dim=2)
        worst = e.view(c, N // 128, 128).amax(dim=2)
        s = osc[i, :c, :N // 128].double()
        # the scale is amax / 448: amax is off by no more than its elements
        assert bool(((s * 448 - amax).abs() <= worst + 4 * U * amax).all()), i
        assert bool((osc[i, :c, N // 128:] == 0).all())
        v = codes[i, :c].view(F8).double() * s.repeat_interleave(128, dim=1)
        sr = s.repeat_interleave(128, dim=1)
        # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale among
        # the subnormals
        tol = e + (y.abs() + e) * 2.0 ** -4 + sr * 2.0 ** -10 + U * y.abs()
        assert bool(((v - y).abs() <= tol).all()), (i, float(((v - y).abs() / tol).max()))
        assert bool((codes[i, c:] == 0xFB).all())
        assert bool((osc[i, c:].contiguous().view(torch.uint8) == 0xFB).all())


def test_expert_matmul_fp8_output_feeds_the_next_product():
    """Both products of an expert in fp8: the first's codes and scales are the
    second's input as they are."""
    say("[experts fp8] chain")
    counts, rows, H, I = [40, 0, 7], 48, 256, 384
    n, (xq, xs, wq, ws, _), _, _ = _experts8(counts, rows, H, I, "silu_gated", False, 11)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    h = torch.zeros(3, rows, I, dtype=F8, device=DEV)
    hs = torch.zeros(3, rows, B.scale_pitch(I, 128), device=DEV)
    B.moe_ep_expert_matmul_fp8(_to(xq), _to(xs), _to(wq), _to(ws), cnt, h, "silu_gated", None, hs)
    g = gen(12)
    w2 = (torch.randn(3, H, I, generator=g) * 3).to(F8)
    s2 = torch.rand(3, H // 128, I // 128, generator=g) + 0.5
    o = _marked((3, rows, H), F32)
    B.moe_ep_expert_matmul_fp8(h, hs, _to(w2), _to(s2), cnt, o)
    torch.cuda.synchronize()
    for i, c in enumerate(n):
        x64 = h[i, :c].cpu().double() * hs[i, :c, :I // 128].cpu().double().repeat_interleave(128, 1)
        w64 = w2[i].double() * s2[i].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        y, e = product64(x64, w64, None, "none", H, extra=4)
        assert_close(o[i, :c].cpu(), y, e, i)


# ---------------------------------------------------------------------------
# Sizes that take the larger tiles: enough experts and columns that every cut
# of the rows (runs of 32 to 256, a last round in halves and quarters) occurs.
# The 64-bit products run on the GPU here (torch, float64).
# ---------------------------------------------------------------------------

def _spread(e, top, seed):
    """Counts from 0 to top, each 32-row class among them, odd ones too."""
    g = gen(seed)
    c = torch.randint(0, top + 1, (e,), generator=g).tolist()
    return [0, top, top - 1, 1, 16, 17, 33] + c[7:]


MANY = [
    # experts, most rows, H, N, act, bias, out
    (46, 256, 200, 2000, "none", True, BF16),           # a whole round and halves
    (33, 256, 264, 1000, "silu_gated", False, F32),
    (20, 700, 136, 2056, "silu", False, BF16),
    (12, 256, 392, 1096, "silu_gated", True, BF16),     # quarters
    (70, 64, 72, 1288, "none", False, F32),             # up to 64 rows each
    (9, 128, 520, 2312, "silu_gated", False, BF16),
    (3, 1500, 1032, 3200, "gelu", True, F32),
]


@pytest.mark.parametrize("e,top,H,N,act,bias,out", MANY)
def test_expert_matmul_on_larger_tiles(e, top, H, N, act, bias, out):
    say(f"[experts, larger] e={e} rows<={top} H={H} N={N} {act} {out}")
    counts = _spread(e, top, e)[:e]
    n, x, w, b = _experts(counts, top + 3, H, N, act, bias, 60)
    x, w, b = _to(x), _to(w), _to(b)
    o = _marked((e, top + 3, N), out)
    B.moe_ep_expert_matmul(x, w, torch.tensor(counts, dtype=torch.int32, device=DEV), o, act, b)
    torch.cuda.synchronize()
    for i, c in enumerate(n):
        if c:
            y, err = product64(x[i, :c].double(), w[i].double(),
                               None if b is None else b[i].double(), act, N)
            assert_close(o[i, :c], y.cpu(), err.cpu(), ("expert", i, c))
        assert bool((o[i, c:].contiguous().view(torch.uint8) == 0xFB).all()), (i, c)


MANY8 = [
    (46, 256, 256, 2048, "none", True, BF16),
    (33, 256, 384, 1024, "silu_gated", False, F32),
    (12, 256, 640, 1152, "silu_gated", True, F8),
    (40, 64, 128, 1280, "none", False, F8),
    (20, 600, 256, 1096, "silu_gated", False, BF16),
    (60, 64, 384, 1280, "none", False, BF16),
]


@pytest.mark.parametrize("e,top,H,N,act,bias,out", MANY8)
def test_expert_matmul_fp8_on_larger_tiles(e, top, H, N, act, bias, out):
    say(f"[experts fp8, larger] e={e} rows<={top} H={H} N={N} {act} {out}")
    counts = _spread(e, top, e + 1)[:e]
    rows = top + 3
    n, (xq, xs, wq, ws, b), x64, w64 = _experts8(counts, rows, H, N, act, bias, 61)
    b = _to(b)
    o = _marked((e, rows, N), torch.uint8 if out == F8 else out)
    osc = _marked((e, rows, B.scale_pitch(N, 128)), F32) if out == F8 else None
    B.moe_ep_expert_matmul_fp8(_to(xq), _to(xs), _to(wq), _to(ws),
                               torch.tensor(counts, dtype=torch.int32, device=DEV), o, act, b, osc)
    torch.cuda.synchronize()
    for i, c in enumerate(n):
        assert bool((o[i, c:].contiguous().view(torch.uint8) == 0xFB).all()), (i, c)
        if not c:
            continue
        y, err = product64(x64[i, :c].to(DEV), w64[i].to(DEV), None if b is None else b[i].double(),
                           act, N, extra=4)
        if out != F8:
            assert_close(o[i, :c], y.cpu(), err.cpu(), ("expert", i, c))
            continue
        s = osc[i, :c, :N // 128].double()
        amax, worst = (t.view(c, N // 128, 128).amax(dim=2) for t in (y.abs(), err))
        assert bool(((s * 448 - amax).abs() <= worst + 4 * U * amax).all()), (i, c)
        assert bool((osc[i, :c, N // 128:] == 0).all())
        sr = s.repeat_interleave(128, dim=1)
        v = o[i, :c].view(F8).double() * sr
        tol = err + (y.abs() + err) * 2.0 ** -4 + sr * 2.0 ** -10 + U * y.abs()
        assert bool(((v - y).abs() <= tol).all()), (i, c, float(((v - y).abs() / tol).max()))


@pytest.mark.parametrize("T,H,N,act,bias,residual,out", [
    (4096, 1032, 2048, "silu_gated", True, True, BF16),
    (2051, 4104, 2056, "none", False, True, BF16),
    (8191, 264, 1544, "none", True, False, F32),
    (700, 2056, 1288, "gelu", True, True, F32),
    (1023, 520, 520, "silu_gated", False, False, BF16),
    (130, 4104, 4104, "none", False, True, F32),
    (20000, 72, 264, "silu", True, False, BF16),
])
def test_matmul_on_larger_tiles(T, H, N, act, bias, residual, out):
    say(f"[matmul, larger] T={T} H={H} N={N} {act} {out}")
    x, w, b, r = (_to(t) for t in _mm_inputs(T, H, N, act, bias, residual, out, 70))
    o = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    B.moe_ep_matmul(x, w, o, act, b, r)
    torch.cuda.synchronize()
    y, e = _mm_ref(x, w, b, r, act, N)
    assert_close(o, y.cpu(), e.cpu(), (T, H, N))


def test_products_do_not_depend_on_what_lies_beside_them():
    """A row's result is the same bits whatever the other groups and rows of
    the same tile cut hold."""
    say("[experts] independence")
    counts, rows, H, N = [200, 40, 0, 256], 256, 264, 520
    n, x, w, _ = _experts(counts, rows, H, N, "none", False, 80)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    outs = []
    for fill in (float("nan"), 3.0):
        xx = x.clone()
        for i, c in enumerate(n):
            xx[i, c:] = fill
        o = _marked((4, rows, N), F32)
        B.moe_ep_expert_matmul(_to(xx), _to(w), cnt, o)
        B.moe_ep_expert_matmul(_to(xx), _to(w), cnt, o)     # and again over its own output
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8))


# ---------------------------------------------------------------------------
# Streams, graphs, repeats
# ---------------------------------------------------------------------------

def _calls():
    """One call of each operator with its outputs (in device buffers)."""
    x, w, b, r = (_to(t) for t in _mm_inputs(90, 264, 136, "silu_gated", True, True, BF16, 21))
    o1 = torch.empty(90, 136, dtype=BF16, device=DEV)
    counts, rows = [70, 0, 300, 9], 304
    n, ex, ew, eb = _experts(counts, rows, 264, 136, "none", True, 22)
    ex, ew, eb = _to(ex), _to(ew), _to(eb)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    o2 = torch.zeros(4, rows, 136, dtype=F32, device=DEV)
    n, (xq, xs, wq, ws, _), _, _ = _experts8([20, 0, 130], 136, 256, 128, "silu_gated", False, 23)
    xq, xs, wq, ws = _to(xq), _to(xs), _to(wq), _to(ws)
    cnt8 = torch.tensor([20, 0, 130], dtype=torch.int32, device=DEV)
    o3 = torch.zeros(3, 136, 128, dtype=F8, device=DEV)
    s3 = torch.zeros(3, 136, 4, device=DEV)
    lg = torch.randn(77, 64, generator=gen(24)).to(DEV)
    ids = torch.zeros(77, 6, dtype=torch.int32, device=DEV)
    wt = torch.zeros(77, 6, device=DEV)

    def go(stream=None):
        B.moe_ep_matmul(x, w, o1, "silu_gated", b, r, stream)
        B.moe_ep_expert_matmul(ex, ew, cnt, o2, "none", eb, stream)
        B.moe_ep_expert_matmul_fp8(xq, xs, wq, ws, cnt8, o3, "silu_gated", None, s3, stream)
        B.moe_ep_route_topk(lg, ids, wt, n_group=8, topk_group=4, stream=stream)

    return go, [o1, o2, o3, s3, ids, wt]


def _bytes(outs):
    return [o.contiguous().view(torch.uint8).clone() for o in outs]


def test_graph_replays_and_side_streams_give_the_eager_bytes():
    say("[experts] graph and streams")
    go, outs = _calls()
    go()
    torch.cuda.synchronize()
    eager = _bytes(outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    go(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, _bytes(outs)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for rep in range(4):
        for o in (outs[0], outs[4], outs[5]):       # written in full
            o.view(torch.uint8).fill_(0xAB)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, _bytes(outs))), rep


def test_counts_change_between_replays():
    """A captured product reads the counts of the replay, not of the capture."""
    say("[experts] counts between replays")
    rows, H, N = 300, 136, 72
    n, x, w, _ = _experts([300, 300], rows, H, N, "none", False, 31)
    dx, dw = _to(x), _to(w)
    cnt = torch.zeros(2, dtype=torch.int32, device=DEV)
    o = _marked((2, rows, N), F32)
    B.moe_ep_expert_matmul(dx, dw, cnt, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_ep_expert_matmul(dx, dw, cnt, o)
    for counts in ([0, 3], [300, 0], [65, 257], [0, 0]):
        o.view(torch.uint8).fill_(0xFB)
        cnt.copy_(torch.tensor(counts, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check_experts(counts, x, w, None, "none", N, F32, o)
