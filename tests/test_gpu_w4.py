"""GPU: the products with 4-bit weights against their plain 64-bit forms, at
the sizes, counts and layouts where they can go wrong. Buffers hold NaN (or a
marker) wherever a call must not read or write."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import assert_close, product64
from w4 import pitch, random_w4, value64

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def _to(t):
    return None if t is None else t.to(DEV)


def _marked(shape, dtype):
    """A buffer of a bit pattern that no result has, to see what is written."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(0xFB)
    return t


def _factor(w64, whole, N):
    """Weights times the factor of their matrix (of gate and up rows)."""
    if whole is None:
        return w64
    return w64 * whole.double().repeat_interleave(N, dim=-1).unsqueeze(-1)


def _dense(T, H, N, group, act, bias, residual, out, whole, seed=0):
    g = gen(seed + T * 7 + H * 3 + N + group)
    halves = 2 if act == "silu_gated" else 1
    x = torch.randn(T, H, generator=g).to(BF16)
    w, s = random_w4((), halves * N, H, group, g)
    b = torch.randn(halves * N, generator=g) if bias else None
    r = torch.randn(T, N, generator=g).to(out) if residual else None
    f = torch.rand(halves, generator=g) + 0.5 if whole else None
    return x, w, s, b, r, f


def _ref(x, w, s, b, r, f, group, act, N):
    # the factor is one more rounding of the sum
    return product64(x.double(), _factor(value64(w, s, group), f, N),
                     None if b is None else b.double(), act, N,
                     None if r is None else r.double(), extra=2)


DENSE = [
    # T, H, N, group, act, bias, residual, out, whole
    (1, 32, 8, 16, "none", False, False, F32, False),
    (1, 7168, 64, 16, "silu_gated", False, False, BF16, True),
    (1, 7168, 2048, 32, "none", True, True, BF16, False),
    (1, 544, 1000, 32, "none", True, True, F32, True),
    (2, 64, 16, 16, "silu", True, False, BF16, False),
    (3, 2080, 264, 16, "silu_gated", True, True, F32, True),
    (5, 16384, 40, 32, "none", False, False, F32, False),
    (7, 1056, 520, 16, "gelu", False, True, BF16, True),
    (8, 96, 24, 32, "gelu", True, True, BF16, False),
    (9, 4128, 72, 16, "none", False, False, BF16, False),
    (15, 96, 24, 32, "gelu", True, True, BF16, True),
    (16, 128, 4, 16, "none", True, False, F32, False),
    (16, 7168, 136, 16, "none", True, False, F32, True),
    (17, 1056, 40, 16, "silu_gated", True, True, BF16, True),
    (31, 2048, 7168, 32, "none", False, True, BF16, False),
    (33, 160, 264, 32, "none", False, True, BF16, False),
    (63, 960, 72, 16, "silu_gated", False, False, F32, True),
    (64, 256, 512, 32, "none", True, False, BF16, False),
    (65, 1024, 136, 16, "silu_gated", True, False, BF16, True),
    (100, 2048, 256, 16, "none", False, False, F32, False),
    (129, 224, 1032, 32, "gelu", False, True, F32, False),
    (255, 512, 392, 16, "silu_gated", True, True, BF16, True),
    (257, 1184, 520, 16, "none", True, True, BF16, False),
    (513, 352, 776, 32, "silu", False, False, BF16, True),
    (1000, 192, 1288, 16, "silu_gated", False, True, BF16, False),
]


@pytest.mark.parametrize("T,H,N,group,act,bias,residual,out,whole", DENSE)
def test_matmul_w4_matches_64_bits(T, H, N, group, act, bias, residual, out, whole):
    say(f"[matmul w4] T={T} H={H} N={N} /{group} {act} bias={bias} res={residual} {out}")
    x, w, s, b, r, f = _dense(T, H, N, group, act, bias, residual, out, whole)
    o = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    B.moe_ep_matmul_w4(_to(x), _to(w), _to(s), o, group, act, _to(b), _to(r), _to(f))
    torch.cuda.synchronize()
    assert_close(o, *_ref(x, w, s, b, r, f, group, act, N), (T, H, N))


@pytest.mark.parametrize("T", [1, 5, 16, 30, 70, 300])
def test_matmul_w4_strided_rows_and_residual_in_place(T):
    """Every operand a column range of a wider tensor whose other columns are
    NaN (or NaN scales); the residual is the output itself; nothing outside is
    written."""
    say(f"[matmul w4] strided, in place, T={T}")
    H, N, group = 288, 344, 16
    x, w, s, b, r, f = _dense(T, H, N, group, "none", True, True, BF16, True, 5)
    s = s[:, :H // group]

    def wide(t, left, right, fill):
        big = torch.full((t.shape[0], left + t.shape[1] + right), fill, dtype=t.dtype, device=DEV)
        big[:, left:left + t.shape[1]] = t.to(DEV)
        return big, big[:, left:left + t.shape[1]]

    bx, vx = wide(x, 8, 24, float("nan"))
    bw, vw = wide(w, 16, 32, 0x77)
    bs, vs = wide(s, 16, 14, 0x7F)
    bo, vo = wide(r, 8, 16, float("nan"))
    before = bo.clone()
    B.moe_ep_matmul_w4(vx, vw, vs, vo, group, "none", _to(b), vo, _to(f))
    torch.cuda.synchronize()
    assert_close(vo, *_ref(x, w, s, b, r, f, group, "none", N), T)
    assert torch.equal(bo[:, :8].view(torch.int16), before[:, :8].view(torch.int16))
    assert torch.equal(bo[:, 8 + N:].view(torch.int16), before[:, 8 + N:].view(torch.int16))


@pytest.mark.parametrize("group", [16, 32])
@pytest.mark.parametrize("T", [2, 14, 40, 150])
def test_every_code_with_every_scale(T, group):
    """Rows of x that pick single columns: each output is one weight, exactly,
    for all 16 codes and all 256 scale codes (NaN ones among them)."""
    say(f"[w4] codes and scales, T={T} /{group}")
    H, N = 16 * group, 256
    codes = torch.arange(16, dtype=torch.uint8).repeat(group // 2)            # of half a row
    low = codes.repeat(2)[:H // 2]
    w = (low + low.flip(0) * 16).repeat(N, 1)
    s = torch.full((N, pitch(H, group)), 0, dtype=torch.uint8)
    s[:, :H // group] = torch.arange(N, dtype=torch.int32).to(torch.uint8)[:, None]
    w64 = value64(w, s, group)
    g = gen(T)
    at = torch.randint(0, H, (T,), generator=g)
    x = torch.zeros(T, H)
    x[torch.arange(T), at] = 1.0
    o = torch.full((T, N), 7.0, device=DEV)
    B.moe_ep_matmul_w4(x.to(BF16).to(DEV), w.to(DEV), s.to(DEV), o, group)
    torch.cuda.synchronize()
    want = w64[:, at].t().contiguous()
    nan = torch.isnan(w64).any(dim=1)                    # a NaN scale spoils its row of w
    top = 255 if group == 16 else 252                    # 6 * 2^125 is within bf16
    fine = ~nan & (torch.arange(N) <= top)
    assert bool(torch.isnan(o.cpu()[:, nan]).all()) and int(nan.sum()) == (2 if group == 16 else 1)
    got = o.cpu().double()[:, fine]
    # fp32 results below its normal range may be zero in the matrix cores' sums
    small = want[:, fine].abs() < 2.0 ** -126
    assert bool(((got == want[:, fine]) | (small & (got.abs() <= 2.0 ** -126))).all())


@pytest.mark.parametrize("T", [4, 16, 40, 150])
def test_matmul_w4_row_independence_and_nonfinite_rows(T):
    """A row of NaN or infinities in x spoils that row of the output only; a NaN
    scale, that column only."""
    say(f"[matmul w4] non-finite rows, T={T}")
    H, N, group = 320, 200, 16
    x, w, s, _, _, _ = _dense(T, H, N, group, "none", False, False, F32, False, 9)
    x[T - 1] = float("nan")
    x[1, 17] = math.inf
    w[:, 8] = 0x22                                   # columns 16 and 17: 1 times their scale
    s[:, 1] = 0x38
    s[199, 3] = 0x7F
    o = torch.zeros(T, N, device=DEV)
    B.moe_ep_matmul_w4(_to(x), _to(w), _to(s), o, group)
    torch.cuda.synchronize()
    o = o.cpu()
    assert bool(torch.isnan(o[T - 1]).all()) and bool(torch.isnan(o[:, 199]).all())
    assert bool(torch.isinf(o[1, :199]).all())
    rows = [t for t in range(T) if t not in (1, T - 1)]
    y, e = _ref(x[rows], w[:199], s[:199], None, None, None, group, "none", 199)
    assert_close(o[rows][:, :199], y, e, "finite part")


EXPERTS = [
    # counts, rows, H, N, group, act, bias, out, whole
    ([0], 16, 64, 16, 16, "none", False, BF16, False),
    ([1], 1, 32, 8, 32, "none", True, F32, True),
    ([3, 0, 1, 16], 16, 160, 40, 16, "silu_gated", True, BF16, True),
    ([1, 0, 2, 5, 0, 9, 13], 32, 2112, 520, 16, "silu_gated", False, BF16, True),
    ([17, 33, 0, 64, 63], 64, 544, 136, 32, "none", True, BF16, False),
    ([-4, 5, 99], 40, 288, 72, 16, "gelu", False, F32, True),          # clamped to [0, rows]
    ([128, 65, 0, 0, 1, 129], 160, 256, 264, 16, "silu_gated", False, BF16, False),
    ([300, 0, 257, 255], 320, 352, 520, 32, "silu_gated", True, BF16, True),
    ([511, 2, 256], 520, 224, 776, 16, "none", True, F32, False),
    ([0] * 70 + [2] + [0] * 60 + [7], 8, 64, 24, 32, "silu", True, BF16, True),
    ([40, 600, 0, 18], 640, 1184, 288, 16, "silu_gated", False, F32, True),
    ([20, 30, 0, 8], 32, 7168, 64, 16, "none", False, BF16, False),
]


def _experts(counts, rows, H, N, group, act, bias, whole, seed=0):
    g = gen(seed + len(counts) * 31 + H + N)
    e = len(counts)
    halves = 2 if act == "silu_gated" else 1
    n = [min(max(c, 0), rows) for c in counts]
    x = torch.full((e, rows, H), float("nan"), dtype=BF16)
    for i in range(e):
        x[i, :n[i]] = torch.randn(n[i], H, generator=g).to(BF16)
    w, s = random_w4((e,), halves * N, H, group, g)
    b = torch.randn(e, halves * N, generator=g) if bias else None
    f = torch.rand(e, halves, generator=g) + 0.5 if whole else None
    return n, x, w, s, b, f


def _check_experts(n, x, w, s, b, f, group, act, N, o, where="cpu"):
    o = o.to(where)
    for i, c in enumerate(n):
        if c:
            w64 = _factor(value64(w[i], s[i], group), None if f is None else f[i], N).to(where)
            y, e = product64(x[i, :c].to(where).double(), w64,
                             None if b is None else b[i].to(where).double(), act, N, extra=2)
            assert_close(o[i, :c], y.cpu(), e.cpu(), ("expert", i, c))
        tail = o[i, c:].contiguous().view(torch.uint8)
        assert bool((tail == 0xFB).all()), ("rows behind the count", i)


@pytest.mark.parametrize("counts,rows,H,N,group,act,bias,out,whole", EXPERTS)
def test_expert_matmul_w4_matches_64_bits(counts, rows, H, N, group, act, bias, out, whole):
    say(f"[experts w4] counts={counts[:8]} rows={rows} H={H} N={N} /{group} {act} {out}")
    n, x, w, s, b, f = _experts(counts, rows, H, N, group, act, bias, whole)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    o = _marked((len(n), rows, N), out)
    B.moe_ep_expert_matmul_w4(_to(x), _to(w), _to(s), cnt, o, group, act, _to(b), _to(f))
    torch.cuda.synchronize()
    _check_experts(n, x, w, s, b, f, group, act, N, o)


def test_expert_matmul_w4_expert_strides():
    """Each operand the inner part of a wider one along the experts, the types
    of the scales both ways."""
    say("[experts w4] strides")
    for group, typed in ((16, torch.float8_e4m3fn), (32, torch.float8_e8m0fnu)):
        counts, rows, H, N = [5, 0, 19], 24, 96, 40
        n, x, w, s, b, f = _experts(counts, rows, H, N, group, "silu_gated", True, True, 3)

        def apart(t, fill):
            big = torch.full((2 * t.shape[0], *t.shape[1:]), fill, dtype=t.dtype, device=DEV)
            big[::2] = t.to(DEV)
            return big, big[::2]

        bx, vx = apart(x, float("nan"))
        bw, vw = apart(w, 0x77)
        bs, vs = apart(s, 0x7F)
        bb, vb = apart(b, float("nan"))
        bo = _marked((6, rows, N), BF16)
        cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
        B.moe_ep_expert_matmul_w4(vx, vw, vs.view(typed), cnt, bo[::2], group, "silu_gated", vb,
                                  _to(f))
        torch.cuda.synchronize()
        _check_experts(n, x, w, s, b, f, group, "silu_gated", N, bo[::2])
        assert bool((bo[1::2].contiguous().view(torch.uint8) == 0xFB).all())


# Sizes that take every cut of the rows; the 64-bit products run on the GPU.

def _spread(e, top, seed):
    c = torch.randint(0, top + 1, (e,), generator=gen(seed)).tolist()
    return [0, top, top - 1, 1, 16, 17, 33] + c[7:]


MANY = [
    # experts, most rows, H, N, group, act, bias, out
    (46, 256, 224, 2000, 16, "none", True, BF16),
    (33, 256, 288, 1000, 32, "silu_gated", False, F32),
    (20, 700, 160, 2056, 16, "silu", False, BF16),
    (12, 256, 416, 1096, 16, "silu_gated", True, BF16),
    (70, 64, 96, 1288, 32, "none", False, F32),
    (9, 128, 544, 2312, 16, "silu_gated", False, BF16),
    (3, 1500, 1056, 3200, 32, "gelu", True, F32),
    (64, 16, 1184, 1024, 16, "silu_gated", False, BF16),
    (40, 31, 2048, 1544, 32, "none", True, BF16),
]


@pytest.mark.parametrize("e,top,H,N,group,act,bias,out", MANY)
def test_expert_matmul_w4_on_larger_tiles(e, top, H, N, group, act, bias, out):
    say(f"[experts w4, larger] e={e} rows<={top} H={H} N={N} /{group} {act} {out}")
    counts = _spread(e, top, e)[:e]
    n, x, w, s, b, f = _experts(counts, top + 3, H, N, group, act, bias, True, 60)
    o = _marked((e, top + 3, N), out)
    x, w, s, b, f = (_to(t) for t in (x, w, s, b, f))
    B.moe_ep_expert_matmul_w4(x, w, s, torch.tensor(counts, dtype=torch.int32, device=DEV), o,
                              group, act, b, f)
    torch.cuda.synchronize()
    _check_experts(n, x, w, s, b, f, group, act, N, o, DEV)


@pytest.mark.parametrize("T,H,N,group,act,bias,residual,out", [
    (4096, 1056, 2048, 16, "silu_gated", True, True, BF16),
    (2051, 4128, 2056, 32, "none", False, True, BF16),
    (8191, 288, 1544, 16, "none", True, False, F32),
    (700, 2080, 1288, 16, "gelu", True, True, F32),
    (1023, 544, 520, 32, "silu_gated", False, False, BF16),
    (130, 4128, 4104, 16, "none", False, True, F32),
    (20000, 96, 264, 32, "silu", True, False, BF16),
    (48, 4096, 5120, 16, "silu_gated", False, False, BF16),
])
def test_matmul_w4_on_larger_tiles(T, H, N, group, act, bias, residual, out):
    say(f"[matmul w4, larger] T={T} H={H} N={N} /{group} {act} {out}")
    x, w, s, b, r, f = (_to(t) for t in _dense(T, H, N, group, act, bias, residual, out, True, 70))
    o = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    B.moe_ep_matmul_w4(x, w, s, o, group, act, b, r, f)
    torch.cuda.synchronize()
    y, e = _ref(x, w, s, b, r, f, group, act, N)
    assert_close(o, y.cpu(), e.cpu(), (T, H, N))


def test_w4_products_do_not_depend_on_what_lies_beside_them():
    """A row's result is the same bits whatever the other groups and rows of
    the same tile cut hold."""
    say("[experts w4] independence")
    counts, rows, H, N = [200, 40, 0, 256, 9], 256, 288, 520
    n, x, w, s, _, _ = _experts(counts, rows, H, N, 16, "none", False, False, 80)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    outs = []
    for fill in (float("nan"), 3.0):
        xx = x.clone()
        for i, c in enumerate(n):
            xx[i, c:] = fill
        o = _marked((5, rows, N), F32)
        B.moe_ep_expert_matmul_w4(_to(xx), _to(w), _to(s), cnt, o)
        B.moe_ep_expert_matmul_w4(_to(xx), _to(w), _to(s), cnt, o)  # again over its own output
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8))


def _calls():
    """Calls of both products with their outputs (in device buffers)."""
    made, outs = [], []
    for T, group, act in ((1, 16, "silu_gated"), (12, 32, "none"), (90, 16, "silu_gated")):
        x, w, s, b, r, f = (_to(t) for t in _dense(T, 288, 136, group, act, True, True, BF16, True,
                                                   21))
        o = torch.empty(T, 136, dtype=BF16, device=DEV)
        made.append(lambda st, x=x, w=w, s=s, b=b, r=r, f=f, o=o, group=group, act=act:
                    B.moe_ep_matmul_w4(x, w, s, o, group, act, b, r, f, st))
        outs.append(o)
    for counts, rows in (([70, 0, 300, 9], 304), ([3, 0, 16, 1], 16)):
        n, x, w, s, b, f = _experts(counts, rows, 288, 136, 16, "none", True, True, 22)
        x, w, s, b, f = (_to(t) for t in (x, w, s, b, f))
        cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
        o = torch.zeros(4, rows, 136, dtype=F32, device=DEV)
        made.append(lambda st, x=x, w=w, s=s, b=b, f=f, o=o, cnt=cnt:
                    B.moe_ep_expert_matmul_w4(x, w, s, cnt, o, 16, "none", b, f, st))
        outs.append(o)

    def go(stream=None):
        for call in made:
            call(stream)

    return go, outs


def test_w4_graph_replays_and_side_streams_give_the_eager_bytes():
    say("[w4] graph and streams")
    go, outs = _calls()
    go()
    torch.cuda.synchronize()
    eager = [o.contiguous().view(torch.uint8).clone() for o in outs]
    same = lambda: all(torch.equal(a, o.contiguous().view(torch.uint8))
                       for a, o in zip(eager, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    go(side)
    side.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for rep in range(4):
        for o in outs[:3]:                      # written in full
            o.view(torch.uint8).fill_(0xAB)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(), rep


def test_w4_counts_change_between_replays():
    """A captured product reads the counts of the replay, not of the capture."""
    say("[experts w4] counts between replays")
    rows, H, N = 300, 160, 72
    n, x, w, s, _, _ = _experts([300, 300], rows, H, N, 32, "none", False, False, 31)
    dx, dw, ds = _to(x), _to(w), _to(s)
    cnt = torch.zeros(2, dtype=torch.int32, device=DEV)
    o = _marked((2, rows, N), F32)
    g = torch.cuda.CUDAGraph()
    B.moe_ep_expert_matmul_w4(dx, dw, ds, cnt, o, 32)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.moe_ep_expert_matmul_w4(dx, dw, ds, cnt, o, 32)
    for counts in ([0, 3], [300, 0], [65, 257], [0, 0], [16, 17]):
        o.view(torch.uint8).fill_(0xFB)
        cnt.copy_(torch.tensor(counts, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check_experts(counts, x, w, s, None, None, 32, "none", N, o)


def test_w4_two_calls_at_once():
    """Calls on two streams at the same time have nothing in common."""
    say("[w4] two streams")
    go, outs = _calls()
    go()
    go2, outs2 = _calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for o in (outs2[0], outs2[1], outs2[2]):
            o.view(torch.uint8).fill_(0xAB)
        torch.cuda.synchronize()
        go(streams[0])
        go2(streams[1])
        torch.cuda.synchronize()
        for a, b in zip(outs, outs2):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
