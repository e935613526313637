"""GPU: the products with 4-bit weights in every kind of their tiles (which cases take
which is checked on the host by test_w4_choice.py): all codes and scales, bounds
against 64 bits, NaN and infinities, strided rows with the residual in place, bits
that neither a stream, a replay nor a neighbour changes."""
import math

import pytest
import torch

from combine_topk_ids_dest_amd import binding as B
from parity import say
from products import assert_close, product64
from w4 import pitch, random_w4, value64
from w4_cases import EXPERTS, H, TOKENS, WIDE_N

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def marked(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(0xFB)
    return t


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == 0xFB).all())


def factor(w64, f, N):
    return w64 * f.double().repeat_interleave(N, dim=-1).unsqueeze(-1)


@pytest.mark.parametrize("name", EXPERTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("group", [16, 32])
def test_every_code_with_every_scale(name, gated, group):
    """Rows of x that pick single columns, so that each output is one weight: all 16
    codes with the 256 scale codes, NaN ones among them, in turn over the rows of w.
    (Gated: times silu(64), which is 64, of a gate that is all bias.)"""
    counts, rows, N, Ng, _, _ = EXPERTS[name]
    N = Ng if gated else N
    e, K = len(counts), 16 * group
    say(f"[w4 tiles] codes and scales, {name} gated={gated} /{group}")
    codes = torch.arange(16, dtype=torch.uint8).repeat(group // 2)
    low = codes.repeat(2)[:K // 2]
    w = (low + low.flip(0) * 16).repeat(N, 1)
    s = torch.zeros((e, N, pitch(K, group)), dtype=torch.uint8)
    code = (torch.arange(N)[None, :] + 7 * torch.arange(e)[:, None]) % 256
    s[:, :, :K // group] = code[:, :, None].to(torch.uint8)
    g = gen(e + group)
    at = torch.randint(0, K, (e, rows), generator=g)
    x = torch.zeros(e, rows, K)
    x.scatter_(2, at[:, :, None], 1.0)
    for i, c in enumerate(counts):
        x[i, c:] = float("nan")
    ws, ss, bias = w.expand(e, N, K // 2), s, None
    if gated:
        ws = torch.cat((torch.zeros_like(ws), ws), dim=1)
        ss = torch.cat((torch.full_like(s, 0x38 if group == 16 else 127), s), dim=1)
        bias = torch.cat((torch.full((e, N), 64.0), torch.zeros(e, N)), dim=1).to(DEV)
    o = marked((e, rows, N), F32)
    B.moe_ep_expert_matmul_w4(x.to(BF16).to(DEV), ws.contiguous().to(DEV), ss.contiguous().to(DEV),
                              torch.tensor(counts, dtype=torch.int32, device=DEV), o, group,
                              "silu_gated" if gated else "none", bias)
    torch.cuda.synchronize()
    top = 255 if group == 16 else 252                # 6 * 2^125 is within bf16
    o, times = o.cpu(), 64.0 if gated else 1.0
    for i, c in enumerate(counts):
        w64 = value64(w, s[i], group)
        nan = torch.isnan(w64).any(dim=1)            # a NaN scale spoils its row of w
        fine = ~nan & (code[i] <= (top if not gated or group == 16 else top - 8))
        want = times * w64[:, at[i, :c]].t()[:, fine]
        got = o[i, :c].double()
        assert bool(torch.isnan(got[:, nan]).all()), i
        assert torch.equal(got[:, fine], want), (i, float((got[:, fine] - want).abs().max()))
        assert untouched(o[i, c:]), i


def operands(name, gated, group, seed=0, columns=H):
    """Host operands of an expert case: (counts, rows, N, x, w, s, bias, factors)."""
    counts, rows, N, Ng, _, _ = EXPERTS[name]
    N = Ng if gated else N
    e, halves = len(counts), 2 if gated else 1
    g = gen(seed + e + N + group)
    x = torch.full((e, rows, columns), float("nan"), dtype=BF16)
    for i, c in enumerate(counts):
        x[i, :c] = torch.randn(c, columns, generator=g).to(BF16)
    w, s = random_w4((e,), halves * N, columns, group, g)
    return (counts, rows, N, x, w, s, torch.randn(e, halves * N, generator=g),
            torch.rand(e, halves, generator=g) + 0.5)


@pytest.mark.parametrize("name", EXPERTS)
@pytest.mark.parametrize("act,out", [("none", F32), ("silu_gated", BF16), ("gelu", BF16),
                                     ("silu_gated", F32)])
@pytest.mark.parametrize("group", [16, 32])
def test_against_64_bits(name, act, out, group):
    say(f"[w4 tiles] {name} {act} {out} /{group}")
    gated = act == "silu_gated"
    # 17 groups of 32 columns: an odd number of every kind of step
    counts, rows, N, x, w, s, b, f = operands(name, gated, group, 5, 544 if out == F32 else H)
    o = marked((len(counts), rows, N), out)
    x, w, s, b, f = (t.to(DEV) for t in (x, w, s, b, f))
    B.moe_ep_expert_matmul_w4(x, w, s, torch.tensor(counts, dtype=torch.int32, device=DEV), o,
                              group, act, b, f)
    torch.cuda.synchronize()
    for i, c in enumerate(counts):
        if c:
            y, e = product64(x[i, :c].double(), factor(value64(w[i], s[i], group), f[i], N),
                             b[i].double(), act, N, extra=2)
            assert_close(o[i, :c], y.cpu(), e.cpu(), (name, i, c))
        assert untouched(o[i, c:]), i


@pytest.mark.parametrize("name", ["tall", "cut", "low"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("group", [16, 32])
def test_nan_and_infinities_stay_in_their_rows_and_columns(name, gated, group):
    """A row of NaN or with an infinity spoils that row of the output, a NaN scale
    that column."""
    say(f"[w4 tiles] non-finite, {name} gated={gated} /{group}")
    counts, rows, N, x, w, s, _, _ = operands(name, gated, group, 9)
    full = [i for i, c in enumerate(counts) if c >= 3]
    for i in full:
        x[i, counts[i] - 1] = float("nan")
        x[i, 1, 17] = math.inf
    w[:, :, 8] = 0x22                                # columns 16 and 17: 1 times their scale
    s[:, :, 16 // group] = 0x38 if group == 16 else 127
    s[:, N - 1, 3] = 0x7F if group == 16 else 0xFF
    o = marked((len(counts), rows, N), F32)
    dx, dw, ds = x.to(DEV), w.to(DEV), s.to(DEV)
    act = "silu_gated" if gated else "none"
    B.moe_ep_expert_matmul_w4(dx, dw, ds, torch.tensor(counts, dtype=torch.int32, device=DEV), o,
                              group, act)
    torch.cuda.synchronize()
    for i in full:
        c = counts[i]
        assert bool(torch.isnan(o[i, c - 1]).all()) and bool(torch.isnan(o[i, :c, N - 1]).all()), i
        assert bool((o[i, 1, :N - 1] == math.inf).all()), i
        keep = [r for r in range(c) if r not in (1, c - 1)]
        ok = torch.arange(dw.shape[1], device=DEV) != N - 1
        if gated:
            ok[2 * N - 1] = False
        y, e = product64(dx[i, keep].double(), value64(dw[i], ds[i], group)[ok], None, act, N - 1)
        assert_close(o[i, keep, :N - 1], y.cpu(), e.cpu(), (name, i, c))


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("gated,group,out", [(False, 16, BF16), (True, 16, F32), (False, 32, F32),
                                             (True, 32, BF16)])
def test_strided_rows_and_the_residual_in_place(T, gated, group, out):
    """Every operand a column range of a wider tensor whose other columns are NaN (or
    NaN scales); the residual is the output itself; nothing outside is written."""
    say(f"[w4 tiles] strided, in place, T={T} gated={gated} /{group}")
    N, halves, act = WIDE_N[gated], 2 if gated else 1, "silu_gated" if gated else "none"
    g = gen(T + group)
    x = torch.randn(T, H, generator=g).to(BF16)
    w, s = random_w4((), halves * N, H, group, g)
    s = s[:, :H // group]
    r = torch.randn(T, N, generator=g).to(out)
    b = torch.randn(halves * N, generator=g).to(DEV)
    f = (torch.rand(halves, generator=g) + 0.5).to(DEV)

    def wide(t, left, right, fill):
        big = torch.full((t.shape[0], left + t.shape[1] + right), fill, dtype=t.dtype, device=DEV)
        big[:, left:left + t.shape[1]] = t.to(DEV)
        return big, big[:, left:left + t.shape[1]]

    _, vx = wide(x, 8, 24, float("nan"))
    _, vw = wide(w, 16, 32, 0x77)
    _, vs = wide(s, 16, 48 - s.shape[1] % 16, 0x7F if group == 16 else 0xFF)
    bo, vo = wide(r, 8, 16, float("nan"))
    B.moe_ep_matmul_w4(vx, vw, vs, vo, group, act, b, vo, f)
    torch.cuda.synchronize()
    y, e = product64(vx.double(), factor(value64(vw, vs, group), f, N), b.double(), act, N,
                     r.to(DEV).double(), extra=2)
    assert_close(vo, y.cpu(), e.cpu(), T)
    assert bool(torch.isnan(bo[:, :8]).all()) and bool(torch.isnan(bo[:, 8 + N:]).all())


def calls():
    """A call of every case and token count, with their outputs."""
    made, outs = [], []
    for k, T in enumerate(TOKENS):
        gated, group = k % 2 == 1, (16, 32)[k // 2 % 2]
        N, halves = WIDE_N[gated], 2 if gated else 1
        g = gen(T)
        w, s = random_w4((), halves * N, H, group, g)
        x = torch.randn(T, H, generator=g).to(BF16).to(DEV)
        w, s = w.to(DEV), s.to(DEV)
        o = marked((T, N), BF16)
        made.append(lambda st, a=(x, w, s, o, group, "silu_gated" if gated else "none"):
                    B.moe_ep_matmul_w4(*a, stream=st))
        outs.append(o)
    for k, name in enumerate(EXPERTS):
        gated, group = k % 2 == 0, (32, 16)[k // 2 % 2]
        counts, rows, N, x, w, s, b, f = operands(name, gated, group, 3)
        cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
        x, w, s, b, f = (t.to(DEV) for t in (x, w, s, b, f))
        o = marked((len(counts), rows, N), F32)
        made.append(lambda st, a=(x, w, s, cnt, o, group, "silu_gated" if gated else "gelu", b, f):
                    B.moe_ep_expert_matmul_w4(*a, stream=st))
        outs.append(o)

    def go(stream=None):
        for call in made:
            call(stream)

    def clear():
        for o in outs:
            o.view(torch.uint8).fill_(0xFB)

    return go, clear, outs


def test_streams_replays_and_two_calls_at_once_give_the_eager_bytes():
    say("[w4 tiles] streams, graph, two at once")
    (go, clear, outs), (go2, clear2, outs2) = calls(), calls()
    go()
    torch.cuda.synchronize()
    eager = [o.clone() for o in outs]
    same = lambda have: all(torch.equal(a.view(torch.uint8), o.view(torch.uint8))
                            for a, o in zip(eager, have))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        clear(), clear2()
        torch.cuda.synchronize()
        go(streams[0])
        go2(streams[1])
        torch.cuda.synchronize()
        assert same(outs) and same(outs2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for rep in range(3):
        clear()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(outs), rep


def test_rows_behind_the_counts_do_not_change_a_bit():
    say("[w4 tiles] what lies behind the counts")
    for name in EXPERTS:
        for gated, group in ((False, 16), (True, 32)):
            counts, rows, N, x, w, s, _, _ = operands(name, gated, group, 80)
            w, s = w.to(DEV), s.to(DEV)
            cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
            outs = []
            for fill in (float("nan"), 3.0):
                for i, c in enumerate(counts):
                    x[i, c:] = fill
                o = marked((len(counts), rows, N), BF16)
                B.moe_ep_expert_matmul_w4(x.to(DEV), w, s, cnt, o, group,
                                          "silu_gated" if gated else "none")
                outs.append(o)
            torch.cuda.synchronize()
            assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8)), name


@pytest.mark.parametrize("rows", [32, 256])
def test_counts_that_change_between_replays_change_the_tiles(rows):
    """A captured product takes the tiles that the counts of the replay ask for."""
    say(f"[w4 tiles] counts between replays, room for {rows}")
    e, N, group = 40, 2056, 16
    g = gen(rows)
    x = torch.randn(e, rows, H, generator=g).to(BF16).to(DEV)
    w, s = (t.to(DEV) for t in random_w4((e,), N, H, group, g))
    w64 = [value64(w[i], s[i], group) for i in range(e)]
    cnt = torch.zeros(e, dtype=torch.int32, device=DEV)
    o = marked((e, rows, N), F32)
    graph = torch.cuda.CUDAGraph()
    B.moe_ep_expert_matmul_w4(x, w, s, cnt, o, group)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.moe_ep_expert_matmul_w4(x, w, s, cnt, o, group)
    for counts in ([0] * e, [rows] * e, [1] * e, [rows] + [0, 2] * 20, [17, 16, 0, 9] * 10):
        counts = counts[:e]
        o.view(torch.uint8).fill_(0xFB)
        cnt.copy_(torch.tensor(counts, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, c in enumerate(counts):
            if c:
                y, err = product64(x[i, :c].double(), w64[i], None, "none", N)
                assert_close(o[i, :c], y.cpu(), err.cpu(), (rows, i, c))
            assert untouched(o[i, c:]), i
