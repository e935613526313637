"""Cases of the operators around the dispatch/combine path: the router's
choice of experts (moe_ep_route_topk), the experts' products over the batched
rows in bf16 and in fp8 e4m3 (moe_ep_expert_matmul, moe_ep_expert_matmul_fp8)
and the products over all tokens of a rank (moe_ep_matmul: the router's
logits, an expert that every token passes through, its residual).

run() computes a case in its plain form, or with `own` set through the
package's binding. Sizes: H, E, K and the rows per expert are those of the
five workloads of workloads.py (decode: 128 tokens on each of 32 ranks, 8 of
256 experts a rank, so about 115 rows an expert; prefill: 32 experts a rank);
the experts' inner width, 2048, is generic.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
BLOCK = 128          # columns of x, and rows and columns of w, under one fp8 scale


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the router of a decode step: 128 tokens, sigmoid scores with a
        # selection bias, 4 of 8 expert groups
        dict(name="route_decode", op="route", T=128, E=256, K=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, dtype="f32", masked=0.0),
        # the router of a prefill batch: softmax over bf16 logits, some experts
        # masked out and some tokens with no expert left
        dict(name="route_prefill", op="route", T=8192, E=256, K=8, score="softmax", bias=False,
             n_group=1, topk_group=1, dtype="bf16", masked=0.05),
        # router logits of a decode step: few output columns, a long sum
        dict(name="logits_decode", op="matmul", T=128, Kd=7168, N=256, act="none", bias=False,
             residual=False, out="f32"),
        # one token through an expert that every token passes through
        dict(name="shared_up_one_token", op="matmul", T=1, Kd=7168, N=2048, act="silu_gated",
             bias=False, residual=False, out="bf16"),
        # the same expert at prefill: gate and up in one product
        dict(name="shared_up_prefill", op="matmul", T=4096, Kd=7168, N=2048, act="silu_gated",
             bias=False, residual=False, out="bf16"),
        # its second product, added to the combine's output; odd token count
        dict(name="shared_down_residual", op="matmul", T=8191, Kd=2048, N=7168, act="none",
             bias=True, residual=True, out="bf16"),
        # a handful of rows on one rank: most experts have none or one
        dict(name="experts_few_rows", op="experts", e_local=8, cap=32, mean=1.0, zipf=0.0,
             Kd=7168, N=2048, act="silu_gated", bias=False, out="bf16"),
        # decode: about 115 rows an expert, bound by the weights' bytes
        dict(name="experts_decode_up", op="experts", e_local=8, cap=256, mean=115.0, zipf=0.0,
             Kd=7168, N=2048, act="silu_gated", bias=False, out="bf16"),
        # prefill under skewed routing, both products
        dict(name="experts_prefill_up", op="experts", e_local=32, cap=1280, mean=512.0, zipf=0.6,
             Kd=7168, N=2048, act="silu_gated", bias=False, out="bf16"),
        dict(name="experts_prefill_down", op="experts", e_local=32, cap=1280, mean=512.0,
             zipf=0.6, Kd=2048, N=7168, act="none", bias=True, out="bf16"),
        # fp8 rows as the quantising pack sends them: decode's second product
        dict(name="experts_fp8_decode_down", op="experts_fp8", e_local=8, cap=256, mean=115.0,
             zipf=0.0, Kd=2048, N=7168, act="none", bias=False, out="bf16"),
        # and prefill's first, quantised again for the second
        dict(name="experts_fp8_prefill_up", op="experts_fp8", e_local=32, cap=1280, mean=512.0,
             zipf=0.6, Kd=7168, N=2048, act="silu_gated", bias=False, out="e4m3"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(step, min(hi, int(v)) // step * step)


def draw(rng):
    op = rng.choice(["route", "matmul", "experts", "experts_fp8"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        n_group = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        topk_group = rng.randint(1, n_group)
        return dict(op=op, T=_log(rng, 1, 8192), E=E,
                    K=rng.randint(1, min(10, topk_group * (E // n_group))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    n_group=n_group, topk_group=topk_group, dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.choice([0.0, 0.05, 0.5]))
    act = rng.choice(["none", "silu", "gelu", "silu_gated", "silu_gated"])
    if op == "matmul":
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), Kd=_log(rng, 128, 8192, 8),
                     N=_log(rng, 8, 7168, 8), act=act, bias=rng.random() < 0.5,
                     residual=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
            if work(c)["flops"] <= 2.4e11:
                return c
    while True:
        c = dict(op=op, e_local=_log(rng, 1, 32), cap=_log(rng, 16, 4096), mean=0.0,
                 zipf=rng.choice([0.0, 0.6, 1.1]), act=act, bias=rng.random() < 0.5,
                 Kd=_log(rng, 128, 8192, 128 if op == "experts_fp8" else 8),
                 N=_log(rng, 128, 7168, 128 if op == "experts_fp8" else 8),
                 out=rng.choice(["bf16", "f32"] + (["e4m3"] if op == "experts_fp8" else [])))
        c["mean"] = round(c["cap"] * rng.uniform(0.05, 0.7), 2)
        if c["e_local"] * c["cap"] * _rows_of_w(c) * c["Kd"] <= 32 * 1280 * 4096 * 7168:
            return c


def _rows_of_w(c):
    return c["N"] * (2 if c["act"] == "silu_gated" else 1)


def _counts(c):
    """Rows per expert: `mean` on average, spread over the experts by their
    popularity (rank^-zipf), the smaller ones odd. Sizes, so made from the
    case alone, as a step's routing makes them."""
    e = c["e_local"]
    pop = [(i + 1.0) ** -c["zipf"] for i in range(e)]
    total = sum(pop)
    cnt = [min(c["cap"], int(c["mean"] * e * p / total + ((i * 7) % 5 - 2) *
                             0.4 * math.sqrt(c["mean"]))) for i, p in enumerate(pop)]
    cnt = [max(0, n) for n in cnt]
    return [cnt[(i * 5 + 3) % e] if math.gcd(5, e) == 1 else cnt[i] for i in range(e)]


def work(c):
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (4 if c["dtype"] == "f32" else 2) + c["K"] * 8) +
                (4 * c["E"] if c["bias"] else 0),
                "flops": c["T"] * c["E"] * 4.0}
    nw, kd, n = _rows_of_w(c), c["Kd"], c["N"]
    ob = {"bf16": 2, "f32": 4, "e4m3": 1}[c["out"]]
    if c["op"] == "matmul":
        t = c["T"]
        return {"bytes": 2 * t * kd + 2 * nw * kd + ob * t * n * (2 if c["residual"] else 1) +
                (4 * nw if c["bias"] else 0),
                "flops": 2.0 * t * nw * kd}
    cnt = _counts(c)
    rows, used = sum(cnt), sum(x > 0 for x in cnt)
    eb = 1 if c["op"] == "experts_fp8" else 2
    b = rows * kd * eb + used * nw * kd * eb + rows * n * ob + 4 * len(cnt)
    if eb == 1:
        b += rows * kd // BLOCK * 4 + used * -(-nw // BLOCK) * (kd // BLOCK) * 4
    if c["out"] == "e4m3":
        b += rows * n // BLOCK * 4
    return {"bytes": b + (4 * used * nw if c["bias"] else 0), "flops": 2.0 * rows * nw * kd}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pitch(columns):
    """fp32 scales of a row: one per 128 columns, padded to 4."""
    return (columns // BLOCK + 3) // 4 * 4


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype).mul_(std)

    s = dict(case=c)
    if c["op"] == "route":
        t, e = c["T"], c["E"]
        logits = normal(t, e)
        if c["masked"]:
            logits[torch.rand((t, e), generator=g, device=dev) < c["masked"]] = -math.inf
            logits[torch.rand((t,), generator=g, device=dev) < 0.02] = -math.inf   # no expert left
        s["logits"] = logits.to(torch.bfloat16) if c["dtype"] == "bf16" else logits
        s["bias"] = normal(e, std=0.1) if c["bias"] else None
        s["ids"] = torch.empty((t, c["K"]), dtype=torch.int32, device=dev)
        s["weights"] = torch.empty((t, c["K"]), dtype=torch.float32, device=dev)
        return s
    nw, kd, n = _rows_of_w(c), c["Kd"], c["N"]
    out_t = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}[c["out"]]
    if c["op"] == "matmul":
        t = c["T"]
        s["x"] = normal(t, kd, dtype=torch.bfloat16)
        s["w"] = normal(nw, kd, dtype=torch.bfloat16, std=kd ** -0.5)
        s["bias"] = normal(nw) if c["bias"] else None
        s["residual"] = normal(t, n, dtype=out_t) if c["residual"] else None
        s["out"] = torch.zeros((t, n), dtype=out_t, device=dev)
        return s
    e, cap = c["e_local"], c["cap"]
    s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
    x = normal(e, cap, kd, dtype=torch.bfloat16)
    w = normal(e, nw, kd, dtype=torch.bfloat16, std=kd ** -0.5)
    s["bias"] = normal(e, nw) if c["bias"] else None
    if c["op"] == "experts_fp8":
        b = kd // BLOCK
        amax = x.view(e, cap, b, BLOCK).abs().amax(dim=3).float()
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        s["x"] = torch.empty((e, cap, kd), dtype=E4M3, device=dev)
        s["x_scale"] = torch.zeros((e, cap, _pitch(kd)), dtype=torch.float32, device=dev)
        s["x_scale"][:, :, :b] = scale
        s["w"] = torch.empty((e, nw, kd), dtype=E4M3, device=dev)
        # one scale per 128 rows (of each half, when gate and up are stacked) and 128 columns
        halves, per = nw // n, -(-n // BLOCK)
        s["w_scale"] = (torch.rand((e, halves * per, b), generator=g, device=dev) + 0.5) * 2.0 ** -8
        for i in range(e):
            q = x[i].float().view(cap, b, BLOCK) / scale[i][:, :, None]
            s["x"][i] = q.clamp(-448.0, 448.0).view(cap, kd).to(E4M3)
            s["w"][i] = (w[i].float() * 2.0 ** 8).clamp(-448.0, 448.0).to(E4M3)
    else:
        s["x"], s["w"] = x, w
    s["out"] = torch.zeros((e, cap, n), dtype=out_t, device=dev)
    s["out_scale"] = (torch.zeros((e, cap, _pitch(n)), dtype=torch.float32, device=dev)
                      if c["out"] == "e4m3" else None)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"] == "route":
        return _plain_route(s, c)
    if c["op"] == "matmul":
        y = s["x"].float() @ s["w"].float().t()
        y = _plain_act(y if s["bias"] is None else y + s["bias"], c)
        s["out"].copy_(y if s["residual"] is None else y + s["residual"].float())
        return s["out"]
    return _plain_experts(s, c)


def _own(s, c):
    from combine_topk_ids_dest_amd import binding as B
    if c["op"] == "route":
        B.moe_ep_route_topk(s["logits"], s["ids"], s["weights"], score=c["score"], bias=s["bias"],
                            n_group=c["n_group"], topk_group=c["topk_group"], renormalize=True,
                            scale=2.5)
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "matmul":
        B.moe_ep_matmul(s["x"], s["w"], s["out"], act=c["act"], bias=s["bias"],
                        residual=s["residual"])
        return s["out"]
    if c["op"] == "experts":
        B.moe_ep_expert_matmul(s["x"], s["w"], s["counts"], s["out"], act=c["act"],
                               bias=s["bias"])
        return s["out"]
    B.moe_ep_expert_matmul_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["counts"], s["out"],
                               act=c["act"], bias=s["bias"], out_scale=s["out_scale"])
    return s["out"] if s["out_scale"] is None else {"out": s["out"], "scale": s["out_scale"]}


def _plain_act(y, c):
    if c["act"] == "silu":
        return y * torch.sigmoid(y)
    if c["act"] == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    if c["act"] == "silu_gated":
        gate, up = y[..., :c["N"]], y[..., c["N"]:]
        return gate * torch.sigmoid(gate) * up
    return y


def _plain_route(s, c):
    # scores in 64 bits, rounded once: whichever expert wins at a near tie
    # goes by the rounded score, and by the lower index at a tie
    x = s["logits"].double()
    t, e = x.shape
    left = x > -math.inf
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(dim=1, keepdim=True).clamp(min=-1e30))
        p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    choice = p.float() if s["bias"] is None else p.float() + s["bias"]
    choice = choice.masked_fill(~left, -math.inf)
    if c["n_group"] > 1:
        by = choice.view(t, c["n_group"], e // c["n_group"])
        if s["bias"] is None:
            of_group = by.amax(dim=2)
        else:
            two = by.topk(min(2, by.shape[2]), dim=2).values
            alone = two[:, :, 1:] == -math.inf        # one expert left: its value alone
            of_group = two[:, :, 0] + two[:, :, 1:].masked_fill(alone, 0.0).sum(dim=2)
        order = of_group.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        taken = torch.zeros((t, c["n_group"]), dtype=torch.bool, device=x.device)
        taken.scatter_(1, order, True)
        choice = by.masked_fill(~taken[:, :, None], -math.inf).reshape(t, e)
    best, order = choice.sort(dim=1, descending=True, stable=True)
    best, order = best[:, :c["K"]], order[:, :c["K"]]
    got = best > -math.inf
    w = p.gather(1, order) * got
    w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300) * 2.5
    s["ids"].copy_(torch.where(got, order, -1))
    s["weights"].copy_(w)
    return {"ids": s["ids"], "weights": s["weights"]}


def _plain_experts(s, c):
    x, w = s["x"].float(), s["w"].float()
    e, cap, kd = x.shape
    if c["op"] == "experts_fp8":
        b = kd // BLOCK
        x = (x.view(e, cap, b, BLOCK) * s["x_scale"][:, :, :b, None]).view(e, cap, kd)
        halves = w.shape[1] // c["N"]
        ws = s["w_scale"].view(e, halves, -1, b).repeat_interleave(BLOCK, dim=2)[:, :, :c["N"]]
        w = (w.view(e, halves, c["N"], b, BLOCK) * ws[..., None]).view(w.shape)
    y = torch.bmm(x, w.transpose(1, 2))
    y = _plain_act(y if s["bias"] is None else y + s["bias"][:, None, :], c)
    # rows behind an expert's last stay as they were
    left = (torch.arange(cap, device=x.device)[None, :] < s["counts"][:, None])[..., None]
    if s["out_scale"] is None:
        s["out"].copy_(torch.where(left, y, s["out"].float()))
        return s["out"]
    b = c["N"] // BLOCK
    y = y.view(e, cap, b, BLOCK)
    amax = y.abs().amax(dim=3)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (y / scale[..., None]).clamp(-448.0, 448.0).view(e, cap, c["N"])
    s["out"].copy_(torch.where(left, q, s["out"].float()))
    full = torch.zeros_like(s["out_scale"])
    full[:, :, :b] = scale
    s["out_scale"].copy_(torch.where(left, full, s["out_scale"]))
    return {"out": s["out"], "scale": s["out_scale"]}


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "route":
        return _exact_route(s, c)
    if c["op"] == "matmul":
        y = _exact_row(s["x"].double(), s["w"].double(), s["bias"], c)
        return y if s["residual"] is None else y + s["residual"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["x"].device)
    scale = None if s["out_scale"] is None else torch.zeros_like(s["out_scale"]).double()
    for i, n in enumerate(s["counts"].tolist()):
        if not n:
            continue
        x, w = s["x"][i, :n].double(), s["w"][i].double()
        if c["op"] == "experts_fp8":
            kb = torch.arange(c["Kd"], device=x.device) // BLOCK
            x = x * s["x_scale"][i, :n].double()[:, kb]
            row = torch.arange(w.shape[0], device=x.device)
            row = row // c["N"] * -(-c["N"] // BLOCK) + row % c["N"] // BLOCK
            w = w * s["w_scale"][i].double()[row][:, kb]
        y = _exact_row(x, w, None if s["bias"] is None else s["bias"][i], c)
        if scale is not None:
            a = y.view(n, -1, BLOCK).abs().amax(dim=2)
            a = torch.where(a > 0, a / 448.0, 1.0)
            scale[i, :n, :a.shape[1]] = a
            y = y / a.repeat_interleave(BLOCK, dim=1)
        out[i, :n] = y
    return out if scale is None else {"out": out, "scale": scale}


def _exact_row(x, w, bias, c):
    y = torch.mm(x, w.t().contiguous())
    if bias is not None:
        y += bias.double()
    if c["act"] == "silu_gated":
        a, b = y.chunk(2, dim=-1)
        return a / (1 + torch.exp(-a)) * b
    if c["act"] == "silu":
        return y / (1 + torch.exp(-y))
    if c["act"] == "gelu":
        return y * torch.special.ndtr(y)
    return y


def _exact_route(s, c):
    x = s["logits"].double().cpu()
    bias = torch.zeros(c["E"]).double() if s["bias"] is None else s["bias"].double().cpu()
    t, per = c["T"], c["E"] // c["n_group"]
    gone = x == -math.inf
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1).nan_to_num(0.0)
    v = (p + bias).masked_fill(gone, -math.inf).view(t, c["n_group"], per)
    if c["n_group"] > 1:
        top = v.sort(dim=2, descending=True).values
        mark = top[:, :, 0].clone()
        if s["bias"] is not None and per > 1:
            mark += top[:, :, 1].nan_to_num(neginf=0.0)
        keep = mark.argsort(dim=1, descending=True, stable=True).argsort(dim=1) < c["topk_group"]
        v = v.masked_fill(~keep[:, :, None], -math.inf)
    v = v.reshape(t, c["E"])
    ids = v.argsort(dim=1, descending=True, stable=True)[:, :c["K"]]
    w = p.gather(1, ids).masked_fill(v.gather(1, ids) == -math.inf, 0.0)
    total = w.sum(dim=1, keepdim=True)
    return {"ids": None, "weights": torch.where(total > 0, 2.5 * w / total, 0.0).cuda()}
