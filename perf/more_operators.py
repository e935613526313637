"""Cases of two further sets of operators around the dispatch/combine path: a
router in training (moe_ep_balance_loss: per-expert counts, mean scores and the
balance loss of each sequence; moe_ep_route_backward: the gradient of the
logits, from the picks' weights and from that loss) and products with 4-bit
weights (moe_ep_matmul_w4 over all tokens of a rank, moe_ep_expert_matmul_w4
over the batched rows: E2M1 codes, with an E4M3 scale per 16 columns or a power
of two per 32, and fp32 factors over a whole matrix).

run() computes a case in its plain form, or with `own` set through the
package's binding. Sizes: H, E, K and the rows per expert are those of the
five workloads of workloads.py; the inner width of the experts, 2048, and the
training batches of 64k tokens are generic.
"""
import math

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # of E2M1 codes; bit 3 is the sign


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence of a micro-batch, sigmoid scores, fp32 logits
        dict(name="balance_one_sequence", op="balance", T=128, E=256, K=8, S=1, score="sigmoid",
             dtype="f32", masked=0.0),
        # a rank's batch of several ragged sequences with padding tokens and masked experts
        dict(name="balance_ragged", op="balance", T=8192, E=256, K=8, S=7, score="softmax",
             dtype="bf16", masked=0.05),
        # a long-context step: 64k tokens as one sequence
        dict(name="balance_long", op="balance", T=65536, E=256, K=8, S=1, score="softmax",
             dtype="f32", masked=0.0),
        # the same three through the router's backward pass
        dict(name="route_grad_one_sequence", op="route_grad", T=128, E=256, K=8, S=1,
             score="sigmoid", dtype="f32", masked=0.0, renormalize=True, weights=True, loss=True),
        dict(name="route_grad_ragged", op="route_grad", T=8192, E=256, K=8, S=7, score="softmax",
             dtype="bf16", masked=0.05, renormalize=True, weights=True, loss=True),
        dict(name="route_grad_long", op="route_grad", T=65536, E=256, K=8, S=1, score="softmax",
             dtype="f32", masked=0.0, renormalize=False, weights=True, loss=True),
        # one token through an expert that every token passes through
        dict(name="w4_up_one_token", op="matmul_w4", T=1, Kd=7168, N=2048, act="silu_gated",
             group=16, bias=False, residual=False, out="bf16"),
        # a few requests' tokens through its second product, added to the combine's output
        dict(name="w4_down_few_tokens", op="matmul_w4", T=13, Kd=2048, N=7168, act="none",
             group=32, bias=True, residual=True, out="bf16"),
        # decode with a handful of rows: most experts have none, one or two
        dict(name="experts_w4_few_rows", op="experts_w4", e_local=32, cap=32, mean=1.5, zipf=0.0,
             Kd=7168, N=2048, act="silu_gated", group=16, bias=False, out="bf16"),
        # decode: about 115 rows an expert, and its second product
        dict(name="experts_w4_decode_up", op="experts_w4", e_local=8, cap=256, mean=115.0, zipf=0.0,
             Kd=7168, N=2048, act="silu_gated", group=16, bias=False, out="bf16"),
        dict(name="experts_w4_decode_down", op="experts_w4", e_local=8, cap=256, mean=115.0,
             zipf=0.0, Kd=2048, N=7168, act="none", group=32, bias=False, out="f32"),
        # prefill under skewed routing
        dict(name="experts_w4_prefill_up", op="experts_w4", e_local=32, cap=1280, mean=512.0,
             zipf=0.6, Kd=7168, N=2048, act="silu_gated", group=16, bias=True, out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(step, min(hi, int(v)) // step * step)


def draw(rng):
    op = rng.choice(["balance", "route_grad", "matmul_w4", "experts_w4"])
    if op in ("balance", "route_grad"):
        T = _log(rng, 1, 65536)
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        c = dict(op=op, T=T, E=E, K=rng.randint(1, min(10, E)), S=_log(rng, 1, min(64, T)),
                 score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["f32", "bf16"]),
                 masked=rng.choice([0.0, 0.05, 0.5]))
        if op == "route_grad":
            weights, loss = rng.choice([(True, True), (True, True), (True, False), (False, True)])
            c.update(renormalize=rng.random() < 0.5, weights=weights, loss=loss)
        return c
    act = rng.choice(["none", "silu", "gelu", "silu_gated", "silu_gated"])
    c = dict(op=op, act=act, group=rng.choice([16, 32]), bias=rng.random() < 0.5,
             out=rng.choice(["bf16", "f32"]))
    while True:
        c.update(Kd=_log(rng, 128, 8192, 32), N=_log(rng, 8, 7168, 8))
        if op == "matmul_w4":
            c.update(T=_log(rng, 1, 8192), residual=rng.random() < 0.5)
            if work(c)["flops"] <= 2.4e11:
                return c
        else:
            c.update(e_local=_log(rng, 1, 32), cap=_log(rng, 16, 4096),
                     zipf=rng.choice([0.0, 0.6, 1.1]))
            c["mean"] = round(c["cap"] * rng.uniform(0.02, 0.7), 2)
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


def _bounds(c):
    """Where the sequences start, and behind them where the last one ends:
    ragged lengths, an empty one among many, a few tokens behind the last."""
    T, S = c["T"], c["S"]
    parts = [1 + (i * 7919) % 13 if i % 9 != 5 else 0 for i in range(S)]
    end, at, got = T - T // 50 if S > 1 else T, 0, [0]
    for p in parts:
        at += p
        got.append(end * at // sum(parts))
    return got


def _pitch(c):
    """Bytes of a row of scales: one per group, padded to 16."""
    return (c["Kd"] // c["group"] + 15) // 16 * 16


def work(c):
    if c["op"] in ("balance", "route_grad"):
        eb = 4 if c["dtype"] == "f32" else 2
        t, e, k, s = c["T"], c["E"], c["K"], c["S"]
        if c["op"] == "balance":
            return {"bytes": t * (e * eb + k * 4) + s * (e * 8 + 12), "flops": 5.0 * t * e}
        return {"bytes": t * (2 * e * eb + k * (8 if c["weights"] else 4)) +
                (s * (e * 4 + 12) if c["loss"] else 0), "flops": 8.0 * t * e}
    nw, kd, n = _rows_of_w(c), c["Kd"], c["N"]
    ob = 2 if c["out"] == "bf16" else 4
    matrix = nw * (kd // 2 + kd // c["group"]) + (4 * nw if c["bias"] else 0) + 4 * nw // n
    if c["op"] == "matmul_w4":
        t = c["T"]
        return {"bytes": 2 * t * kd + matrix + ob * t * n * (2 if c["residual"] else 1),
                "flops": 2.0 * t * nw * kd}
    cnt = _counts(c)
    rows, used = sum(cnt), sum(x > 0 for x in cnt)
    return {"bytes": rows * (2 * kd + ob * n) + used * matrix + 4 * len(cnt),
            "flops": 2.0 * rows * nw * kd}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _quantise(w, group):
    """Codes [rows, cols / 2] (the even column in the low nibble), scales
    [rows, cols / group] as bytes, and the factor over the whole matrix."""
    rows, cols = w.shape
    by = w.view(rows, cols // group, group)
    amax = by.abs().amax(dim=2)
    if group == 16:
        whole = amax.max() / (6.0 * 448.0)
        code = (amax / (6.0 * whole)).to(torch.float8_e4m3fn)
        scale, code = code.float(), code.view(torch.uint8)
    else:
        whole = torch.ones_like(amax.max())
        power = torch.floor(torch.log2(amax.clamp(min=1e-30))) - 2.0
        scale, code = torch.exp2(power), (power + 127.0).to(torch.uint8)
    v = by / (scale * whole).clamp(min=1e-30)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    q = torch.bucketize(v.abs(), edges).to(torch.uint8) + (v < 0).to(torch.uint8) * 8
    q = q.view(rows, cols)
    return q[:, 0::2] + q[:, 1::2] * 16, code, whole


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype).mul_(std)

    s = dict(case=c)
    if c["op"] in ("balance", "route_grad"):
        t, e, k, n = c["T"], c["E"], c["K"], c["S"]
        logits = normal(t, e) + normal(e, std=0.5)             # some experts are more popular
        if c["masked"]:
            logits[torch.rand((t, e), generator=g, device=dev) < c["masked"]] = -math.inf
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["logits"] = logits.to(dtype)
        top = logits.topk(k, dim=1)
        ids = torch.where(top.values > -math.inf, top.indices, -1).to(torch.int32)
        ids[torch.rand((t,), generator=g, device=dev) < 0.02] = -1     # padding tokens
        s["ids"] = ids
        bounds = _bounds(c)
        s["start"] = (None if n == 1 and bounds == [0, t] else
                      torch.tensor(bounds, dtype=torch.int32, device=dev))
        s["counts"] = torch.zeros((n, e), dtype=torch.int32, device=dev)
        s["tokens"] = torch.zeros((n,), dtype=torch.int32, device=dev)
        s["mean"] = torch.zeros((n, e), device=dev)
        s["loss"] = torch.zeros((n,), device=dev)
        if c["op"] == "balance":
            s["workspace"] = _workspace(c, dev)
            return s
        # the forward pass has left the counts; its own gradient comes from above
        for i in range(n):
            mine = ids[bounds[i]:bounds[i + 1]]
            s["counts"][i] = torch.bincount(mine[mine >= 0].long(), minlength=e).int()
            s["tokens"][i] = (mine >= 0).any(dim=1).sum().int()
        s["grad_weights"] = normal(t, k, std=0.1) if c["weights"] else None
        s["grad_loss"] = (torch.rand((n,), generator=g, device=dev) + 0.5) if c["loss"] else None
        s["grad"] = torch.zeros((t, e), dtype=dtype, device=dev)
        return s
    nw, kd, n = _rows_of_w(c), c["Kd"], c["N"]
    out_t = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    halves = nw // n
    lead = () if c["op"] == "matmul_w4" else (c["e_local"],)
    many = lead[0] if lead else 1
    w = torch.empty((many, nw, kd // 2), dtype=torch.uint8, device=dev)
    sc = torch.zeros((many, nw, _pitch(c)), dtype=torch.uint8, device=dev)
    whole = torch.empty((many, halves), device=dev)
    for i in range(many):
        for h in range(halves):
            at = slice(h * n, (h + 1) * n)
            w[i, at], sc[i, at, :kd // c["group"]], whole[i, h] = _quantise(
                normal(n, kd, std=kd ** -0.5), c["group"])
    rows = (c["T"],) if c["op"] == "matmul_w4" else (c["cap"],)
    s["x"] = normal(*lead, *rows, kd, dtype=torch.bfloat16)
    s["w"], s["scale"], s["whole"] = (w, sc, whole) if lead else (w[0], sc[0], whole[0])
    s["bias"] = normal(*lead, nw) if c["bias"] else None
    s["residual"] = normal(*rows, n, dtype=out_t) if c.get("residual") else None
    s["out"] = torch.zeros((*lead, *rows, n), dtype=out_t, device=dev)
    if lead:
        s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
    return s


def _workspace(c, dev):
    if not own:
        return None
    from combine_topk_ids_dest_amd import binding as B
    size = B.moe_ep_balance_workspace_bytes(c["T"], c["E"], c["S"])
    return torch.empty(max(size, 16), dtype=torch.uint8, device=dev)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"] == "balance":
        return _plain_balance(s, c)
    if c["op"] == "route_grad":
        return _plain_route_grad(s, c)
    return _plain_w4(s, c)


def _own(s, c):
    from combine_topk_ids_dest_amd import binding as B
    if c["op"] == "balance":
        B.moe_ep_balance_loss(s["logits"], s["ids"], s["counts"], s["tokens"], s["mean"],
                              s["loss"], s["workspace"], score=c["score"], seq_start=s["start"])
        return {k: s[k] for k in ("counts", "tokens", "mean", "loss")}
    if c["op"] == "route_grad":
        B.moe_ep_route_backward(s["logits"], s["ids"], s["grad"], score=c["score"],
                                renormalize=c["renormalize"], scale=2.5,
                                grad_weights=s["grad_weights"], grad_loss=s["grad_loss"],
                                counts=s["counts"] if c["loss"] else None,
                                tokens=s["tokens"] if c["loss"] else None,
                                seq_start=s["start"] if c["loss"] else None)
        return s["grad"]
    if c["op"] == "matmul_w4":
        B.moe_ep_matmul_w4(s["x"], s["w"], s["scale"], s["out"], group=c["group"], act=c["act"],
                           bias=s["bias"], residual=s["residual"], w_global=s["whole"])
        return s["out"]
    B.moe_ep_expert_matmul_w4(s["x"], s["w"], s["scale"], s["counts"], s["out"], group=c["group"],
                              act=c["act"], bias=s["bias"], w_global=s["whole"])
    return s["out"]


def _plain_scores(x, c):
    """Scores of each expert that sum to 1 over a token's experts (0 for one
    whose logit is -inf), and for sigmoid scores the ones before that."""
    x = x.float()
    left = x > -math.inf
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(dim=1, keepdim=True).clamp(min=-1e30)) * left
        raw = None
    else:
        p = raw = 1.0 / (1.0 + torch.exp(-x)) * left
    return p / p.sum(dim=1, keepdim=True).clamp(min=1e-30), raw


def _plain_balance(s, c):
    q, _ = _plain_scores(s["logits"], c)
    counted = (s["ids"] >= 0).any(dim=1)
    q = q * counted[:, None]
    bounds = _bounds(c)
    for i in range(c["S"]):
        at = slice(bounds[i], bounds[i + 1])
        ids = s["ids"][at].reshape(-1, 1)
        hit = torch.zeros((c["E"] + 1,), dtype=torch.int32, device=q.device)
        hit.index_add_(0, torch.where(ids < 0, c["E"], ids).flatten(),
                       torch.ones_like(ids).flatten())
        s["counts"][i] = hit[:-1]
        s["tokens"][i] = counted[at].sum()
        s["mean"][i] = q[at].sum(dim=0) / s["tokens"][i].clamp(min=1)
    share = s["counts"].float() / s["counts"].sum(dim=1, keepdim=True).clamp(min=1)
    s["loss"].copy_(c["E"] * (share * s["mean"]).sum(dim=1))
    return {k: s[k] for k in ("counts", "tokens", "mean", "loss")}


def _plain_route_grad(s, c):
    q, raw = _plain_scores(s["logits"], c)
    grad = torch.zeros_like(q)
    if c["loss"]:
        up = torch.zeros_like(q)                              # d loss / d score
        share = s["counts"].float() / s["counts"].sum(dim=1, keepdim=True).clamp(min=1)
        each = (c["E"] * s["grad_loss"] / s["tokens"].clamp(min=1))[:, None] * share
        bounds = _bounds(c)
        for i in range(c["S"]):
            up[bounds[i]:bounds[i + 1]] = each[i]
        up = up * (s["ids"] >= 0).any(dim=1, keepdim=True)
        grad = q * (up - (q * up).sum(dim=1, keepdim=True))
        if raw is not None:                                   # d q / d logit = q (1 - raw) (...)
            grad = grad * (1.0 - raw)
    if c["weights"]:
        got = s["ids"] >= 0
        at = torch.where(got, s["ids"], 0).long()
        w = (q if raw is None else raw).gather(1, at) * got
        g = s["grad_weights"] * 2.5
        if c["renormalize"]:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-30)
            g = g - (g * w).sum(dim=1, keepdim=True)
        back = w * g
        if raw is not None:
            back = back * (1.0 - raw.gather(1, at))
        grad = grad.scatter_add(1, at, back)
        if raw is None and not c["renormalize"]:
            grad = grad - q * back.sum(dim=1, keepdim=True)
    s["grad"].copy_(grad)
    return s["grad"]


def _plain_w4(s, c):
    dev = s["w"].device
    e2m1 = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=dev)
    pairs = torch.stack((e2m1.repeat(16), e2m1.repeat_interleave(16)), dim=1)     # of a byte
    w = pairs[s["w"].int()].flatten(-2)
    sc = s["scale"][..., :c["Kd"] // c["group"]].contiguous()
    sc = (sc.view(torch.float8_e4m3fn).float() if c["group"] == 16 else
          (sc.int() << 23).view(torch.float32))
    w = (w.view(*sc.shape, c["group"]) * sc[..., None]).view(w.shape)
    y = torch.matmul(s["x"].float(), w.transpose(-1, -2))
    y = y * s["whole"].repeat_interleave(c["N"], dim=-1).unsqueeze(-2)
    y = y if s["bias"] is None else y + s["bias"].unsqueeze(-2)
    if c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] == "silu_gated":
        gate, up = y[..., :c["N"]], y[..., c["N"]:]
        y = gate * torch.sigmoid(gate) * up
    if c["op"] == "matmul_w4":
        s["out"].copy_(y if s["residual"] is None else y + s["residual"].float())
        return s["out"]
    # rows behind an expert's last stay as they were
    left = (torch.arange(c["cap"], device=dev)[None, :] < s["counts"][:, None])[..., None]
    s["out"].copy_(torch.where(left, y, s["out"].float()))
    return s["out"]


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "balance":
        x = s["logits"].double()
        counts, tokens, mean, loss = _exact_balance(x, s, c)
        return {"counts": None, "tokens": None, "mean": mean, "loss": loss}
    if c["op"] == "route_grad":
        # by differentiating the definition
        x = s["logits"].double().requires_grad_(True)
        total = x.sum() * 0.0 if not c["masked"] else x.clamp(min=-1e300).sum() * 0.0
        if c["loss"]:
            _, _, _, loss = _exact_balance(x, s, c)
            total = total + (loss * s["grad_loss"].double()).sum()
        if c["weights"]:
            p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
            got = s["ids"] >= 0
            w = p.gather(1, s["ids"].clamp(min=0).long())
            w = torch.where(got, w, torch.zeros_like(w))
            if c["renormalize"]:
                all_ = w.sum(dim=1, keepdim=True)
                w = w / torch.where(all_ > 0, all_, torch.ones_like(all_))
            total = total + (2.5 * w * s["grad_weights"].double()).sum()
        total.backward()
        return torch.where(x.detach() > -math.inf, x.grad, 0.0)
    if c["op"] == "matmul_w4":
        y = _exact_row(s["x"], s["w"], s["scale"], s["whole"], s["bias"], c)
        return y if s["residual"] is None else y + s["residual"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["x"].device)
    for i, n in enumerate(s["counts"].tolist()):
        if n:
            out[i, :n] = _exact_row(s["x"][i, :n], s["w"][i], s["scale"][i], s["whole"][i],
                                    None if s["bias"] is None else s["bias"][i], c)
    return out


def _exact_balance(x, s, c):
    if c["score"] == "softmax":
        q = torch.softmax(x, dim=1)
    else:
        p = torch.sigmoid(x)
        q = p / p.sum(dim=1, keepdim=True)
    real = (s["ids"] > -1).sum(dim=1) > 0
    q = torch.where(real[:, None], q, torch.zeros_like(q))
    picked = torch.zeros((c["T"], c["E"]), dtype=torch.float64, device=x.device)
    for k in range(c["K"]):
        id_ = s["ids"][:, k:k + 1].long()
        picked += torch.zeros_like(picked).scatter_(1, id_.clamp(min=0), (id_ >= 0).double())
    counts, tokens, mean, loss = [], [], [], []
    b = _bounds(c)
    for lo, hi in zip(b[:-1], b[1:]):
        counts.append(picked[lo:hi].sum(dim=0))
        tokens.append(real[lo:hi].sum().double())
        mean.append(q[lo:hi].sum(dim=0) / max(1.0, float(tokens[-1])))
        loss.append(c["E"] * (counts[-1] / max(1.0, float(counts[-1].sum())) * mean[-1]).sum())
    return tuple(torch.stack(v) for v in (counts, tokens, mean, loss))


def _exact_row(x, w, scale, whole, bias, c):
    code = torch.stack((w & 15, w >> 4), dim=2).flatten(1).long()
    sign, power, half = code >> 3, (code >> 1) & 3, code & 1
    v = torch.where(power > 0, (1.0 + 0.5 * half.double()) * 2.0 ** (power.double() - 1.0),
                    0.5 * half.double()) * (1.0 - 2.0 * sign.double())
    cols = torch.arange(c["Kd"], device=w.device) // c["group"]
    sc = scale[:, :c["Kd"] // c["group"]].contiguous()
    sc = (sc.view(torch.float8_e4m3fn).double() if c["group"] == 16 else
          torch.exp2(sc.double() - 127.0))
    y = torch.mm(x.double(), (v * sc[:, cols]).t().contiguous())
    y = y * whole.double()[torch.arange(w.shape[0], device=w.device) // c["N"]]
    if bias is not None:
        y = y + bias.double()
    if c["act"] == "silu_gated":
        a, b = y.chunk(2, dim=-1)
        return a / (1 + torch.exp(-a)) * b
    if c["act"] == "silu":
        return y / (1 + torch.exp(-y))
    if c["act"] == "gelu":
        return y * torch.special.ndtr(y)
    return y
