"""Plain 64-bit forms of the router's choice and of the products, with bounds
on how far fp32 sums and one rounding may be from them.

Bounds. A sum of n products of exact factors, added in fp32 in any order, is
off by at most n * u * sum |x_k w_k| with u the error of one addition; u is
taken as 2^-23 (a full last place, so that a truncating adder is covered).
An activation moves an error e by at most 1.13 e (the largest slope of silu
is 1.0999, of gelu 1.1290) and is itself good to 8 roundings of its operand;
gate * up adds the two factors' errors, each times the other factor. The
result is rounded once, by at most half a step: eps / 2 of its type."""
import math

import torch

U = 2.0 ** -23
SLOPE = 1.13


def act64(v, e, act, N):
    """(value, bound) of the activation of v +- e along the last dim."""
    if act == "none":
        return v, e
    if act == "silu":
        return v * torch.sigmoid(v), SLOPE * e + 8 * U * v.abs()
    if act == "gelu":
        y = 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
        return y, SLOPE * e + 8 * U * v.abs()
    g, up = v[..., :N], v[..., N:]
    eg, eu = e[..., :N], e[..., N:]
    s = g * torch.sigmoid(g)
    es = SLOPE * eg + 8 * U * g.abs()
    return s * up, es * (up.abs() + eu) + s.abs() * eu + U * (s * up).abs()


def product64(x, w, bias, act, N, residual=None, extra=0):
    """(value, bound before the last rounding) of act(x w^T + bias) +
    residual; x, w, bias, residual as float64 tensors of exact values; extra:
    further roundings that a factor of every term goes through."""
    v = x @ w.t()
    e = (x.shape[1] + extra) * U * (x.abs() @ w.abs().t())
    if bias is not None:
        v = v + bias
        e = e + U * v.abs()
    y, e = act64(v, e, act, N)
    if residual is not None:
        y = y + residual
        e = e + U * y.abs()
    return y, e


def allowed(y, e, dtype):
    """How far an output of dtype may be from the exact y, given its sum's
    bound e: one rounding on top (and the smallest subnormal's half)."""
    return e + (y.abs() + e) * torch.finfo(dtype).eps / 2 + 2.0 ** -134


def assert_close(got, y, e, what):
    tol = allowed(y, e, got.dtype)
    off = (got.double().cpu() - y).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((off / tol).max()))


def route64(logits, bias, K, score, n_group, topk_group, renormalize, scale):
    """(ids, weights) by the definition, token by token in plain Python on
    float64; the choice goes by the score rounded to fp32 plus the bias."""
    T, E = logits.shape
    x = logits.double()
    ids = torch.full((T, K), -1, dtype=torch.int32)
    wts = torch.zeros((T, K), dtype=torch.float64)
    top = torch.finfo(torch.float32).max
    per = E // n_group
    for t in range(T):
        row = [min(v, top) for v in x[t].tolist()]
        live = [e for e in range(E) if row[e] > -math.inf]     # false for NaN too
        if score == "softmax":
            m = max([row[e] for e in live], default=0.0)
            z = {e: math.exp(row[e] - m) for e in live}
            s = math.fsum(z.values())
            p = {e: z[e] / s for e in live}
        else:
            p = {e: 1.0 / (1.0 + math.exp(-row[e])) if row[e] > -700 else math.exp(max(row[e], -745.0))
                 if row[e] >= -745 else 0.0 for e in live}
        pf = {e: torch.tensor(p[e], dtype=torch.float64).float() for e in live}
        c = {e: float(pf[e] if bias is None else pf[e] + bias[e]) for e in live}
        c = {e: v for e, v in c.items() if v > -math.inf}
        if n_group > 1:
            mark = {}
            for g in range(n_group):
                best = sorted((c[e] for e in range(g * per, (g + 1) * per) if e in c),
                              reverse=True)
                if best:
                    two = best[:1] if bias is None else best[:2]
                    mark[g] = float(torch.tensor(two, dtype=torch.float32).sum())
            keep = sorted(mark, key=lambda g: (-mark[g], g))[:topk_group]
            c = {e: v for e, v in c.items() if e // per in keep}
        pick = sorted(c, key=lambda e: (-c[e], e))[:K]
        total = math.fsum(p[e] for e in pick)
        for k, e in enumerate(pick):
            w = p[e]
            if renormalize:
                w = w / total if total > 0 else 0.0
            ids[t, k] = e
            wts[t, k] = w * scale
    return ids, wts
