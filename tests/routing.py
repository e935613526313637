"""Plain 64-bit forms of a router's training terms, with bounds on how far the
fp32 exponentials and sums may be from them.

Bounds, with u = 2^-23 (a whole last place; a rounding is off by half of it).
An exponential's argument is one difference, off by half a place, and the
exponential by two places; scaling by the largest logit's own and the division
add a few more, and the sum of E terms E / 64 + 6 additions. So a score q is
off by a factor of at most 1 +- u (|x| + |m| + D + E / 64 + 24), with m the
largest logit and D the mean of |x| + |m| under the scores (the sum's share),
and by 2^-126 where an exponential underflows."""
import math

import torch

U = 2.0 ** -23


def clean(logits):
    """Logits as the operators take them: (values, which experts take part)."""
    x = logits.double()
    live = x > -math.inf                                     # false for NaN too
    x = x.clamp(max=torch.finfo(torch.float32).max)
    return torch.where(live, x, torch.zeros_like(x)), live


def scores64(logits, score):
    """(q, its bound, 1 - sigmoid(x) or 1) in float64."""
    x, live = clean(logits)
    low = torch.where(live, x, -math.inf)
    m = low.amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    if score == "softmax":
        p = torch.where(live, torch.exp(x - m), 0.0)
        rest = torch.ones_like(x)
        size = (x - m).abs()
    else:
        m = m.clamp(max=0.0)
        # times e^-m, so that far negative logits keep their ratios
        p = torch.where(x > 0, 1.0 / (1.0 + torch.exp(-x.abs())),
                        torch.exp(torch.where(x > 0, 0.0, x) - m) / (1.0 + torch.exp(-x.abs())))
        p = torch.where(live, p, 0.0)
        rest = torch.where(x > 0, torch.exp(-x.abs()), 1.0) / (1.0 + torch.exp(-x.abs()))
        size = x.abs() + m.abs()
    q = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    mean = (q * size).sum(dim=1, keepdim=True)
    e = q * U * (size + mean + logits.shape[1] / 64 + 24) + 2.0 ** -126
    return q, torch.where(live, e, 0.0), rest


def counted64(ids, E):
    return ((ids >= 0) & (ids < E)).any(dim=1)


def balance64(logits, ids, score, bounds):
    """(counts, tokens, mean, loss, bound of mean, bound of loss)"""
    T, E = logits.shape
    q, e, _ = scores64(logits, score)
    real = counted64(ids, E)
    q, e = q * real[:, None], e * real[:, None]
    S = len(bounds) - 1
    counts = torch.zeros(S, E, dtype=torch.int64)
    tokens = torch.zeros(S, dtype=torch.int64)
    mean, loss = torch.zeros(S, E).double(), torch.zeros(S).double()
    emean, eloss = torch.zeros(S, E).double(), torch.zeros(S).double()
    # additions of a block's tokens in fp32, over its waves and in them
    adds = max(32, -(-T // 256)) / 16 + 24 if T > 256 else T / 16 + 24
    for s in range(S):
        at = slice(bounds[s], max(bounds[s], bounds[s + 1]))
        pick = ids[at][(ids[at] >= 0) & (ids[at] < E)].long()
        counts[s] = torch.bincount(pick, minlength=E)
        tokens[s] = real[at].sum()
        n = max(1, int(tokens[s]))
        mean[s] = q[at].sum(dim=0) / n
        emean[s] = e[at].sum(dim=0) / n + mean[s] * U * adds
        share = counts[s].double() / max(1, int(counts[s].sum()))
        loss[s] = E * (share * mean[s]).sum()
        eloss[s] = E * (share * emean[s]).sum() + loss[s] * U
    return counts, tokens, mean, loss, emean, eloss


def grad64(logits, ids, score, renormalize, scale, grad_weights, bounds=None, counts=None,
           tokens=None, grad_loss=None):
    """(gradient of the logits, its bound) by the formulas, in float64."""
    T, E = logits.shape
    K = ids.shape[1]
    q, eq, rest = scores64(logits, score)
    x, live = clean(logits)
    real = counted64(ids, E)
    dx, e = torch.zeros(T, E).double(), torch.zeros(T, E).double()
    if grad_loss is not None:
        a = torch.zeros(T, E).double()
        for s in range(len(bounds) - 1):
            picks, n = int(counts[s].sum()), int(tokens[s])
            if picks and n:
                a[bounds[s]:max(bounds[s], bounds[s + 1])] = \
                    float(grad_loss[s]) * E * counts[s].double() / picks / n
        a = a * real[:, None]
        mean = (q * a).sum(dim=1, keepdim=True)
        emean = (eq * a.abs() + q * a.abs() * U * (E / 64 + 16)).sum(dim=1, keepdim=True)
        dx = q * (a - mean) * rest
        e = eq * (a - mean).abs() * rest + q * rest * (emean + 8 * U * (a.abs() + mean.abs()))
    if grad_weights is not None:
        got = (ids >= 0) & (ids < E)
        at = torch.where(got, ids, 0).long()
        got = got & live.gather(1, at)
        xp = x.gather(1, at)
        g = torch.where(got, grad_weights.double(), 0.0)
        if score == "softmax":
            top = torch.where(live, x, -math.inf).amax(dim=1, keepdim=True)
            w = torch.where(got, torch.exp(xp - top), 0.0)
        else:
            w = torch.where(got, 1.0 / (1.0 + torch.exp(-xp)), 0.0)
        ew = 0.0
        if renormalize:
            all_ = w.sum(dim=1, keepdim=True)
            w = torch.where(all_ > 0, w / all_, 0.0)
            g = g - (g * w).sum(dim=1, keepdim=True)
        elif score == "softmax":
            w = q.gather(1, at) * got
            ew = eq.gather(1, at) * got
        left = (1.0 / (1.0 + torch.exp(xp))) if score == "sigmoid" else torch.ones_like(xp)
        back = torch.where(got, scale * w * g * left, 0.0)
        eback = (scale * g).abs() * ew + 2 * U * back.abs()
        dx = dx.scatter_add(1, at, back)
        # a pick's terms are added one by one
        e = e.scatter_add(1, at, eback + K * U * back.abs()) + U * dx.abs()
        if score == "softmax" and not renormalize:
            total, etotal = back.sum(dim=1, keepdim=True), eback.sum(dim=1, keepdim=True)
            etotal = etotal + 8 * U * back.abs().sum(dim=1, keepdim=True)
            dx = dx - q * total
            e = e + eq * total.abs() + q * (etotal + 8 * U * total.abs())
    return torch.where(live, dx, 0.0), e


def definition64(x, ids, score, renormalize, scale, grad_weights, bounds, counts, tokens,
                 grad_loss):
    """The scalar whose gradient the backward pass gives, as a function of
    float64 logits (finite ones; autograd and differences go through it)."""
    E = x.shape[1]
    p = torch.softmax(x, dim=1) if score == "softmax" else torch.sigmoid(x)
    q = p / p.sum(dim=1, keepdim=True)
    got = (ids >= 0) & (ids < E)
    total = x.new_zeros(())
    if grad_weights is not None:
        w = torch.where(got, p.gather(1, torch.where(got, ids, 0).long()), 0.0)
        if renormalize:
            w = w / torch.where(got.any(dim=1, keepdim=True), w.sum(dim=1, keepdim=True), 1.0)
        total = total + (torch.where(got, grad_weights.double(), 0.0) * scale * w).sum()
    if grad_loss is not None:
        q = q * got.any(dim=1, keepdim=True)
        for s in range(len(bounds) - 1):
            n, picks = max(1, int(tokens[s])), max(1, int(counts[s].sum()))
            mean = q[bounds[s]:max(bounds[s], bounds[s + 1])].sum(dim=0) / n
            total = total + grad_loss[s].double() * E * (counts[s].double() / picks * mean).sum()
    return total
