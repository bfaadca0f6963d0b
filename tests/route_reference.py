"""The experts' router and its gradient in 64 bits on the CPU, token by token from the
definition (test helper)."""
import math

import torch


def choose(x, k, mask=None):
    """(experts, order of the slots, place, counts, offsets) of logits x (a CPU tensor)."""
    T, E = x.shape
    experts = []
    for t in range(T):
        row = [(float("-inf") if math.isnan(v) else v) for v in x[t].double().tolist()]
        there = [e for e in range(E) if row[e] > -math.inf and (mask is None or bool(mask[t]))]
        best = sorted(there, key=lambda e: (-row[e], e))[:k]
        experts.append(best + [-1] * (k - len(best)))
    flat = [e if e >= 0 else E for row in experts for e in row]
    order = sorted(range(len(flat)), key=lambda s: flat[s])
    place = [0] * len(flat)
    for i, s in enumerate(order):
        place[s] = i
    counts = [flat.count(e) for e in range(E)]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return (torch.tensor(experts, dtype=torch.int32).reshape(T, k), torch.tensor(order, dtype=torch.int32),
            torch.tensor(place, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32),
            torch.tensor(offsets, dtype=torch.int32))


def softmax_parts(x, experts, normalize, mask=None):
    """(p, lse, weights) in 64 bits; tokens that do not count: p = 0, lse = +inf."""
    x = x.double()
    dead = ~(x > -math.inf).any(1) if mask is None else ~((x > -math.inf).any(1) & mask.bool())
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    p[dead] = 0.0
    lse = torch.where(dead, torch.full_like(lse, math.inf), lse)
    at, none = experts.long().clamp_min(0), experts < 0
    w = torch.gather(p, 1, at).masked_fill(none, 0.0)
    if normalize:
        chosen = torch.gather(x, 1, at).masked_fill(none, -math.inf)
        w = torch.softmax(chosen.masked_fill(dead[:, None], 0.0), 1).masked_fill(none, 0.0)
    return p, lse, w


def losses(p, lse, counts):
    live = lse != math.inf
    n = max(1, int(live.sum()))
    share = counts.double() / max(1, int(counts.sum()))
    return p.shape[1] * (share * p.sum(0)).sum() / n, (lse[live] ** 2).sum() / n


def gradient(x, experts, counts, normalize, dw, balance, z, mask=None):
    """(gradient in x, magnitudes of what it is a sum of)"""
    p, lse, w = softmax_parts(x, experts, normalize, mask)
    live = lse != math.inf
    n = max(1, int(live.sum()))
    g = balance * p.shape[1] * counts.double() / max(1, int(counts.sum())) / n
    zl = torch.where(live, 2 * z / n * lse, torch.zeros_like(lse))[:, None]
    d = p * (g - (p * g).sum(1, keepdim=True) + zl)
    size = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True) + zl.abs())
    if dw is not None:
        none = experts < 0
        back = (w * dw.double()).masked_fill(none, 0.0)
        at = experts.long().clamp_min(0)
        all_, alls = back.sum(1, keepdim=True), back.abs().sum(1, keepdim=True)
        if normalize:
            d.scatter_add_(1, at, (back - w * all_).masked_fill(none, 0.0))
            size.scatter_add_(1, at, (back.abs() + w * alls).masked_fill(none, 0.0))
        else:
            d.scatter_add_(1, at, back)
            d -= p * all_
            size.scatter_add_(1, at, back.abs())
            size += p * alls
    return d, size
