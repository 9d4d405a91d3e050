"""Plain 64-bit form of the draw on the CPU, for the tests. Written from the formulas of
include/lp_head.h, one row at a time, filters as sets of tokens."""

import math

import torch

SMALLEST = -40.0 * math.log(2.0)


def draw(x, u, tau=1.0, k=0, p=1.0, q=0.0):
    """(token, logprob, margin) of one row [V]: margin is how far, relative to the sums they are compared with,
    the nearest comparison that decides the token is from turning over (inf: none could), less the share of the
    weights below the smallest, which sums may hold or not."""
    x = x.double() + 0.0
    V = x.numel()
    m = float(x.max()) if V else math.nan
    if not math.isfinite(m):
        return None, math.nan, math.inf
    if tau == 0.0:
        return int((x == m).nonzero()[0]), 0.0, math.inf
    margin = math.inf
    d = (x - m) / tau
    w = torch.where(d >= SMALLEST, torch.exp(d), torch.zeros_like(d))
    light = float(torch.exp(d[d < SMALLEST]).sum()) / float(w.sum())
    order = torch.sort(x, descending=True, stable=True).indices
    if 0 < k < V:
        order = order[:k]
    if p < 1.0:
        ws = w[order]
        upto = torch.cumsum(ws, 0)
        before = upto - ws
        before[1:] = upto[:-1]
        want = p * float(upto[-1])
        stay = before < want
        stay[0] = True
        if len(order) > 1:
            margin = min(margin, float((before[1:][ws[1:] > 0] - want).abs().min() / upto[-1]) if bool((ws[1:] > 0).any()) else math.inf)
        order = order[stay]
    if q > 0.0:
        order = order[d[order] >= math.log(q)]
    ids = torch.sort(order).values
    ws = w[ids]
    upto = torch.cumsum(ws, 0)
    z = float(upto[-1])
    at = int((upto <= u * z).sum())
    inner = upto[:-1][ws[1:] > 0] if len(ids) > 1 else upto[:0]
    if inner.numel():
        margin = min(margin, float((inner - u * z).abs().min()) / z if u > 0.0 else math.inf)
    t = int(ids[at])
    return t, float(d[t]) - math.log(z), margin - (light if u > 0.0 else 0.0)
