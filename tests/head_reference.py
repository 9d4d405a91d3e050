"""Plain 64-bit forms of the head operators on the CPU, for the tests. Written from the
formulas of include/lp_head.h, one row or one request at a time."""

import torch

E4M3_MAX = 448.0
TINY = 2.0 ** -126


def norm(x, weight, eps, residual=None, rows=None):
    """(h, y) in float64: the sum before its rounding, and the normed row."""
    idx = range(x.shape[0]) if rows is None else rows
    hs, ys = [], []
    for i in idx:
        h = x[i].double()
        if residual is not None:
            h = h + residual[i].double()
        y = h / torch.sqrt((h * h).mean() + eps) * weight.double()
        hs.append(h)
        ys.append(y)
    return torch.stack(hs), torch.stack(ys)


def e4m3_scale(y):
    return (y.abs().amax(1) / E4M3_MAX).clamp_min(TINY)


def requests_of_rows(T, row_offsets):
    if row_offsets is None:
        return list(range(T))
    of = [-1] * T
    for b in range(len(row_offsets) - 1):
        for t in range(row_offsets[b], row_offsets[b + 1]):
            of[t] = b
    return of


def process(logits, row_offsets=None, history=None, prompt_lens=None, rep=None, freq=None, pres=None, bias=None,
            mask=None, mask_index=None):
    """(values, magnitudes) in float64: the processed logits, and for each value the sum of
    the magnitudes that its f32 form rounds. history: a list of token lists; bias: a list of
    {token: value}; mask: [rows, V] bool, True = allowed."""
    T, V = logits.shape
    out, mag = logits.double().clone(), torch.zeros(T, V, dtype=torch.float64)
    for t, b in enumerate(requests_of_rows(T, row_offsets)):
        row = out[t]
        m = row.abs()
        if history is not None:
            n_prompt = prompt_lens[b] if prompt_lens is not None else 0
            r = rep[b] if rep is not None else 1.0
            f = freq[b] if freq is not None else 0.0
            p = pres[b] if pres is not None else 0.0
            count = {}
            for i, tok in enumerate(history[b]):
                if tok < V:
                    count[tok] = count.get(tok, 0) + (i >= n_prompt)
            for tok, c in count.items():
                v = row[tok] / r if row[tok] > 0 else row[tok] * r
                m[tok] = abs(v) + 2 * abs(f) * c + abs(p)
                row[tok] = v - f * c - (p if c else 0.0)
        if bias is not None:
            for tok, v in bias[b].items():
                row[tok] += v
                m[tok] += abs(v)
        mag[t] = m
        if mask is not None:
            k = mask_index[t] if mask_index is not None else t
            if k >= 0:
                row[~mask[k]] = float("-inf")
    return out, mag


def pack_mask(allowed):
    """[rows, V] bool -> [rows, words] int32, bit v % 32 of word v / 32."""
    M, V = allowed.shape
    words = (V + 31) // 32
    padded = torch.zeros(M, words * 32, dtype=torch.int64)
    padded[:, :V] = allowed
    w = (padded.view(M, words, 32) << torch.arange(32)).sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
