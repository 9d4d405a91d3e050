"""Plain 64-bit forms of the 4-bit rows on the CPU, for the tests. Written from the formulas of
include/lp_head.h; a code is found by its distance to every level, not by thresholds."""

import math

import torch

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nearest(q):
    """Levels' numbers nearest to |q| (float64), of two as near the even one."""
    dist = (q.abs().unsqueeze(-1) - torch.tensor(LEVELS, dtype=torch.float64)).abs()
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    return order[dist[..., order].argmin(-1)]


def power_floor(v):
    """floor(log2 v) of a positive Python float."""
    return math.frexp(v)[1] - 1


def e4m3(v):
    """The e4m3 value nearest to a Python float in 0..448, of two as near the even one."""
    if v == 0.0:
        return 0.0
    step = 2.0 ** (max(power_floor(v), -6) - 3)
    return round(v / step) * step  # (v / step is exact; round() takes the even one of two)


def quantise(x, block):
    """(levels' numbers [T, H], negative [T, H], scales [T, H / block] in float64, row scales or None)."""
    x = x.double()
    T, H = x.shape
    number, negative = torch.zeros(T, H, dtype=torch.long), torch.signbit(x)
    scales, rows = torch.zeros(T, H // block, dtype=torch.float64), None
    if block == 16:
        rows = torch.zeros(T, dtype=torch.float64)
    for t in range(T):
        r = 1.0
        if block == 16:
            top = float(x[t].abs().max())
            if not math.isfinite(top):
                rows[t], scales[t] = math.nan, math.nan
                continue
            r = 2.0 ** -100
            if top > 0:
                e = power_floor(top / 2688.0)
                e += top > 2688.0 * 2.0 ** e
                r = 2.0 ** max(e, -100)
            rows[t] = r
        for b in range(H // block):
            part = x[t, b * block:(b + 1) * block]
            top = float(part.abs().max())
            if block == 16:
                s = e4m3(top / (6.0 * r))
            elif not math.isfinite(top):
                scales[t, b] = math.nan
                continue
            else:
                s = 2.0 ** max(power_floor(top) - 2, -127) if top > 0 else 2.0 ** -127
            scales[t, b] = s
            if s > 0:
                number[t, b * block:(b + 1) * block] = nearest(part / (s * r))
    return number, negative, scales, rows


def values(number, negative, scales, rows, block):
    v = torch.tensor(LEVELS, dtype=torch.float64)[number]
    v = torch.where(negative, -v, v) * scales.repeat_interleave(block, 1)
    return v if rows is None else v * rows.double()[:, None]


def unpack(codes):
    """(numbers, negative) of packed codes [T, H / 2] uint8."""
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1).long()
    return c & 7, c >= 8


def pack(number, negative):
    c = (number + 8 * negative.long()).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def scale_values(scales, rows, H, block):
    """Scales [rows, H / block] in float64 out of their tiles, byte by byte, and the bytes that are left over
    in the tiles of the rows' own blocks."""
    n = H // block
    cb = -(-n // 4)
    at = lambda i, j: ((i // 128) * cb + j // 4) * 512 + (i % 32) * 16 + (i // 32 % 4) * 4 + j % 4
    index = torch.tensor([[at(i, j) for j in range(cb * 4)] for i in range(rows)])
    byte = scales.view(torch.uint8)[index]
    own, left = byte[:, :n].contiguous(), byte[:, n:]
    if block == 16:
        return own.view(torch.float8_e4m3fn).double(), left
    return torch.where(own == 255, math.nan, 2.0 ** (own.double() - 127.0)), left


def scale_bytes(values_, block):
    """The bytes of scales given by value."""
    if block == 16:
        return values_.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isnan(values_), 255.0, torch.log2(values_) + 127.0).round().to(torch.uint8)


def random_rows(T, H, block, seed, exponents=6):
    """Random 4-bit rows: codes, scales by value [T, H / block], row scales (f32, not powers of two) or None."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (T, H // 2), generator=g).to(torch.uint8)
    if block == 16:
        byte = torch.randint(0x20, 0x50, (T, H // 16), generator=g).to(torch.uint8)
        return codes, byte.view(torch.float8_e4m3fn).double(), 0.01 + torch.rand(T, generator=g)
    return codes, 2.0 ** torch.randint(-exponents, exponents, (T, H // 32), generator=g).double(), None
