"""Timed cases of the operators round a 4-bit head and of the draw of the next token: rows in
microscaled 4-bit floating point (quantised, read back, looked up), the vocabulary projection of
such rows, and sampling with temperature, top-k, top-p and min-p.

``own`` false: the operators in plain torch, 32-bit arithmetic (the sums of probabilities, and
what is compared with them, in 64), rounded once at the end.
``own`` true: the calls a serving program makes of this package.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the 3 bits below the sign
SMALLEST = 40.0  # a token's weight counts from 2^-40 of the largest on
SCRATCH = 4 << 20  # bytes of scratch a serving program keeps for these calls


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # the next token of one request with the usual settings, top-k and top-p
        {"name": "sample_token", "op": "sample", "T": 1, "B": 1, "V": 128256, "dtype": "f32", "mix": "both",
         "masked": 0.0},
        # draft verification of a small batch, odd vocabulary, every kind of setting
        {"name": "sample_odd", "op": "sample", "T": 77, "B": 19, "V": 50001, "dtype": "f16", "mix": "all", "masked": 0.2},
        # draft verification: about five rows a request, a grammar on some of the rows, bf16 logits
        {"name": "sample_verify", "op": "sample", "T": 240, "B": 48, "V": 152064, "dtype": "bf16", "mix": "all",
         "masked": 0.3},
        # a decode step of 256 requests, every kind of setting
        {"name": "sample_decode", "op": "sample", "T": 256, "B": 256, "V": 128256, "dtype": "f32", "mix": "all",
         "masked": 0.1},
        # hidden states of odd width, blocks of 32
        {"name": "pack_odd", "op": "pack", "T": 333, "H": 5024, "dtype": "f16", "block": 32},
        # a head's weight laid out once at load time, blocks of 16
        {"name": "pack_weight", "op": "pack", "T": 32000, "H": 4096, "dtype": "bf16", "block": 16},
        # the sampled tokens of a decode step looked up in a tied 4-bit weight
        {"name": "lookup_decode", "op": "lookup", "n": 256, "V": 128256, "H": 4096, "dtype": "bf16", "block": 16},
        # the tokens of a long prefill
        {"name": "lookup_prefill", "op": "lookup", "n": 16384, "V": 32000, "H": 4096, "dtype": "bf16", "block": 32},
        # one token of one request, 4-bit head
        {"name": "head4_token", "op": "head4", "T": 1, "H": 2048, "V": 32000, "dtype": "bf16", "out": "f32", "block": 32},
        # a small batch with odd sizes, float16
        {"name": "head4_odd", "op": "head4", "T": 77, "H": 1056, "V": 50001, "dtype": "f16", "out": "f16", "block": 16},
        # a decode step of 48 requests
        {"name": "head4_decode", "op": "head4", "T": 48, "H": 4096, "V": 152064, "dtype": "bf16", "out": "f32",
         "block": 16},
        # echo of 8 prompts: logits of 2048 positions
        {"name": "head4_echo", "op": "head4", "T": 2048, "H": 4096, "V": 32000, "dtype": "bf16", "out": "bf16",
         "block": 16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "pack", "lookup", "head4", "head4"])
    if op == "sample":
        V = _log_int(rng, 1000, 256000)
        T = _log_int(rng, 1, max(2, min(1024, 32_000_000 // V)))
        B = T if rng.random() < 0.6 else max(1, T // rng.randrange(2, 8))
        return {"op": op, "T": T, "B": B, "V": V, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
                "mix": rng.choice(["all", "all", "both", "top_k", "top_p", "min_p", "temperature", "greedy"]),
                "masked": rng.choice([0.0, 0.3, 1.0])}
    H = 32 * _log_int(rng, 2, 256)
    dtype, block = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([16, 32])
    if op == "pack":
        return {"op": op, "T": _log_int(rng, 1, max(2, min(40000, 130_000_000 // H))), "H": H, "dtype": dtype,
                "block": block}
    if op == "lookup":
        return {"op": op, "n": _log_int(rng, 1, max(2, min(16384, 67_000_000 // H))), "V": _log_int(rng, 1000, 152064),
                "H": H, "dtype": dtype, "block": block}
    V = _log_int(rng, 1000, 152064)
    T = _log_int(rng, 1, max(2, min(4096, 260_000_000_000 // (H * V))))
    return {"op": op, "T": T, "H": H, "V": V, "dtype": dtype, "out": rng.choice(["f32", "f16" if dtype == "f16" else "bf16"]),
            "block": block}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _offsets(g, B, T):
    """B nonempty requests over T rows."""
    if B >= T:
        return torch.arange(T + 1, device="cuda", dtype=torch.int32)
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:B - 1].sort().values + 1
    z = torch.zeros(1, dtype=cuts.dtype, device="cuda")
    return torch.cat([z, cuts, z + T]).to(torch.int32)


def _settings(g, mix, B):
    """Temperature, top-k, top-p and min-p of B requests."""
    u = _rand(g, 5, B)
    kinds = {"greedy": 0, "temperature": 1, "top_p": 2, "top_k": 3, "both": 4, "min_p": 5}
    if mix == "all":
        kind = torch.bucketize(u[0], torch.tensor([0.1, 0.25, 0.55, 0.75, 0.9], device="cuda"))
    else:
        kind = torch.full((B,), kinds[mix], device="cuda")
    on = lambda *names: torch.isin(kind, torch.tensor([kinds[n] for n in names], device="cuda"))  # noqa: E731
    one = torch.ones(B, device="cuda")
    return {"temperature": torch.where(on("greedy"), 0 * one, 0.6 + 0.7 * u[1]),
            "top_k": torch.where(on("top_k", "both"), (2.0 * 500.0 ** u[2]).floor(), 0 * one).to(torch.int32),
            "top_p": torch.where(on("top_p", "both"), 0.5 + 0.48 * u[3], one),
            "min_p": torch.where(on("min_p"), 0.02 + 0.18 * u[4], 0 * one)}


def _packed_rows(g, rows, H, block, dtype):
    """A random weight in 4 bits: codes, scales in their tiles, row scales."""
    codes = torch.empty(rows, H // 2, dtype=torch.uint8, device="cuda")
    blocks = torch.empty(rows, H // block, dtype=torch.uint8, device="cuda")
    row_scale = torch.empty(rows, device="cuda") if block == 16 else None
    for a in range(0, rows, 16384):
        w = (_randn(g, min(16384, rows - a), H) * (2.0 / math.sqrt(H))).to(dtype)
        c, s, r = _quantise(w, block)
        codes[a:a + 16384] = c
        blocks[a:a + 16384] = s
        if r is not None:
            row_scale[a:a + 16384] = r
    return codes, _tiled(blocks), row_scale


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c, "scratch": torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda")}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        s["offsets"] = _offsets(g, c["B"], T)
        B = s["offsets"].numel() - 1
        s["logits"] = torch.empty(T, V, dtype=dt, device="cuda")
        for a in range(0, T, 256):
            n = min(256, T - a)
            # a bulk of unlikely tokens and some tens that the context asks for
            x = 2.5 * _randn(g, n, V) + (_rand(g, n, V) < 30.0 / V) * 12.0 * _rand(g, n, 1)
            some = (_rand(g, n, 1) < c["masked"]) & (_rand(g, n, V) > 0.02)  # a grammar allows few tokens
            s["logits"][a:a + n] = torch.where(some, float("-inf"), x).to(dt)
        s.update(_settings(g, c["mix"], B))
        s["uniform"] = _rand(g, T)
        s["out"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["logprob"] = torch.empty(T, device="cuda")
    elif c["op"] == "pack":
        T, H = c["T"], c["H"]
        chan = 1.0 + 30.0 * (_rand(g, H) < 0.002)  # a few channels far larger than the rest
        s["x"] = (_randn(g, T, H) * chan).to(dt)
        s["codes"] = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(_scale_bytes(T, H, c["block"]), dtype=torch.uint8, device="cuda")
        s["row_scale"] = torch.empty(T, device="cuda") if c["block"] == 16 else None
        s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    elif c["op"] == "lookup":
        s["weight"] = _packed_rows(g, c["V"], c["H"], c["block"], dt)
        s["rows"] = torch.randint(0, c["V"], (c["n"],), generator=g, device="cuda").to(torch.int32)
        s["out"] = torch.empty(c["n"], c["H"], dtype=dt, device="cuda")
    else:
        T, H, V = c["T"], c["H"], c["V"]
        s["x"] = _randn(g, T, H).to(dt)
        s["weight"] = _packed_rows(g, V, H, c["block"], dt)
        s["codes"] = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(_scale_bytes(T, H, c["block"]), dtype=torch.uint8, device="cuda")
        s["row_scale"] = torch.empty(T, device="cuda") if c["block"] == 16 else None
        s["out"] = torch.empty(T, V, dtype=DTYPES[c["out"]], device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"sample": _own_sample, "pack": _own_pack, "lookup": _own_lookup, "head4": _own_head4}[op](s)
    return {"sample": _plain_sample, "pack": _plain_pack, "lookup": _plain_lookup, "head4": _plain_head4}[op](s)


def _own_sample(s):
    import ragged_log_probs_gb300 as lp
    lp.sample(s["logits"], s["uniform"], row_offsets=s["offsets"], temperature=s["temperature"], top_k=s["top_k"],
              top_p=s["top_p"], min_p=s["min_p"], out=s["out"], out_logprob=s["logprob"], workspace=s["scratch"])
    return [s["out"], s["logprob"]]


def _own_pack(s):
    import ragged_log_probs_gb300 as lp
    lp.quantize_fp4(s["x"], block=s["case"]["block"], out=s["codes"], out_scales=s["scales"],
                    out_row_scale=s["row_scale"])
    # (the codes are returned as the values they stand for)
    return lp.dequantize_fp4(s["codes"], s["scales"], row_scale=s["row_scale"], block=s["case"]["block"], out=s["out"])


def _own_lookup(s):
    import ragged_log_probs_gb300 as lp
    codes, scales, row_scale = s["weight"]
    return lp.dequantize_fp4(codes, scales, row_scale=row_scale, block=s["case"]["block"], rows=s["rows"], out=s["out"],
                             workspace=s["scratch"])


def _own_head4(s):
    import ragged_log_probs_gb300 as lp
    codes, scales, row_scale = s["weight"]
    block = s["case"]["block"]
    lp.quantize_fp4(s["x"], block=block, out=s["codes"], out_scales=s["scales"], out_row_scale=s["row_scale"])
    return lp.project_fp4(s["codes"], s["scales"], codes, scales, block=block, x_row_scale=s["row_scale"],
                          weight_row_scale=row_scale, out=s["out"], workspace=s["scratch"])


def _rows_to_requests(offsets, T):
    return torch.searchsorted(offsets, torch.arange(T, device=offsets.device, dtype=offsets.dtype), right=True) - 1


def _plain_sample(s):
    x = s["logits"].float()
    T, V = x.shape
    of = _rows_to_requests(s["offsets"], T)
    tau = s["temperature"][of].double()[:, None]
    k = s["top_k"][of].long()[:, None]
    p, floor = s["top_p"][of].double()[:, None], s["min_p"][of].double()[:, None]
    k = torch.where(tau == 0, 1, torch.where(k <= 0, V, k))
    tau = torch.where(tau == 0, 1.0, tau)
    top = x.amax(1, keepdim=True).double()
    d = (x.double() - top) / tau
    w = torch.where(d >= -SMALLEST * math.log(2.0), torch.exp(d), 0.0)
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    ranked = w.gather(1, order) * (torch.arange(V, device=x.device) < k)
    upto = ranked.cumsum(1)
    before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
    keep = (p >= 1) | (before < p * upto[:, -1:])
    keep[:, 0] = True
    keep &= value.double() >= top + tau * torch.log(floor)
    kept = torch.zeros_like(w).scatter_(1, order, ranked * keep)
    upto = kept.cumsum(1)
    token = (upto <= s["uniform"].double()[:, None] * upto[:, -1:]).sum(1, keepdim=True)
    return [token[:, 0].to(torch.int32), torch.log(kept.gather(1, token) / upto[:, -1:])[:, 0].float()]


def _scale_bytes(rows, H, block):
    return -(-rows // 128) * -(-(H // block) // 4) * 512


def _tiled(blocks):
    """Scales [rows, blocks] in tiles of 128 rows by 4, each [row % 32][row / 32 % 4][block % 4]; zeros around them."""
    rows, n = blocks.shape
    rb, cb = -(-rows // 128), -(-n // 4)
    full = torch.nn.functional.pad(blocks, (0, cb * 4 - n, 0, rb * 128 - rows))
    return full.view(rb, 4, 32, cb, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(scales, rows, n):
    rb, cb = -(-rows // 128), -(-n // 4)
    return scales.view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)[:rows, :n]


def _two(e):
    """2^e of whole numbers e, from its bits (torch.ldexp goes through a power, which need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x, block):
    """Codes (two to a byte, the first in the low half), scale bytes [rows, blocks], row scales."""
    y, rows = x.float(), x.shape[0]
    row_scale = None
    if block == 16:
        # the smallest power of two r with max|x| <= 6 * 448 * r
        m, e = torch.frexp(y.abs().amax(1))
        e = torch.where(m <= 2688.0 / 4096.0, e - 12, e - 11).clamp_min(-100)
        e = torch.where(m == 0, -100, e)
        row_scale = _two(e).float()
        y = (y * _two(-e).float()[:, None]).view(rows, -1, block)
        scale = (y.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
        byte, s = scale.view(torch.uint8), scale.float()[:, :, None]
    else:
        y = y.view(rows, -1, block)
        m, e = torch.frexp(y.abs().amax(2))
        e = torch.where(m == 0, -127, e - 3).clamp(-127, 127)
        byte = (e + 127).to(torch.uint8)
        y, s = y * _two(-e).float()[:, :, None], torch.ones(1, device=x.device)
    q = torch.where(s > 0, y.abs() / s, 0.0).view(rows, -1)
    # to the nearest of LEVELS, the even one of two as near, at most 6
    code = ((q > 0.25).byte() + (q >= 0.75).byte() + (q > 1.25).byte() + (q >= 1.75).byte() + (q > 2.5).byte()
            + (q >= 3.5).byte() + (q > 5.0).byte()) | (torch.signbit(y).view(rows, -1).byte() << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte, row_scale


def _values(codes, byte, row_scale, block):
    """The rows' values in 32 bits."""
    rows, half = codes.shape
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], 2).view(-1).int()
    v = table.index_select(0, both).view(rows, -1, block)
    if block == 16:
        v *= byte.contiguous().view(torch.float8_e4m3fn).float()[:, :, None]
        return v.view(rows, 2 * half) * row_scale[:, None]
    return (v * _two(byte.int() - 127).float()[:, :, None]).view(rows, 2 * half)


def _plain_pack(s):
    block = s["case"]["block"]
    return _values(*_quantise(s["x"], block), block).to(s["out"].dtype)


def _plain_lookup(s):
    codes, scales, row_scale = s["weight"]
    c, rows = s["case"], s["rows"].long()
    byte = _untiled(scales, c["V"], c["H"] // c["block"])[rows]
    return _values(codes[rows], byte, None if row_scale is None else row_scale[rows], c["block"]).to(s["out"].dtype)


def _plain_head4(s):
    codes, scales, row_scale = s["weight"]
    c, block = s["case"], s["case"]["block"]
    w = _values(codes, _untiled(scales, c["V"], c["H"] // block), row_scale, block)
    x = _values(*_quantise(s["x"], block), block)
    return (x @ w.t()).to(s["out"].dtype)


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "pack": _exact_pack, "lookup": _exact_lookup, "head4": _exact_head4}[case["op"]](s)


def _exact_sample(s):
    off, T = s["offsets"].tolist(), s["case"]["T"]
    tokens, logs = [], []
    u = s["uniform"].tolist()
    per = [s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p")]
    for b in range(len(off) - 1):
        tau, k, p, floor = (v[b] for v in per)
        for t in range(off[b], off[b + 1]):
            x = s["logits"][t].double()
            if tau == 0.0:
                tokens.append(int((x == x.max()).nonzero()[0]))
                logs.append(0.0)
                continue
            z = (x - x.max()) / tau
            ids = torch.argsort(-z, stable=True)
            ids = ids[:k] if k > 0 else ids
            w = torch.exp(z[ids])
            w[z[ids] < -SMALLEST * math.log(2.0)] = 0.0
            n = len(ids)
            if p < 1.0:
                # as many as are needed to reach p of the whole
                n = 1 + int((torch.cumsum(w, 0) < p * w.sum()).sum())
            if floor > 0.0:
                n = min(n, int((z[ids] >= math.log(floor)).sum()))
            ids, place = ids[:n].sort()
            w = w[:n][place]
            share = torch.cumsum(w, 0) / w.sum()
            at = int(torch.searchsorted(share, torch.tensor([u[t]], dtype=torch.float64, device="cuda"), right=True))
            tokens.append(int(ids[at]))
            logs.append(float(torch.log(w[at]) - torch.log(w.sum())))
    assert len(tokens) == T
    return [torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)]


def _exact_codes(x, scale):
    """The nearest level of x / scale, by its distance to each."""
    q = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    best, gap = torch.zeros_like(q), q.abs()
    for i in (2, 4, 6, 1, 3, 5, 7):  # even codes first: they win where two are as near
        g = (q.abs() - LEVELS[i]).abs()
        best = torch.where(g < gap, LEVELS[i], best)
        gap = torch.minimum(g, gap)
    return torch.where(q < 0, -best, best) * scale


def _exact_power(b):
    """The largest power of two that is not above b."""
    e = torch.floor(torch.log2(torch.where(b > 0, b, 1.0)))
    e = e + (_two(e + 1) <= b).double() - (_two(e) > b).double()  # (log2 need not be exact next to whole numbers)
    return torch.where(b > 0, _two(e), 0.0)


def _exact_rows(x, block):
    x = x.double()
    rows, H = x.shape
    if block == 16:
        most = x.abs().max(1).values / 2688.0
        r = _exact_power(most)
        r = torch.where(r < most, 2.0 * r, r).clamp_min(2.0 ** -100)
        b = x.view(rows, H // 16, 16).abs().max(2).values / (6.0 * r[:, None])
        scale = b.float().to(torch.float8_e4m3fn).double() * r[:, None]
    else:
        b = x.view(rows, H // 32, 32).abs().max(2).values
        scale = (_exact_power(b) / 4.0).clamp_min(2.0 ** -127)
    return _exact_codes(x, scale.repeat_interleave(block, 1))


def _exact_values(codes, scales, row_scale, V, H, block, rows):
    """Rows `rows` of a packed weight."""
    n = H // block
    low, high = (codes[rows] % 16).long(), (codes[rows] // 16).long()
    both = torch.empty(len(rows), H, dtype=torch.long, device="cuda")
    both[:, 0::2], both[:, 1::2] = low, high
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")[both % 8] * (1.0 - 2.0 * (both // 8))
    j = torch.arange(n, device="cuda")
    at = ((rows // 128)[:, None] * -(-n // 4) + (j // 4)[None]) * 512 \
        + (rows % 32)[:, None] * 16 + (rows // 32 % 4)[:, None] * 4 + (j % 4)[None]
    byte = scales[at]
    if block == 16:
        scale = byte.view(torch.float8_e4m3fn).double() * row_scale[rows].double()[:, None]
    else:
        scale = _two(byte.int() - 127)
    return level * scale.repeat_interleave(block, 1)


def _exact_pack(s):
    x = s["x"]
    return torch.cat([_exact_rows(x[a:a + 4096], s["case"]["block"]) for a in range(0, x.shape[0], 4096)])


def _exact_lookup(s):
    c = s["case"]
    return _exact_values(*s["weight"], c["V"], c["H"], c["block"], s["rows"].long())


def _exact_head4(s):
    c = s["case"]
    x = _exact_rows(s["x"], c["block"])
    y = torch.empty(c["T"], c["V"], dtype=torch.float64, device="cuda")
    for a in range(0, c["V"], 8192):
        rows = torch.arange(a, min(a + 8192, c["V"]), device="cuda")
        y[:, a:a + 8192] = x @ _exact_values(*s["weight"], c["V"], c["H"], c["block"], rows).t()
    return y


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(c):
    if c["op"] == "sample":
        return {"bytes": c["T"] * (c["V"] * SIZE[c["dtype"]] + 12) + 16 * c["B"], "flops": 4 * c["T"] * c["V"]}
    e, per = SIZE[c["dtype"]], 0.5 + 1.0 / c["block"]
    row = 4 if c["block"] == 16 else 0
    if c["op"] == "pack":  # quantised, and read back as values
        return {"bytes": c["T"] * (c["H"] * (2 * e + 2 * per) + 2 * row), "flops": 6 * c["T"] * c["H"]}
    if c["op"] == "lookup":
        return {"bytes": c["n"] * (c["H"] * (e + per) + row + 4), "flops": 2 * c["n"] * c["H"]}
    T, H, V = c["T"], c["H"], c["V"]
    return {"bytes": V * (H * per + row) + T * (H * e + 2 * (H * per + row)) + T * V * SIZE[c["out"]], "flops": 2 * T * H * V}
