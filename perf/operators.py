"""Timed cases of the head operators: the final norm, the vocabulary projection with
low-rank adapters, and the processing of logits before they are scored.

``own`` false: the operators in plain torch, 32-bit arithmetic, rounded once at the end.
``own`` true: the calls a serving program makes of this package.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-5
SCRATCH = 32 << 20  # bytes of scratch a serving program keeps for these calls


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request between the last layer and the head
        {"name": "norm_token", "op": "norm", "T": 1, "n": 1, "H": 4096, "dtype": "bf16", "residual": True,
         "keep": True, "out": "bf16"},
        # a decode step of 256 requests, 8-bit output for an 8-bit head
        {"name": "norm_decode_e4m3", "op": "norm", "T": 256, "n": 256, "H": 4096, "dtype": "bf16", "residual": True,
         "keep": False, "out": "e4m3"},
        # the last positions of 333 prompts picked out of their 9001 tokens, odd width
        {"name": "norm_rows_odd", "op": "norm", "T": 9001, "n": 333, "H": 5001, "dtype": "f16", "residual": True,
         "keep": False, "out": "f16"},
        # every position of a long prefill (echo), 8-bit output and the updated residual
        {"name": "norm_prefill_e4m3", "op": "norm", "T": 16384, "n": 16384, "H": 8192, "dtype": "bf16",
         "residual": True, "keep": True, "out": "e4m3"},
        # one token of one request, no adapter
        {"name": "head_token", "op": "head", "T": 1, "B": 1, "H": 2048, "V": 32000, "dtype": "bf16", "out": "f32",
         "adapters": 0, "rank": 0, "bare": 1.0},
        # a small batch with odd sizes, float16, tiny rank
        {"name": "head_odd_f16", "op": "head", "T": 77, "B": 19, "H": 1000, "V": 50001, "dtype": "f16", "out": "f16",
         "adapters": 5, "rank": 5, "bare": 0.2},
        # a decode step of an 8-bit head, a quarter of the requests without an adapter
        {"name": "head_decode_e4m3", "op": "head", "T": 48, "B": 48, "H": 4096, "V": 152064, "dtype": "e4m3",
         "out": "f32", "adapters": 12, "rank": 32, "bare": 0.25},
        # a decode step of 256 requests over the decode workload's vocabulary, 32 adapters
        {"name": "head_decode", "op": "head", "T": 256, "B": 256, "H": 4096, "V": 128256, "dtype": "bf16",
         "out": "bf16", "adapters": 32, "rank": 16, "bare": 0.1},
        # echo of 8 prompts over the prefill workload's vocabulary, long segments of one adapter
        {"name": "head_echo", "op": "head", "T": 2048, "B": 8, "H": 4096, "V": 32000, "dtype": "bf16", "out": "f32",
         "adapters": 4, "rank": 64, "bare": 0.0},
        # one request with a short history
        {"name": "logits_token", "op": "logits", "T": 1, "B": 1, "V": 128256, "dtype": "f32", "history": 600,
         "bias": 20, "masked": 0.0},
        # draft verification: about five rows a request, a grammar on half of the rows, bf16 logits
        {"name": "logits_verify", "op": "logits", "T": 240, "B": 48, "V": 152064, "dtype": "bf16", "history": 3000,
         "bias": 100, "masked": 0.5},
        # a decode step of 256 requests with long histories
        {"name": "logits_decode", "op": "logits", "T": 256, "B": 256, "V": 128256, "dtype": "f32", "history": 30000,
         "bias": 300, "masked": 0.3},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "head", "logits"])
    if op == "norm":
        H = _log_int(rng, 64, 16384)
        n = _log_int(rng, 1, max(2, min(20000, 134_000_000 // H)))
        picked = rng.random() < 0.3
        T = n + rng.randrange(1, 2000) if picked else n
        return {"op": op, "T": T, "n": n, "H": H, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "residual": rng.random() < 0.7, "keep": not picked and rng.random() < 0.5,
                "out": rng.choice(["same", "e4m3", "e4m3"])}
    if op == "head":
        dtype = rng.choice(["bf16", "bf16", "f16", "e4m3"])
        H = 16 * _log_int(rng, 16, 512)
        V = _log_int(rng, 1000, 152064)
        T = _log_int(rng, 1, max(2, min(4096, 250_000_000_000 // (H * V))))
        B = T if rng.random() < 0.6 else max(1, T // rng.randrange(2, 400))
        adapters = rng.choice([0, 1, 3, 8, 20, 32])
        return {"op": op, "T": T, "B": B, "H": H, "V": V, "dtype": dtype,
                "out": rng.choice(["f32", "f16" if dtype == "f16" else "bf16"]), "adapters": adapters,
                "rank": rng.choice([4, 8, 16, 32, 64, rng.randrange(1, 65)]) if adapters else 0,
                "bare": rng.choice([0.0, 0.1, 0.5])}
    V = _log_int(rng, 1000, 256000)
    T = _log_int(rng, 1, max(2, min(1024, 30_000_000 // V)))
    B = T if rng.random() < 0.6 else max(1, T // rng.randrange(2, 8))
    return {"op": op, "T": T, "B": B, "V": V, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
            "history": _log_int(rng, 1, 30000), "bias": rng.choice([0, 1, 17, 300]),
            "masked": rng.choice([0.0, 0.3, 1.0])}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device="cuda")


def _offsets(g, B, T):
    """B nonempty requests over T rows."""
    if B >= T:
        return torch.arange(T + 1, device="cuda", dtype=torch.int32)
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:B - 1].sort().values + 1
    z = torch.zeros(1, dtype=cuts.dtype, device="cuda")
    return torch.cat([z, cuts, z + T]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c, "scratch": torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda")}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        T, n, H = c["T"], c["n"], c["H"]
        # activations of a last layer: a few channels far larger than the rest
        chan = 1.0 + 30.0 * (torch.rand(H, generator=g, device="cuda") < 0.002)
        s["x"] = (_randn(g, T, H) * chan).to(dt)
        s["residual"] = (4.0 * _randn(g, T, H) * chan).to(dt) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(g, H)).to(dt)
        s["rows"] = torch.randperm(T, generator=g, device="cuda")[:n].sort().values.to(torch.int32) if n < T else None
        out = dt if c["out"] == "same" else DTYPES[c["out"]]
        s["out"] = torch.empty(n, H, dtype=out, device="cuda")
        s["scale"] = torch.empty(n, dtype=torch.float32, device="cuda") if c["out"] == "e4m3" else None
        s["kept"] = torch.empty(n, H, dtype=dt, device="cuda") if c["keep"] else None
    elif c["op"] == "head":
        T, B, H, V, A, r = c["T"], c["B"], c["H"], c["V"], c["adapters"], c["rank"]
        s["offsets"] = _offsets(g, B, T)
        B = s["offsets"].numel() - 1
        x = _randn(g, T, H)
        s["weight_scale"] = s["x_scale"] = None
        w = torch.empty(V, H, dtype=dt, device="cuda")
        if c["dtype"] == "e4m3":
            s["x_scale"] = x.abs().amax(1) / E4M3_MAX
            s["x"] = (x / s["x_scale"][:, None]).to(dt)
            s["weight_scale"] = torch.empty(V, device="cuda")
        else:
            s["x"] = x.to(dt)
        for a in range(0, V, 16384):
            blk = _randn(g, min(16384, V - a), H) * (2.0 / math.sqrt(H))
            if c["dtype"] == "e4m3":
                sw = blk.abs().amax(1) / E4M3_MAX
                s["weight_scale"][a:a + 16384] = sw
                blk /= sw[:, None]
            w[a:a + 16384] = blk.to(dt)
        s["weight"] = w
        if A:
            at = torch.bfloat16 if c["dtype"] == "e4m3" else dt
            s["lora_a"] = (_randn(g, A, r, H) / math.sqrt(H)).to(at)
            s["lora_b"] = (_randn(g, A, V, r) * 0.3).to(at)
            s["adapter_scale"] = 0.5 + torch.rand(A, generator=g, device="cuda")
            ids = _ints(g, 0, A, B)
            ids = torch.where(torch.rand(B, generator=g, device="cuda") < c["bare"], -1, ids)
            # requests of one adapter stand together where each request has one row
            s["ids"] = (ids.sort().values if B == T else ids).to(torch.int32)
        s["out"] = torch.empty(T, V, dtype=DTYPES[c["out"]], device="cuda")
    else:
        T, B, V = c["T"], c["B"], c["V"]
        s["offsets"] = _offsets(g, B, T)
        B = s["offsets"].numel() - 1
        s["logits"] = torch.empty(T, V, dtype=dt, device="cuda")
        for a in range(0, T, 256):
            s["logits"][a:a + 256] = (3.0 * _randn(g, min(256, T - a), V)).to(dt)
        # histories: lengths up to the case's, tokens from a skewed distribution, the prompt first
        lens = (c["history"] * torch.rand(B, generator=g, device="cuda") ** 2).long().clamp_min(1)
        if B == 1:
            lens.fill_(c["history"])
        z = torch.zeros(1, dtype=torch.int64, device="cuda")
        s["history_offsets"] = torch.cat([z, lens.cumsum(0)]).to(torch.int32)
        total = int(s["history_offsets"][-1])
        s["history"] = (V * torch.rand(total, generator=g, device="cuda") ** 4).long().clamp_max(V - 1).to(torch.int32)
        s["prompt_lens"] = (lens * torch.rand(B, generator=g, device="cuda")).to(torch.int32)
        u = torch.rand(3, B, generator=g, device="cuda")
        s["repetition"] = torch.where(u[0] < 0.3, torch.ones_like(u[0]), 0.8 + 0.6 * u[0])
        s["frequency"] = torch.where(u[1] < 0.3, torch.zeros_like(u[1]), 1.5 * u[1] - 0.5)
        s["presence"] = torch.where(u[2] < 0.3, torch.zeros_like(u[2]), 1.5 * u[2] - 0.5)
        s["bias"] = None
        if c["bias"]:
            k = min(c["bias"], V // 4)
            # strictly ascending ids of each request: k places of V/k tokens each
            step = V // k
            tok = torch.arange(k, device="cuda") * step + torch.randint(0, step, (B, k), generator=g, device="cuda")
            val = 5.0 * _randn(g, B, k)
            s["bias"] = (tok.reshape(-1).to(torch.int32), val.reshape(-1).contiguous(),
                         (torch.arange(B + 1, device="cuda") * k).to(torch.int32))
        s["mask"] = s["mask_index"] = None
        if c["masked"]:
            on = torch.rand(T, generator=g, device="cuda") < c["masked"]
            on[0] = True
            M, words = int(on.sum()), (V + 31) // 32
            # grammars: some rows allow nearly every token, others only a few words of them
            m = torch.randint(-2 ** 31, 2 ** 31, (M, words), generator=g, device="cuda").to(torch.int32)
            few = torch.rand(M, 1, generator=g, device="cuda") < 0.5
            keep = torch.rand(M, words, generator=g, device="cuda") < 0.02
            s["mask"] = torch.where(few, torch.where(keep, m, 0), torch.where(keep, m, -1)).contiguous()
            s["mask_index"] = torch.where(on, on.cumsum(0) - 1, -1).to(torch.int32)
        s["out"] = torch.empty(T, V, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "head": _own_head, "logits": _own_logits}[op](s)
    return {"norm": _plain_norm, "head": _plain_head, "logits": _plain_logits}[op](s)


def _own_norm(s):
    import ragged_log_probs_gb300 as lp
    lp.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], rows=s["rows"], out=s["out"], out_scale=s["scale"],
                residual_out=s["kept"], workspace=s["scratch"])
    return [s["out"]] + [t for t in (s["scale"], s["kept"]) if t is not None]


def _own_head(s):
    import ragged_log_probs_gb300 as lp
    if s["case"]["adapters"]:
        lp.project(s["x"], s["weight"], x_scale=s["x_scale"], weight_scale=s["weight_scale"], lora_a=s["lora_a"],
                   lora_b=s["lora_b"], adapter_scale=s["adapter_scale"], adapter_ids=s["ids"],
                   row_offsets=s["offsets"], out=s["out"], workspace=s["scratch"])
    else:
        lp.project(s["x"], s["weight"], x_scale=s["x_scale"], weight_scale=s["weight_scale"], out=s["out"],
                   workspace=s["scratch"])
    return s["out"]


def _own_logits(s):
    import ragged_log_probs_gb300 as lp
    bt, bv, bo = s["bias"] if s["bias"] is not None else (None, None, None)
    lp.process_logits(s["logits"], row_offsets=s["offsets"], history=s["history"],
                      history_offsets=s["history_offsets"], prompt_lens=s["prompt_lens"], repetition=s["repetition"],
                      frequency=s["frequency"], presence=s["presence"], bias_tokens=bt, bias_values=bv,
                      bias_offsets=bo, mask=s["mask"], mask_index=s["mask_index"], out=s["out"],
                      workspace=s["scratch"])
    return s["out"]


def _rows_to_requests(offsets, T):
    return torch.searchsorted(offsets, torch.arange(T, device=offsets.device, dtype=offsets.dtype), right=True) - 1


def _plain_norm(s):
    x, r = s["x"], s["residual"]
    if s["rows"] is not None:
        rows = s["rows"].long()
        x = x[rows]
        r = r[rows] if r is not None else None
    h = x.float()
    if r is not None:
        h = h + r.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if s["scale"] is not None:
        scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
        got = [(y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale]
    else:
        got = [y.to(s["out"].dtype)]
    return got + ([h.to(x.dtype)] if s["kept"] is not None else [])


def _plain_head(s):
    x, w = s["x"].float(), s["weight"].float()
    if s["x_scale"] is not None:
        x *= s["x_scale"][:, None]
        w *= s["weight_scale"][:, None]
    y = x @ w.t()
    if s["case"]["adapters"]:
        T, A, r = x.shape[0], s["lora_a"].shape[0], s["lora_a"].shape[1]
        ids = s["ids"].long()[_rows_to_requests(s["offsets"], T)]
        # every adapter's part of every row, those of other requests' adapters set to zero
        u = (x @ s["lora_a"].float().reshape(A * r, -1).t()).reshape(T, A, r)
        u = u * ((ids[:, None] == torch.arange(A, device=ids.device)) * s["adapter_scale"])[:, :, None]
        y += u.reshape(T, A * r) @ s["lora_b"].float().transpose(1, 2).reshape(A * r, -1)
    return y.to(s["out"].dtype)


def _plain_logits(s):
    x = s["logits"].float()
    T, V = x.shape
    B = s["offsets"].numel() - 1
    of = _rows_to_requests(s["offsets"], T)
    n = s["history"].numel()
    req = _rows_to_requests(s["history_offsets"], n)
    cell = req * V + s["history"].long()
    written = torch.arange(n, device=x.device) - s["history_offsets"].long()[req] >= s["prompt_lens"].long()[req]
    count = torch.zeros(B * V, device=x.device).index_add_(0, cell, written.float()).view(B, V)[of]
    seen = torch.zeros(B * V, dtype=torch.bool, device=x.device)
    seen[cell] = True
    rep = s["repetition"][of][:, None]
    x = torch.where(seen.view(B, V)[of], torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][of][:, None] * count - s["presence"][of][:, None] * (count > 0)
    if s["bias"] is not None:
        tok, val, off = s["bias"]
        k = tok.numel()
        add = torch.zeros(B * V, device=x.device)
        add[_rows_to_requests(off, k) * V + tok.long()] = val
        x = x + add.view(B, V)[of]
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        bits = bits.reshape(s["mask"].shape[0], -1)[:, :V].bool()
        idx = s["mask_index"].long()
        banned = (idx >= 0)[:, None] & ~bits[idx.clamp_min(0)]
        x = torch.where(banned, float("-inf"), x)
    return x


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "head": _exact_head, "logits": _exact_logits}[case["op"]](s)


def _exact_norm(s):
    x = s["x"].double()
    if s["residual"] is not None:
        x += s["residual"].double()
    if s["rows"] is not None:
        x = x.index_select(0, s["rows"].int())
    y = x / torch.sqrt((x * x).sum(1) / x.shape[1] + EPS).unsqueeze(1)
    y *= s["weight"].double()
    got = [y]
    if s["scale"] is not None:
        top = torch.maximum(y.max(1).values, -y.min(1).values)
        scale = torch.where(top / E4M3_MAX < TINY, torch.full_like(top, TINY), top / E4M3_MAX)
        got = [y / scale.unsqueeze(1), scale]
    return got + ([x] if s["kept"] is not None else [])


def _exact_head(s):
    T, V = s["out"].shape
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().unsqueeze(1)
    y = torch.empty(T, V, dtype=torch.float64, device="cuda")
    for a in range(0, V, 16384):
        w = s["weight"][a:a + 16384].double()
        if s["weight_scale"] is not None:
            w = w * s["weight_scale"][a:a + 16384].double().unsqueeze(1)
        torch.matmul(x, w.t(), out=y[:, a:a + 16384]) if V <= 16384 else y[:, a:a + 16384].copy_(x @ w.t())
    if s["case"]["adapters"]:
        off, ids = s["offsets"].tolist(), s["ids"].tolist()
        rows = {}
        for b, a in enumerate(ids):
            if a >= 0:
                rows.setdefault(a, []).extend(range(off[b], off[b + 1]))
        for a, mine in rows.items():
            at = torch.tensor(mine, device="cuda")
            u = (x[at] @ s["lora_a"][a].double().t()) * float(s["adapter_scale"][a])
            y[at] += u @ s["lora_b"][a].double().t()
    return y


def _exact_logits(s):
    x = s["logits"].double()
    T, V = x.shape
    off, hoff, plen = s["offsets"].tolist(), s["history_offsets"].tolist(), s["prompt_lens"].tolist()
    for b in range(len(off) - 1):
        row = x[off[b]:off[b + 1]]
        h = s["history"][hoff[b]:hoff[b + 1]].long()
        out = torch.bincount(h[plen[b]:], minlength=V).double()
        met = torch.unique(h)
        rep = float(s["repetition"][b])
        old = row[:, met]
        row[:, met] = torch.where(old > 0, old / rep, old * rep)
        row -= float(s["frequency"][b]) * out + float(s["presence"][b]) * out.clamp_max(1.0)
        if s["bias"] is not None:
            tok, val, bo = s["bias"]
            a, e = int(bo[b]), int(bo[b + 1])
            row[:, tok[a:e].long()] += val[a:e].double()
    if s["mask"] is not None:
        for t, m in enumerate(s["mask_index"].tolist()):
            if m >= 0:
                v = torch.arange(V, device="cuda")
                x[t, (s["mask"][m][v // 32].long() >> (v % 32)) % 2 == 0] = float("-inf")
    return x


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(c):
    if c["op"] == "norm":
        e, o = SIZE[c["dtype"]], SIZE[c["dtype"] if c["out"] == "same" else c["out"]]
        each = e * (1 + c["residual"] + c["keep"]) + o
        return {"bytes": c["n"] * c["H"] * each + c["H"] * e + (4 * c["n"] if c["out"] == "e4m3" else 0),
                "flops": 6 * c["n"] * c["H"]}
    if c["op"] == "head":
        T, H, V, r, e = c["T"], c["H"], c["V"], c["rank"], SIZE[c["dtype"]]
        used = min(c["adapters"], c["B"])
        return {"bytes": V * H * e + T * H * e + T * V * SIZE[c["out"]] + 2 * used * r * (H + V),
                "flops": 2 * T * H * V + 2 * T * r * (H + V)}
    T, V = c["T"], c["V"]
    return {"bytes": T * V * (SIZE[c["dtype"]] + 4) + c["masked"] * T * V / 8 + c["B"] * (c["history"] * 4 / 3 + 8 * c["bias"]),
            "flops": 6 * T * V}
