"""Processing of logits (lp_head_process) against the 64-bit formula."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import head_reference as ref
from tests import parity

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


def i32(v):
    return torch.tensor(v, dtype=torch.int64).to(torch.int32).cuda()


def offsets(lists):
    o = [0]
    for x in lists:
        o.append(o[-1] + len(x))
    return i32(o)


def flat(lists):
    return i32([v for x in lists for v in x])


def make(T, V, B, dtype=torch.float32, hist=20, n_bias=3, masked=True, seed=0):
    g = torch.Generator().manual_seed(seed * 31 + V)
    ri = lambda hi, n: torch.randint(0, hi, (n,), generator=g).tolist()
    c = {"x": (torch.randn(T, V, generator=g) * 3).to(dtype)}
    cuts = sorted(torch.randperm(T - 1, generator=g)[:B - 1].add(1).tolist()) if B < T else list(range(1, T))
    c["off"] = [0] + cuts + [T]
    c["history"] = [ri(max(1, V // 3), int(ri(hist + 1, 1)[0])) for _ in range(B)]
    c["prompt"] = [int(ri(len(h) + 1, 1)[0]) for h in c["history"]]
    c["rep"] = (0.7 + torch.rand(B, generator=g)).tolist()
    c["freq"] = (torch.rand(B, generator=g) - 0.3).tolist()
    c["pres"] = (torch.rand(B, generator=g) - 0.3).tolist()
    c["rep"][0], c["freq"][0], c["pres"][0] = 1.0, 0.0, 0.0
    c["bias"] = [{t: float(torch.randn(1, generator=g)) for t in sorted(set(ri(V, n_bias)))} for _ in range(B)]
    M = max(1, T // 2)
    c["allowed"] = torch.rand(M, V, generator=g) < 0.5 if masked else None
    c["mask_index"] = [(t % M if t % 3 else -1) for t in range(T)] if masked else None
    f32 = lambda v: torch.tensor(v, dtype=torch.float32)
    for k in ("rep", "freq", "pres"):
        c[k] = f32(c[k]).tolist()
    return c


def call(c, x=None, **kw):
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = lp.new_head_workspace(requests=len(c["off"]) - 1, history=sum(len(h) for h in c["history"]))
    f = lambda v: torch.tensor(v, dtype=torch.float32).cuda()
    args = dict(row_offsets=i32(c["off"]), history=flat(c["history"]), history_offsets=offsets(c["history"]),
                prompt_lens=i32(c["prompt"]), repetition=f(c["rep"]), frequency=f(c["freq"]), presence=f(c["pres"]),
                bias_tokens=flat([list(b) for b in c["bias"]]), bias_values=f([v for b in c["bias"] for v in b.values()]),
                bias_offsets=offsets(c["bias"]))
    if c["allowed"] is not None:
        args.update(mask=ref.pack_mask(c["allowed"]).cuda(), mask_index=i32(c["mask_index"]))
    args.update(kw)
    out = lp.process_logits(c["x"].cuda() if x is None else x, workspace=ws, **args)
    return out, lp.read_status(ws)


def want_of(c, **kw):
    args = dict(row_offsets=c["off"], history=c["history"], prompt_lens=c["prompt"], rep=c["rep"], freq=c["freq"],
                pres=c["pres"], bias=c["bias"], mask=c["allowed"], mask_index=c["mask_index"])
    args.update(kw)
    return ref.process(c["x"], **args)


def check(out, want):
    want, mag = want
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]) and torch.isfinite(got[~inf & ~torch.isnan(want)]).all()
    fine = torch.isfinite(want)
    # at most six f32 roundings, each of a value below the sum of magnitudes
    bound = 6 * 2.0 ** -24 * mag * (1 + 2.0 ** -20)
    assert ((got - want).abs() <= bound)[fine].all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 3, 31, 32, 33, 100, 1000, 8191, 32000, 40001])
def test_vocabularies_and_types(V, dtype):
    c = make(9, V, 4, dtype, seed=1)
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


@pytest.mark.parametrize("T,B", [(1, 1), (2, 2), (7, 7), (40, 40), (60, 7)])
def test_rows_and_requests(T, B):
    c = make(T, 5000, B, hist=300, n_bias=20, seed=2)
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


@pytest.mark.parametrize("V", [128256, 152064, 256001])
def test_large_vocabularies(V):
    c = make(3, V, 2, hist=5000, n_bias=50, seed=3)
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


def test_many_rows_use_one_chunk():
    c = make(400, 3001, 400, hist=30, seed=4)
    out, _ = call(c)
    check(out, want_of(c))


def test_long_history_of_few_tokens():
    c = make(2, 2000, 2, seed=5)
    c["history"] = [[7] * 70000 + [8, 9] * 1000, [1999] * 3]
    c["prompt"] = [100, 0]
    c["rep"], c["freq"], c["pres"] = [1.5, 2.0], [0.25, -0.5], [1.0, 0.0]
    out, _ = call(c)
    check(out, want_of(c))


def test_empty_lists_and_defaults():
    c = make(5, 700, 5, seed=6, masked=False)
    c["history"], c["prompt"], c["bias"] = [[] for _ in range(5)], [0] * 5, [{} for _ in range(5)]
    out, status = call(c)
    assert status == 0 and torch.equal(out.cpu(), c["x"])
    ws = lp.new_head_workspace()
    assert torch.equal(lp.process_logits(c["x"].cuda(), workspace=ws).cpu(), c["x"])
    # a prompt length past the history: all of it is prompt
    c["history"], c["prompt"] = [[1, 1, 2]] * 5, [99] * 5
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


def test_bias_alone_and_mask_alone():
    c = make(6, 3333, 6, seed=7)
    ws = lp.new_head_workspace()
    bias = dict(bias_tokens=flat([list(b) for b in c["bias"]]),
                bias_values=torch.tensor([v for b in c["bias"] for v in b.values()]).cuda(),
                bias_offsets=offsets(c["bias"]))
    out = lp.process_logits(c["x"].cuda(), workspace=ws, **bias)
    check(out, ref.process(c["x"], bias=c["bias"]))
    allowed = torch.rand(6, 3333, generator=torch.Generator().manual_seed(1)) < 0.1
    out = lp.process_logits(c["x"].cuda(), workspace=ws, mask=ref.pack_mask(allowed).cuda())
    check(out, ref.process(c["x"], mask=allowed))
    assert lp.read_status(ws) == 0


@pytest.mark.parametrize("V", [64, 1001])
def test_rows_left_with_nothing_and_special_values(V):
    c = make(6, V, 6, seed=8)
    c["x"][1, :4] = torch.tensor([INF, -INF, float("nan"), torch.finfo(torch.float32).min])
    c["x"][2, :] = -INF
    c["x"][3, 0] = float("nan")
    c["history"], c["rep"] = [[0, 1, 2, 3]] * 6, [0.5] * 6   # (a factor above 1 would overflow f32 lowest)
    c["prompt"] = [1] * 6
    c["allowed"] = torch.ones(6, V, dtype=torch.bool)
    c["allowed"][0] = False                      # nothing left
    c["allowed"][3, 0] = False                   # a NaN in a masked place
    c["mask_index"] = list(range(6))
    c["bias"] = [{0: 1.0, V - 1: -INF} for _ in range(6)]
    out, status = call(c)
    assert status == 0 and (out[0] == -INF).all() and float(out[3, 0]) == -INF
    check(out, want_of(c))


def test_in_place():
    c = make(11, 4099, 5, hist=200, n_bias=9, seed=9)
    x = c["x"].cuda()
    out, _ = call(c, x=x, out=x)
    assert out.data_ptr() == x.data_ptr()
    check(x, want_of(c))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sx,so,shift", [(0, 0, 1), (4, 8, 0), (3, 3, 2), (1, 2, 0), (0, 5, 3)])
def test_strides_and_bases(dtype, sx, so, shift):
    T, V = 6, 2050
    c = make(T, V, 3, dtype, seed=10)
    xb = torch.zeros(T, V + sx + shift, dtype=dtype, device="cuda")
    ob = torch.full((T, V + so + shift), 5.0, device="cuda")
    xv, ov = xb[:, shift:shift + V], ob[:, shift:shift + V]
    xv.copy_(c["x"])
    wide = torch.zeros(c["allowed"].shape[0], (V + 31) // 32 + 3, dtype=torch.int32, device="cuda")
    wide[:, :(V + 31) // 32] = ref.pack_mask(c["allowed"]).cuda()
    out, status = call(c, x=xv, out=ov, mask=wide)
    assert status == 0
    check(ov, want_of(c))
    assert (ob[:, :shift] == 5).all() and (ob[:, shift + V:] == 5).all()


def test_same_result_each_time():
    c = make(4, 20000, 4, hist=4000, n_bias=40, seed=11)
    first, _ = call(c)
    for _ in range(3):
        assert torch.equal(call(c)[0], first)


def bits(*codes):
    return sum(1 << k for k in codes)


def test_bad_requests_get_nan_and_a_bit():
    c = make(6, 900, 6, seed=12, masked=False)
    good = want_of(c)
    for key, value in (("rep", 0.0), ("rep", INF), ("freq", float("nan")), ("pres", -INF)):
        d = dict(c, **{key: list(c[key])})
        d[key][2] = value
        out, status = call(d)
        assert status == bits(11) and torch.isnan(out[2]).all()
        keep = [0, 1, 3, 4, 5]
        check(out[keep], (good[0][keep], good[1][keep]))


def test_bad_offsets_get_nan_and_a_bit():
    c = make(6, 900, 6, seed=13, masked=False)
    c["rep"] = [1.25] * 6
    good = want_of(c)
    n = sum(len(h) for h in c["history"])
    bad = offsets(c["history"]).clone()
    bad[6] = n + 5                                # past the total
    out, status = call(c, history_offsets=bad)
    assert status == bits(4) and torch.isnan(out[5]).all()
    check(out[:5], (good[0][:5], good[1][:5]))
    bad = offsets(c["bias"]).clone()
    bad[1] = bad[2] + 1                           # decreasing
    out, status = call(c, bias_offsets=bad)
    assert status & bits(4) and torch.isnan(out[1]).all()
    off = i32([1, 2, 3, 4, 5, 5, 5])              # rows 0 and 5 belong to no request
    out, status = call(c, row_offsets=off)
    assert status == bits(4) and torch.isnan(out[[0, 5]]).all() and torch.isfinite(out[1:5]).all()
    allowed = torch.ones(2, 900, dtype=torch.bool)
    out, status = call(c, mask=ref.pack_mask(allowed).cuda(), mask_index=i32([0, 1, 2, -1, -2147483648, 0]))
    assert status == bits(4) and torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3, 4, 5]]).all()


def test_tokens_past_the_vocabulary_are_skipped_with_a_bit():
    c = make(3, 500, 3, seed=14)
    c["rep"] = [1.25] * 3
    c["history"][1] = c["history"][1] + [500, 2 ** 31 - 1, -1]
    d = dict(c, history=[[t for t in h if 0 <= t < 500] for h in c["history"]])
    out, status = call(c)
    assert status == bits(5)
    check(out, want_of(d))


def test_bias_ids_must_ascend():
    c = make(2, 500, 2, seed=15)
    out, status = call(c, bias_tokens=i32([5, 5, 9, 3]), bias_values=torch.zeros(4).cuda(), bias_offsets=i32([0, 2, 4]))
    assert status == bits(4)
    out, status = call(c, bias_tokens=i32([5, 9, 500]), bias_values=torch.zeros(3).cuda(), bias_offsets=i32([0, 2, 3]))
    assert status == bits(5)


def test_graph_replay_and_other_stream():
    c = make(8, 9000, 8, hist=100, seed=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = call(c, stream=s)
    s.synchronize()
    check(out, want_of(c))
    x, out = c["x"].cuda(), torch.empty(8, 9000, device="cuda")
    h, ho, ws = flat(c["history"]), offsets(c["history"]), lp.new_head_workspace()
    rep = torch.tensor(c["rep"]).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.process_logits(x, history=h, history_offsets=ho, repetition=rep, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    check(out, ref.process(c["x"], history=c["history"], rep=c["rep"]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_many_biases_and_uneven_requests(dtype):
    # more biases in a slice than a CTA keeps, requests of 0 to 70 rows
    V = 9000
    c = make(90, V, 6, dtype, hist=500, seed=17)
    c["off"] = [0, 1, 1, 5, 75, 76, 90]
    g = torch.Generator().manual_seed(9)
    c["bias"] = [{int(t): float(torch.randn(1, generator=g)) for t in torch.randperm(V, generator=g)[:3000].sort().values}
                 for _ in range(6)]
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


@pytest.mark.parametrize("T,B,V", [(3, 3, 50000), (6, 2, 9000), (40, 40, 40000)])
def test_long_histories_are_sorted_first(T, B, V):
    # a mean of more than 4096 tokens; one request neutral, one with few, prompts of any length
    c = make(T, V, B, hist=10, n_bias=30, seed=18)
    g = torch.Generator().manual_seed(7)
    lens = [9000 + int(torch.randint(0, 2000, (1,), generator=g)) for _ in range(B)]
    c["history"] = [(V * torch.rand(n, generator=g) ** 3).long().clamp_max(V - 1).tolist() for n in lens]
    c["prompt"] = [n // 3 for n in lens]
    if B > 2:
        c["history"][1], c["prompt"][1] = [5, 5, V - 1], 1
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))
    c["history"][-1][100] = V
    d = dict(c, history=[[t for t in h if t < V] for h in c["history"]])
    d["prompt"] = list(c["prompt"])
    d["prompt"][-1] -= 1
    c["rep"][-1] = d["rep"][-1] = 1.25
    out, status = call(c)
    assert status == bits(5)
    check(out, want_of(d))


def test_workspace_for_long_histories_is_checked():
    c = make(2, 5000, 2, seed=19)
    c["history"], c["prompt"] = [[1, 2, 3] * 3000] * 2, [0, 0]
    with pytest.raises(lp.LpError):
        call(c, workspace=lp.new_head_workspace())


def test_long_histories_in_place():
    c = make(20, 40001, 20, hist=12000, n_bias=50, seed=21)
    x = c["x"].cuda()
    _, status = call(c, x=x, out=x)
    assert status == 0
    check(x, want_of(c))


def test_long_history_of_few_tokens_sorted():
    # more than 15 bits of the output part, in slices of a table of 32 bits
    c = make(2, 60000, 2, seed=22)
    c["history"] = [[7] * 70000 + [8, 59999] * 1000, [1999] * 9000]
    c["prompt"] = [100, 9000]
    c["rep"], c["freq"], c["pres"] = [1.5, 2.0], [0.25, -0.5], [1.0, 0.0]
    out, status = call(c)
    assert status == 0
    check(out, want_of(c))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_far_apart(dtype):
    # the third row begins past 2^32 elements
    T, V, step = 3, 3001, 2 ** 31 + 20
    c = make(T, V, 2, dtype, hist=100, seed=23)
    far = torch.empty(2 * step + V, dtype=dtype, device="cuda")
    xv = far.as_strided((T, V), (step, 1))
    xv.copy_(c["x"])
    out, status = call(c, x=xv, out=xv if dtype == torch.float32 else None)
    assert status == 0
    check(out, want_of(c))
    del far, xv, out
    torch.cuda.empty_cache()


def test_a_smaller_call_in_a_larger_ones_workspace():
    # sized for a batch of short histories, used by the few long ones that are left of it
    c = make(4, 9000, 4, hist=10, seed=24)
    g = torch.Generator().manual_seed(24)
    c["history"] = [torch.randint(0, 9000, (10000 + 7 * b,), generator=g).tolist() for b in range(4)]
    ws = lp.new_head_workspace(requests=64, history=60000)
    out, status = call(c, workspace=ws)
    assert status == 0
    check(out, want_of(c))
