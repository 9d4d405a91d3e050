"""Draw of tokens (lp_head_sample) against the 64-bit formula: every filter and their combinations, types,
lengths and alignments, ties, masks, extreme values, the errors found on the device."""

import math

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import parity
from tests import sample_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
LAST = 1.0 - 2.0 ** -24  # the largest random number
# A weight is within 2^-32 of the formula's: three roundings of f32 to what is left of a power of two after a
# table of 256 (2^-8.5 of the weight, so 3 * 2^-33.5) and the table's own 2^-49. A comparison of sums of such
# weights that is nearer than twice that may turn over.
NEAR = 2.0 ** -31


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


def run(x, u, tau=None, k=None, p=None, q=None, off=None, ws=None, **kw):
    t = lambda v, d: None if v is None else torch.tensor(v, dtype=d, device="cuda")
    ws = lp.new_head_workspace(draws=x.shape[0], vocab=x.shape[1]) if ws is None else ws
    logprob = torch.full((x.shape[0],), 7.0, device="cuda")
    x = x if x.is_cuda else x.cuda()
    got = lp.sample(x, t(u, F32), t(off, torch.int32), t(tau, F32), t(k, torch.int32), t(p, F32), t(q, F32),
                    out_logprob=logprob, workspace=ws, **kw)
    return got.tolist(), logprob.tolist(), lp.read_status(ws)


def check(x, u, tau=None, k=None, p=None, q=None, off=None, skipped=0.02, **kw):
    """Tokens are the formula's, logprobs to four roundings of f32 (the difference, the quotient, the logarithm
    and the sum, all of one sign): 4 * 2^-24 of the value and the logarithm's two units in the last place."""
    T = x.shape[0]
    got, logprob, status = run(x, u, tau, k, p, q, off, **kw)
    assert status == 0
    of = list(range(T)) if off is None else [b for b in range(len(off) - 1) for _ in range(off[b], off[b + 1])]
    at = lambda v, t, d: d if v is None else torch.tensor(v[of[t]], dtype=F32).item()
    x, close = x.cpu(), 0
    for t in range(T):
        token, lw, margin = ref.draw(x[t], torch.tensor(u[t], dtype=F32).item(), at(tau, t, 1.0), 0 if k is None else k[of[t]],
                                     at(p, t, 1.0), at(q, t, 0.0))
        if margin < NEAR:
            close += 1
            continue
        assert got[t] == token, (t, got[t], token, margin)
        assert abs(logprob[t] - lw) <= (4 * 2.0 ** -24 + 2 * 2.0 ** -23) * abs(lw) + 2.0 ** -40, (t, logprob[t], lw)
    assert close <= skipped * T
    return got


def logits(T, V, dtype=F32, seed=0, scale=3.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + V)
    return (scale * torch.randn(T, V, generator=g)).to(dtype)


def uniforms(T, seed=0):
    return torch.rand(T, generator=torch.Generator().manual_seed(seed + 99)).tolist()


SETTINGS = {
    "none": {}, "hot": dict(tau=1.7), "cold": dict(tau=0.3), "greedy": dict(tau=0.0),
    "k1": dict(k=1), "k2": dict(k=2), "k50": dict(k=50), "k300": dict(k=300), "k1024": dict(k=1024), "k1025": dict(k=1025),
    "k5000": dict(k=5000), "p0": dict(p=0.0), "p1e-9": dict(p=1e-9), "p0.5": dict(p=0.5), "p0.9": dict(p=0.9),
    "p0.999": dict(p=0.999), "p_last": dict(p=LAST), "q0.05": dict(q=0.05), "q1": dict(q=1.0), "q1e-6": dict(q=1e-6),
    "k50_p0.9": dict(k=50, p=0.9), "k50_p0.1": dict(k=50, p=0.1), "k2000_p0.3": dict(k=2000, p=0.3),
    "k2000_p0.999": dict(k=2000, p=0.999), "p0.95_q0.1": dict(p=0.95, q=0.1), "k20_q0.3": dict(k=20, q=0.3),
    "all": dict(tau=0.8, k=100, p=0.95, q=0.02), "k2000_q": dict(k=2000, p=0.9, q=0.01),
}


@pytest.mark.parametrize("name", SETTINGS)
@pytest.mark.parametrize("V,dtype", [(50001, F32), (20000, BF16), (128256, F32), (1000, F16), (160000, BF16)])
def test_settings(name, V, dtype):
    s, T = SETTINGS[name], 5
    x = logits(T, V, dtype, seed=1)
    # (p next to 1 ends among tokens of a share of 2^-30 or less: the margin is often below 2^-31 there)
    check(x, uniforms(T - 2) + [0.0, LAST], skipped=1.0 if name == "p_last" else 0.02, **{n: [v] * T for n, v in s.items()})


@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 7, 8, 9, 31, 33, 127, 2047, 2048, 2049, 4096, 16381, 16384, 16385, 16388,
                               32767, 32769, 65537, 131073, 262144, 393216])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(V, dtype):
    x = logits(4, V, dtype, seed=2, scale=2.0)
    for s in (dict(), dict(p=[0.8] * 4), dict(k=[40] * 4, p=[0.9] * 4), dict(q=[0.1] * 4), dict(tau=[0.0] * 4)):
        check(x, uniforms(4, V), **s)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift,extra", [(0, 1), (1, 0), (1, 1), (3, 5), (7, 8)])
def test_places_and_strides(dtype, shift, extra):
    T, V = 9, 5003
    g = torch.Generator().manual_seed(3)
    flat = (3 * torch.randn(T * (V + extra) + shift + 8, generator=g)).to(dtype).cuda()
    flat[:shift] = float("nan")  # what lies around the rows is not read as theirs
    flat[shift + T * (V + extra):] = float("inf")
    x = flat[shift:shift + T * (V + extra)].view(T, V + extra)
    x[:, V:] = float("inf")
    x = x[:, :V]
    for s in (dict(), dict(p=[0.9] * T), dict(k=[30] * T), dict(q=[0.02] * T)):
        check(x, uniforms(T), **s)


@pytest.mark.parametrize("V", [3000, 40000, 200000])
@pytest.mark.parametrize("name", ["none", "greedy", "k1", "k50", "k1024", "k1025", "k2000_p0.3", "p0.5", "p0.9", "p0.999",
                                  "q1", "k50_p0.1"])
def test_all_values_alike(V, name):
    T = 6
    x = torch.full((T, V), -2.5)
    u = [0.0, 0.25, 0.5, 0.123456, 0.999, LAST]
    # equal weights: the sums are whole numbers of them, and the borders lie exactly at i / n; the numbers above
    # that fall on one belong to the token behind it
    s = {n: [v] * T for n, v in SETTINGS[name].items()}
    check(x, u, skipped=1.0, **s)


@pytest.mark.parametrize("V", [5000, 50000])
def test_ties_of_every_size(V):
    # three values, each held by thousands: cuts inside each of them
    g = torch.Generator().manual_seed(5)
    x = torch.randint(0, 3, (12, V), generator=g).float()
    k = [1, 10, V // 3 - 100, V // 3 + 500, V // 2, 2 * V // 3 + 700, V - 5, V, V + 9, 1024, 1025, 2000]
    check(x, uniforms(12), k=k)
    check(x, uniforms(12, 1), p=[0.01, 0.1, 0.3, 0.5, 0.6, 0.7, 0.8, 0.9, 0.95, 0.97, 0.99, 0.9999])
    # (of equal weights the sums can meet p of the whole exactly: not decided here)
    check(x, uniforms(12, 2), k=k, p=[0.9, 0.5, 0.3, 0.9, 0.7, 0.95, 0.2, 0.99, 0.5, 0.6, 0.7, 0.8], skipped=0.3)
    check(x, uniforms(12, 3), k=k, q=[0.2, 0.13, 0.5, 0.01] * 3)


def test_many_random_numbers_cover_the_row():
    # one row, random numbers all over [0, 1): every token whose share is wider than their distance appears
    T, V = 2000, 300
    x = logits(1, V, F32, seed=6).expand(T, V).contiguous()
    u = [(i + 0.5) / T for i in range(T)]
    got = check(x, u)
    share = torch.softmax(x[0].double(), 0)
    assert all(got.count(t) > 0 for t in range(V) if float(share[t]) > 1.0 / T)
    assert sorted(got) == got  # in the order of the ids
    check(x, u, p=[0.7] * T)
    check(x, u, k=[17] * T)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("allowed", [0.5, 0.01, 0.0005])
def test_masked_rows(dtype, allowed):
    T, V = 8, 30011
    g = torch.Generator().manual_seed(8)
    x = logits(T, V, dtype, seed=8)
    keep = torch.rand(T, V, generator=g) < allowed
    keep[:, 17] = True
    x[~keep] = -math.inf
    x[0] = -math.inf
    x[0, V - 1] = -1e4  # a single token
    for s in (dict(), dict(p=[0.9] * T), dict(k=[50] * T), dict(k=[2000] * T, p=[0.8] * T), dict(q=[0.1] * T), dict(tau=[0.0] * T)):
        got = check(x, uniforms(T), **s)
        assert got[0] == V - 1


@pytest.mark.parametrize("s", [dict(), dict(k=[5] * 6), dict(p=[0.5] * 6), dict(tau=[0.0] * 6), dict(q=[0.5] * 6)])
@pytest.mark.parametrize("V", [7, 50000])
def test_rows_without_a_distribution(s, V):
    x = logits(6, V, seed=9)
    x[1] = -math.inf
    x[2, V - 1] = math.nan
    x[4, 0] = math.inf
    x[5, :] = math.nan
    u = uniforms(6)
    got, logprob, status = run(x, u, **s)
    assert status == 1 << 14  # LP_ERR_LOGITS
    assert [got[t] for t in (1, 2, 4, 5)] == [-1] * 4 and all(math.isnan(logprob[t]) for t in (1, 2, 4, 5))
    for t in (0, 3):
        one = {n: v[0] for n, v in s.items()}
        assert got[t] == ref.draw(x[t], torch.tensor(u[t]).item(), **one)[0]


def test_values_and_temperatures_far_out():
    V, T = 4000, 10
    x = logits(T, V, seed=10)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] += 1e6
    x[3] -= 3e4
    x[4] = torch.linspace(-1.7e38, 1.7e38, V)
    x[5, ::2] *= 1e-42
    x[6] = -torch.arange(V).float() * 0.01
    x[7] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    x[8] = -x[8].abs() * 1e20
    tau = [1e30, 1e-30, 0.5, 2.0, 1e30, 1.0, 0.25, 1.0, 1e20, 1e-6]
    for s in (dict(), dict(p=[0.9] * T), dict(k=[100] * T, p=[0.99] * T), dict(q=[0.3] * T), dict(p=[0.9999] * T)):
        check(x, uniforms(T, 4), tau=tau, skipped=0.2, **s)


def test_both_zeros_are_one_value():
    x = torch.full((3, 100), -5.0)
    x[:, 40], x[:, 60] = -0.0, 0.0
    assert check(x, [0.1, 0.5, 0.9], tau=[0.0] * 3) == [40, 40, 40]
    assert check(x, [0.1, 0.5, 0.9], k=[1] * 3) == [40, 40, 40]
    assert check(x, [0.1, 0.4999, 0.9], k=[2] * 3) == [40, 40, 60]


def test_weights_below_the_smallest():
    # 2^-40 of the largest counts, less does not; a random number of 0 takes the first that counts
    x = torch.full((2, 3000), -40.0 * math.log(2.0) - 0.001)
    x[:, 2000] = 0.0
    x[0, 1000] = -40.0 * math.log(2.0) + 0.001
    assert check(x, [0.0, 0.0]) == [1000, 2000]


def test_requests_of_several_rows_and_bad_settings():
    V, off = 6000, [0, 1, 4, 4, 9, 10]
    x = logits(10, V, seed=11)
    tau, k, p, q = [0.7, 1.0, 1.0, 1.3, 0.0], [0, 3, 1, 0, 9], [0.9, 1.0, 0.5, 0.8, 1.0], [0.0, 0.0, 0.0, 0.05, 0.0]
    check(x, uniforms(10), tau, k, p, q, off)
    # rows in no request
    got, logprob, status = run(x, uniforms(10), tau, k, p, q, [1, 2, 4, 4, 8, 8])
    assert status == 1 << 4 and [t for t in range(10) if got[t] == -1] == [0, 8, 9]
    # settings out of range
    bad, nan, inf = [1.0] * 10, math.nan, math.inf
    got, _, status = run(x, uniforms(10), tau=[1.0, -1.0, nan, inf, 0.0] + [1.0] * 5)
    assert status == 1 << 8 and [t for t in range(10) if got[t] == -1] == [1, 2, 3]
    got, _, status = run(x, uniforms(10), p=[1.0, 1.5, -0.1, nan, 0.0] + [1.0] * 5)
    assert status == 1 << 13 and [t for t in range(10) if got[t] == -1] == [1, 2, 3]
    got, _, status = run(x, uniforms(10), q=[1.0, 1.5, -0.1, nan, 0.0] + [1.0] * 5)
    assert status == 1 << 13 and [t for t in range(10) if got[t] == -1] == [1, 2, 3]
    got, _, status = run(x, [0.0, 1.0, -1e-9, nan, inf] + [0.5] * 5)
    assert status == 1 << 13 and [t for t in range(10) if got[t] == -1] == [1, 2, 3, 4]
    # a negative or large k is none
    assert run(x, uniforms(10), k=[-1, -2 ** 31, 2 ** 31 - 1, V, 0] * 2)[0] == run(x, uniforms(10))[0]


def test_streams_graphs_and_repetition():
    T, V = 64, 50001
    x = logits(T, V, BF16, seed=12).cuda()
    u = torch.tensor(uniforms(T), device="cuda")
    p, k = torch.full((T,), 0.9, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda") * 40
    ws = [lp.new_head_workspace(draws=T, vocab=V) for _ in range(2)]
    want = lp.sample(x, u, top_p=p, top_k=k, workspace=ws[0])
    torch.cuda.synchronize()
    outs, streams = [torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for o, s, w in zip(outs, streams, ws):
            lp.sample(x, u, top_p=p, top_k=k, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.sample(x, u, top_p=p, top_k=k, out=outs[0], workspace=ws[0])
    u.copy_(torch.tensor(uniforms(T, 5), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    again = lp.sample(x, u, top_p=p, top_k=k, workspace=ws[0])
    assert torch.equal(outs[0], again) and not torch.equal(again, want)


def test_rows_past_32_bits():
    # a matrix of more than 2^32 elements, its last rows
    T, V = 16500, 262144
    x = torch.empty(T, V, dtype=F16, device="cuda")
    x.fill_(-3.0)
    x[-2:] = logits(2, V, F16, seed=13).cuda()
    u = torch.full((T,), 0.37, device="cuda")
    got = lp.sample(x, u, top_p=torch.full((T,), 0.5, device="cuda"), workspace=lp.new_head_workspace(draws=T, vocab=V)).tolist()
    for t in (T - 2, T - 1, 0):
        token, _, margin = ref.draw(x[t].cpu(), torch.tensor(0.37).item(), p=0.5)
        assert got[t] == token or margin < NEAR
    assert len(set(got[:-2])) == 1


@pytest.mark.parametrize("T,V,dtype", [(256, 32000, BF16), (300, 9973, F32)])
def test_mixed_batches(T, V, dtype):
    g = torch.Generator().manual_seed(14)
    x = logits(T, V, dtype, seed=14, scale=2.5)
    r = lambda: torch.rand(T, generator=g)
    tau = torch.where(r() < 0.1, 0.0, 0.4 + r()).tolist()
    k = torch.where(r() < 0.5, 0, (2 * 500 ** r()).int()).tolist()
    p = torch.where(r() < 0.5, 1.0, 0.3 + 0.69 * r()).tolist()
    q = torch.where(r() < 0.8, 0.0, 0.2 * r()).tolist()
    check(x, r().tolist(), tau, k, p, q)


@pytest.mark.parametrize("T", [200, 456, 457, 1500, 4096, 4097])
def test_every_row_of_many_is_drawn(T):
    # rows of all kinds in turn, some without a token: each is drawn once, whatever the order they are taken in
    V = 130
    x = logits(T, V, F32, seed=15)
    off = [0] + [i for i in range(1, T) if i % 5 in (1, 2)] + [T]  # requests of one row and of four
    B = len(off) - 1
    tau = [0.0 if b % 11 == 3 else 0.5 + b % 7 / 7 for b in range(B)]
    k = [(0, 1, 20, 0, 129, 500)[b % 6] for b in range(B)]
    p = [(1.0, 0.9, 0.3)[b % 3] for b in range(B)]
    q = [0.05 if b % 4 == 0 else 0.0 for b in range(B)]
    u = uniforms(T, 15)
    check(x, u, tau, k, p, q, off)
    bad = [b for b in range(B) if b % 13 == 5]
    of = [b for b in range(B) for _ in range(off[b], off[b + 1])]
    want, want_logprob, _ = run(x, u, tau, k, p, q, off)
    got, logprob, status = run(x, u, [math.nan if b in set(bad) else v for b, v in enumerate(tau)], k, p, q, off)
    assert status == 1 << 8
    for t in range(T):
        if of[t] in set(bad):
            assert got[t] == -1 and math.isnan(logprob[t])
        else:
            assert got[t] == want[t] and logprob[t] == want_logprob[t]


@pytest.mark.parametrize("V,dtype", [(30001, F16), (128256, F32), (5000, BF16)])
@pytest.mark.parametrize("scale", [0.5, 3.0])
def test_large_k_with_top_p(V, dtype, scale):
    k = [300, 383, 384, 385, 500, 700, 900, 991, 992, 993, 1000, 1023, 1024, 1025, 1500, 3000]
    x, u = logits(len(k), V, dtype, seed=16, scale=scale), uniforms(len(k), 16)
    for p in (1.0, 0.999, 0.8, 0.2):
        check(x, u, k=k, p=[p] * len(k))
    check(x, u, k=k, p=[0.8] * len(k), q=[0.1] * len(k))


def test_graphs_that_share_a_workspace():
    # more rows than are drawn at a time: the order is made anew by every call
    T, V = 500, 9000
    x = [logits(T, V, BF16, seed=17 + i).cuda() for i in range(2)]
    u = torch.tensor(uniforms(T, 17), device="cuda")
    t = torch.arange(T, device="cuda")
    k = [torch.where(t % 3 == i, 700, 0).int() for i in range(2)]
    p = [torch.where(t % 5 == i, 0.9, 1.0).float() for i in range(2)]
    ws = lp.new_head_workspace(draws=T, vocab=V)
    want = [lp.sample(x[i], u, top_k=k[i], top_p=p[i], workspace=lp.new_head_workspace(draws=T, vocab=V)) for i in range(2)]
    outs = [torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            lp.sample(x[i], u, top_k=k[i], top_p=p[i], out=outs[i], workspace=ws)
    for _ in range(5):
        for i in range(2):
            graphs[i].replay()
            lp.sample(x[1 - i], u, top_k=k[1 - i], top_p=p[1 - i], workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and lp.read_status(ws) == 0
