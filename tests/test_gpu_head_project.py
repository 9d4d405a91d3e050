"""Projection with adapters (lp_head_project) against the 64-bit formula: types, row counts
across the tile sizes, odd vocabularies and widths, strides, adapters in any order, ragged
requests, and the errors found on the device."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import parity

pytestmark = pytest.mark.gpu

BF16, F16, E4M3, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


class Case:
    """Inputs on the CPU; ``want`` and ``mag`` (the sum of the products' magnitudes) in 64 bits."""

    def __init__(self, T, H, V, dtype=BF16, A=0, rank=0, ids=None, off=None, seed=0, lora_dtype=None, unit=False):
        g = torch.Generator().manual_seed(seed * 977 + T * 31 + V)
        rn = lambda *s: torch.randn(*s, generator=g)
        self.T, self.V, self.A, self.rank = T, V, A, rank
        x, w = rn(T, H), rn(V, H) * (2.0 / H ** 0.5)
        self.sx = self.sw = None
        if dtype == E4M3:
            self.sx, self.sw = x.abs().amax(1) / 448, w.abs().amax(1) / 448
            x, w = x / self.sx[:, None], w / self.sw[:, None]
        self.x, self.w = x.to(dtype), w.to(dtype)
        xd, wd = self.x.double(), self.w.double()
        if dtype == E4M3:
            xd, wd = xd * self.sx.double()[:, None], wd * self.sw.double()[:, None]
        self.want, self.mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
        self.off, self.scale = off, None
        if A:
            at = dtype if lora_dtype is None else lora_dtype
            self.la, self.lb = (rn(A, rank, H) / H ** 0.5).to(at), (rn(A, V, rank) * 0.4).to(at)
            self.scale = None if unit else (0.5 + torch.rand(A, generator=g))
            B = T if off is None else len(off) - 1
            self.ids = torch.randint(-1, A, (B,), generator=g).tolist() if ids is None else ids
            of = list(range(T)) if off is None else [b for b in range(B) for _ in range(off[b], off[b + 1])]
            for t, b in enumerate(of):
                a = self.ids[b]
                if a >= 0:
                    s = 1.0 if unit else float(self.scale[a])
                    u, um = s * (self.la[a].double() @ xd[t]), abs(s) * (self.la[a].double().abs() @ xd[t].abs())
                    self.want[t] += self.lb[a].double() @ u
                    self.mag[t] += self.lb[a].double().abs() @ um

    def run(self, out_dtype=F32, out=None, x=None, w=None, ws=None, **kw):
        c = lambda t: None if t is None else t.cuda()
        self.ws = lp.new_head_workspace(self.T, self.rank) if ws is None else ws
        args = dict(x_scale=c(self.sx), weight_scale=c(self.sw))
        if self.A:
            args.update(lora_a=c(self.la), lora_b=c(self.lb), adapter_scale=c(self.scale),
                        adapter_ids=torch.tensor(self.ids, dtype=torch.int32).cuda(),
                        row_offsets=None if self.off is None else torch.tensor(self.off, dtype=torch.int32).cuda())
        args.update(kw)
        return lp.project(c(self.x) if x is None else x, c(self.w) if w is None else w, workspace=self.ws,
                          out=out, out_dtype=out_dtype if out is None else None, **args)

    def check(self, out, rows=slice(None)):
        """Exact products in a chain of f32 sums: each of the H / 16 (or 32) steps and of the
        rank's terms loses at most 2^-23 of a partial sum, itself below the sum of magnitudes;
        in practice errors add like a random walk or cancel, but the bound used is the proven
        one, per step, over 16 products at a time: (H / 16 + 2 rank + 8) 2^-23 of it."""
        got = out.double().cpu()[rows]
        want, mag = self.want[rows], self.mag[rows]
        steps = self.x.shape[1] / 16 + 2 * self.rank + 8
        half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[out.dtype]
        bound = mag * steps * 2.0 ** -23 + want.abs() * half * (1 + 2.0 ** -10) + 2.0 ** -25 * (out.dtype == F16)
        assert torch.isfinite(got).all()
        worst = ((got - want).abs() - bound).max()
        assert worst <= 0, float(worst)
        assert lp.read_status(self.ws) == 0


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 100, 129, 256])
def test_rows_of_one_tile(T, dtype):
    c = Case(T, 512, 1000, dtype, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("T", [257, 300, 513, 1000])
def test_rows_of_several_tiles(T):
    c = Case(T, 256, 777, BF16, seed=2)
    c.check(c.run(BF16))
    c.check(c.run(F32))


@pytest.mark.parametrize("V", [1, 2, 127, 128, 129, 1000, 20001, 50048])
def test_vocabularies(V):
    c = Case(19, 192, V, BF16, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("dtype,H", [(BF16, 8), (BF16, 64), (BF16, 72), (F16, 1000), (BF16, 4096), (F16, 8200),
                                     (E4M3, 16), (E4M3, 128), (E4M3, 144), (E4M3, 4096)])
def test_widths(dtype, H):
    c = Case(40, H, 300, dtype, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("out_dtype", [F32, BF16, F16])
def test_output_types(dtype, out_dtype):
    c = Case(50, 320, 555, dtype, A=3, rank=8, seed=5, lora_dtype=BF16 if dtype == E4M3 else None)
    c.check(c.run(out_dtype))


@pytest.mark.parametrize("rank", [1, 2, 5, 8, 12, 16, 17, 24, 32, 48, 63, 64])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_ranks(rank, dtype):
    c = Case(37, 256, 333, dtype, A=4, rank=rank, seed=6, lora_dtype=F16 if dtype == E4M3 else None)
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 16, 31, 64, 200, 300])
def test_adapters_in_any_order(T):
    c = Case(T, 128, 400, F16, A=7, rank=16, seed=7)
    c.check(c.run())


def test_every_row_its_own_adapter_and_none_and_all_one():
    T = 70
    for ids in ([i for i in range(T)], [-1] * T, [3] * T, [0, 69] * (T // 2)):
        c = Case(T, 128, 260, BF16, A=T, rank=8, ids=ids, seed=8, unit=True)
        c.check(c.run())


@pytest.mark.parametrize("off", [[0, 5, 6, 40], [0, 130, 131, 300, 520], [0, 0, 7, 7, 9]])
def test_ragged_requests(off):
    c = Case(off[-1], 192, 300, BF16, A=3, rank=24, off=off, seed=9)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_strides(dtype):
    c = Case(21, 256, 501, dtype, A=2, rank=4, seed=10, lora_dtype=BF16)
    xb = torch.zeros(21, 256 + 48, device="cuda").to(dtype)
    wb = torch.zeros(501, 256 + 16, device="cuda").to(dtype)
    xb[:, 16:272].copy_(c.x)
    wb[:, :256].copy_(c.w)
    ob = torch.full((21, 510), 7.0, device="cuda")
    c.run(out=ob[:, 3:504], x=xb[:, 16:272], w=wb[:, :256])
    c.check(ob[:, 3:504])
    assert (ob[:, :3] == 7).all() and (ob[:, 504:] == 7).all()


def test_values_of_other_rows_do_not_leak():
    # rows and vocabulary entries of the same tile: NaN and infinity stay in theirs
    c = Case(20, 128, 200, BF16, A=2, rank=8, ids=[0, 1] * 10, seed=11)
    x, w = c.x.clone(), c.w.clone()
    x[3, 5] = float("nan")
    w[77, 0] = float("inf")
    out = c.run(x=x.cuda(), w=w.cuda())
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[:, 77]).any()
    keep = [i for i in range(20) if i != 3]
    cols = [v for v in range(200) if v != 77]
    good = c.run()
    assert torch.equal(out[keep][:, cols], good[keep][:, cols])
    c.check(good)


def test_bad_adapter_ids_and_offsets():
    c = Case(9, 128, 150, BF16, A=2, rank=8, ids=[0, 1, 0, 1, -1, 0, 1, 0, 1], seed=12)
    good = c.run()
    ids = torch.tensor([0, 1, 2, 1, -5, 0, 2 ** 31 - 1, 0, 1], dtype=torch.int32).cuda()
    out = c.run(adapter_ids=ids)
    assert lp.read_status(c.ws) == 1 << 10
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.isnan(out[[2, 6]]).all() and torch.equal(out[keep], good[keep])
    off = torch.tensor([1, 2, 3, 4, 5, 6, 7, 8, 8, 8], dtype=torch.int32).cuda()
    out = c.run(row_offsets=off)
    assert lp.read_status(c.ws) == 1 << 4
    assert torch.isnan(out[[0, 8]]).all() and torch.isfinite(out[1:8]).all()


def test_same_result_each_time_and_in_a_graph():
    c = Case(48, 1024, 3000, BF16, A=5, rank=16, seed=13)
    first = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), first)
    x, w, la, lb, sc = (t.cuda() for t in (c.x, c.w, c.la, c.lb, c.scale))
    ids = torch.tensor(c.ids, dtype=torch.int32).cuda()
    ws, out = lp.new_head_workspace(48, 16), torch.empty(48, 3000, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            lp.project(x, w, lora_a=la, lora_b=lb, adapter_scale=sc, adapter_ids=ids, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_chain_on_one_stream():
    # norm -> projection -> processing without a wait between: each sees what came before
    T, H, V = 33, 1024, 5000
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(T, H, generator=g).cuda(), (torch.randn(V, H, generator=g) / 16).to(BF16).cuda()
    ws = lp.new_head_workspace()
    gain = torch.ones(H, device="cuda")
    for _ in range(20):
        y = lp.rms_norm(x, gain, 1e-5).to(BF16)
        want = lp.project(y, w, workspace=ws)
        torch.cuda.synchronize()
        z = lp.rms_norm(x.to(BF16), gain, 1e-5)
        one = lp.project(z, w, workspace=ws)
        two = lp.process_logits(one, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(two, lp.process_logits(lp.project(z, w, workspace=ws), workspace=ws))
        assert (two - want).abs().max() < 0.5
    assert lp.read_status(ws) == 0


@pytest.mark.parametrize("dtype,lora_dtype", [(BF16, BF16), (F16, F16), (E4M3, BF16), (E4M3, F16)])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_long_requests(dtype, lora_dtype, rank, out_dtype):
    # whole blocks of 32 rows with one adapter, blocks of several, rows without one; two tiles
    off = [0, 3, 130, 200, 232, 296, 330]
    c = Case(330, 272, 300, dtype, A=3, rank=rank, ids=[0, 2, -1, 1, 1, 0], off=off, seed=14, lora_dtype=lora_dtype)
    c.check(c.run(out_dtype))


@pytest.mark.parametrize("scale", [1e-18, 1e18])
def test_sizes_of_u_far_from_one(scale):
    # float16 adapters of values whose u leaves float16's range, through adapter_scale
    off = [0, 100, 230]
    c = Case(230, 256, 200, F16, A=2, rank=16, ids=[0, 1], off=off, seed=15)
    factor = torch.full((2,), scale)
    base = Case(230, 256, 200, F16, seed=15)
    base.x, base.w = c.x, c.w
    zero = base.run()
    out = c.run(adapter_scale=factor.cuda()).double().cpu()
    xd = c.x.double()
    for b in range(2):
        r = slice(off[b], off[b + 1])
        u = xd[r] @ c.la[b].double().t()
        part = u @ c.lb[b].double().t() * scale
        mag = (xd[r].abs() @ c.la[b].double().abs().t()) @ c.lb[b].double().abs().t() * scale
        ref = zero.double().cpu()[r] + part
        assert ((out[r] - ref).abs() <= (mag + zero.double().cpu()[r].abs()) * 64 * 2.0 ** -23).all()


@pytest.mark.parametrize("T,off", [(40, None), (256, None), (200, [0, 64, 130, 200])])
def test_infinities_of_one_adapter_stay_with_its_rows(T, off):
    B = T if off is None else len(off) - 1
    c = Case(T, 128, 140, BF16, A=2, rank=16, ids=[b % 2 for b in range(B)], off=off, seed=16)
    lb = c.lb.clone()
    lb[1, 7, 3] = float("inf")
    lb[1, 9, 0] = float("nan")
    out = c.run(lora_b=lb.cuda())
    mine = torch.tensor([b for b in range(B) for _ in range(1 if off is None else off[b + 1] - off[b])]) % 2 == 1
    assert torch.isfinite(out.cpu()[~mine]).all()
    assert not torch.isfinite(out.cpu()[mine][:, [7, 9]]).any()
    cols = [v for v in range(140) if v not in (7, 9)]
    assert torch.isfinite(out.cpu()[mine][:, cols]).all()


def test_many_tiles_of_mixed_requests():
    off = [0]
    g = torch.Generator().manual_seed(5)
    while off[-1] < 1500:
        off.append(off[-1] + int(torch.randint(1, 120, (1,), generator=g)))
    c = Case(off[-1], 128, 700, BF16, A=6, rank=32, off=off, seed=17)
    c.check(c.run())
    c.check(c.run(BF16))


# Sizes for which pairs of CTAs are taken, whose tensor cores also multiply the adapters of
# blocks of 32 rows with one adapter or two.
SEGMENTS = {
    # blocks of one adapter, of two, of one and none; tiles of 160 rows
    "ragged": ([0, 3, 130, 200, 232, 296, 300], [0, 2, -1, 1, 1, 0], 64),
    "one tile": ([0, 40, 96, 160, 168, 256], [0, 1, 2, 0, 1], 16),
    # two or three adapters in every block: more second ones than there are free columns
    "short": (list(range(0, 241, 20)) + [256], [b % 3 for b in range(13)], 24),
    "a row aside": ([0, 63, 64, 65, 200], [1, 0, -1, 1], 8),
}


@pytest.mark.parametrize("dtype,lora_dtype", [(BF16, BF16), (F16, F16), (E4M3, BF16), (E4M3, F16)])
@pytest.mark.parametrize("name", sorted(SEGMENTS))
def test_segments_on_pairs(name, dtype, lora_dtype):
    off, ids, rank = SEGMENTS[name]
    c = Case(off[-1], 512, 20001, dtype, A=3, rank=rank, ids=ids, off=off, seed=18, lora_dtype=lora_dtype)
    for out_dtype in (F32, BF16, F16):
        c.check(c.run(out_dtype))


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_infinities_of_one_adapter_on_pairs(dtype, out_dtype):
    off, ids, rank = SEGMENTS["one tile"]
    c = Case(256, 512, 20001, dtype, A=3, rank=rank, ids=ids, off=off, seed=19, lora_dtype=BF16 if dtype == E4M3 else None)
    lb = c.lb.clone()
    lb[1, 7, 3] = float("inf")
    lb[1, 19999, 0] = float("nan")
    out = c.run(out_dtype, lora_b=lb.cuda()).cpu()
    mine = torch.tensor([ids[b] == 1 for b in range(len(ids)) for _ in range(off[b], off[b + 1])])
    assert torch.isfinite(out[~mine]).all()
    assert not torch.isfinite(out[mine][:, [7, 19999]]).any()
    cols = [v for v in range(20001) if v not in (7, 19999)]
    assert torch.isfinite(out[mine][:, cols]).all()


def test_rows_far_apart():
    # x's and out's third row begin past 2^32 elements
    T, step = 3, 2 ** 31 + 64
    c = Case(T, 128, 300, BF16, A=2, rank=8, ids=[0, 1, -1], seed=20)
    far, fo = (torch.empty(2 * step + 300, dtype=BF16, device="cuda") for _ in range(2))
    xv, ov = far.as_strided((T, 128), (step, 1)), fo.as_strided((T, 300), (step, 1))
    xv.copy_(c.x)
    c.run(out=ov, x=xv)
    c.check(ov)
    del far, fo, xv, ov
    torch.cuda.empty_cache()
