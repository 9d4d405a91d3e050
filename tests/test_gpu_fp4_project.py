"""Projection of 4-bit rows (lp_head_project4) against the 64-bit formula: both blocks, output types, row
counts across the tile sizes, odd vocabularies and widths, strides, scales that are not finite."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import fp4_reference as ref
from tests import parity

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


class Case:
    def __init__(self, T, H, V, block, seed=0, row_scales=True):
        self.T, self.H, self.V, self.block = T, H, V, block
        self.x, self.xs, self.xr = ref.random_rows(T, H, block, seed * 7 + T)
        self.w, self.ws, self.wr = ref.random_rows(V, H, block, seed * 7 + V + 100000)
        if not row_scales:
            self.xr = self.wr = None
        xd, wd = (ref.values(*ref.unpack(c), s, r, block) for c, s, r in ((self.x, self.xs, self.xr), (self.w, self.ws, self.wr)))
        self.want, self.mag = xd @ wd.t(), xd.abs() @ wd.abs().t()

    def tiles(self):
        return (lp.tile_fp4_scales(ref.scale_bytes(s, self.block)).cuda() for s in (self.xs, self.ws))

    def run(self, out_dtype=F32, out=None, x=None, w=None):
        c = lambda t: None if t is None else t.cuda()
        xs, ws = self.tiles()
        self.space = lp.new_head_workspace()
        return lp.project_fp4(c(self.x) if x is None else x, xs, c(self.w) if w is None else w, ws, self.block,
                              c(self.xr), c(self.wr), out=out, out_dtype=out_dtype if out is None else None,
                              workspace=self.space)

    def check(self, out):
        """The products of two codes and their scales are exact, and so is the sum of a block's in f32 (12 bits and
        4 more); each of the H / 16 sums of blocks loses at most 2^-23 of a partial sum, itself below the sum of
        magnitudes; the row scales are two products more. In f16 a value of 65520 (half a step past the
        largest, 65504) or more rounds to infinity."""
        got = out.double().cpu()
        half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[out.dtype]
        bound = self.mag * (self.H / 16 + 8) * 2.0 ** -23 + self.want.abs() * half * (1 + 2.0 ** -10)
        bound += 2.0 ** -25 * (out.dtype == F16)
        most = 65520.0 if out.dtype == F16 else float("inf")
        fine = self.want.abs() + bound < most
        assert bool((got[self.want.abs() - bound >= most].abs() == float("inf")).all())
        assert torch.isfinite(got[fine]).all()
        worst = ((got - self.want).abs() - bound)[fine].max()
        assert worst <= 0, float(worst)
        assert lp.read_status(self.space) == 0


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 100, 128])
def test_rows_of_one_tile(T, block):
    c = Case(T, 512, 1000, block, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [129, 160, 255, 256])
def test_rows_of_one_tile_of_pairs(T, block):
    c = Case(T, 512, 1000, block, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [257, 300, 384, 400, 513, 1000])
def test_rows_of_several_tiles(T, block):
    c = Case(T, 256, 777, block, seed=2)
    c.check(c.run(BF16))
    c.check(c.run(F32))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [19, 200])
@pytest.mark.parametrize("V", [1, 2, 127, 128, 129, 256, 257, 1000, 20001, 40000])
def test_vocabularies(V, T, block):
    c = Case(T, 192, V, block, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [40, 140])
@pytest.mark.parametrize("H", [32, 64, 96, 128, 224, 256, 288, 1056, 4096, 8224])
def test_widths(H, T, block):
    c = Case(T, H, 300, block, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out_dtype", [F32, BF16, F16])
def test_output_types_and_no_row_scales(block, out_dtype):
    c = Case(50, 320, 555, block, seed=5, row_scales=False)
    c.check(c.run(out_dtype))


@pytest.mark.parametrize("block", [16, 32])
def test_each_element_with_its_scale(block):
    """One element of every row at a time: its products with a weight that is 1 there say where it and its scale lie."""
    T, H, V = 70, 256, 256
    x = torch.zeros(T, H)
    for t in range(T):
        x[t, (t * 37) % H] = (1.0 + t % 5) * 2.0 ** (t % 7 - 3)
    w = torch.eye(V, H)
    c = lambda r: (r[0], r[1], r[2])
    xq, wq = c(lp.quantize_fp4(x.cuda(), block)), c(lp.quantize_fp4(w.cuda(), block))
    ws = lp.new_head_workspace()
    got = lp.project_fp4(xq[0], xq[1], wq[0], wq[1], block, xq[2], wq[2], workspace=ws).cpu()
    xv = lp.dequantize_fp4(*xq, block, out_dtype=F32).cpu().double()
    wv = lp.dequantize_fp4(*wq, block, out_dtype=F32).cpu().double()
    assert torch.equal(got.double(), xv @ wv.t())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [30, 150])
def test_strides(T, block):
    c = Case(T, 96, 333, block, seed=6)
    x = torch.full((T, 80), 0x77, dtype=torch.uint8, device="cuda")
    x[:, :48] = c.x.cuda()
    w = torch.full((333, 64), 0x77, dtype=torch.uint8, device="cuda")
    w[:, :48] = c.w.cuda()
    out = torch.full((T, 350), 9.0, device="cuda")
    c.check(c.run(out=out[:, :333], x=x[:, :48], w=w[:, :48]))
    assert bool((out[:, 333:] == 9.0).all())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [40, 170])
def test_scales_behind_the_last_row_may_be_anything(T, block):
    # the tiles of scales end in rows that no one wrote: NaN there touches nothing
    c = Case(T, 96, 200, block, seed=7)
    xs, ws = c.tiles()
    for tiles, rows in ((xs, T), (ws, 200)):
        cb = tiles.numel() // (512 * (-(-rows // 128)))
        view = tiles.view(-1, cb, 32, 4, 4)
        i = torch.arange(128, device="cuda").view(4, 32).t()  # row of [row % 32][row / 32]
        for b in range(view.shape[0]):
            view[b][:, b * 128 + i >= rows] = 0x7F if block == 16 else 0xFF
    space = lp.new_head_workspace()
    cu = lambda t: None if t is None else t.cuda()
    c.space = space
    c.check(lp.project_fp4(c.x.cuda(), xs, c.w.cuda(), ws, block, cu(c.xr), cu(c.wr), workspace=space))


@pytest.mark.parametrize("block", [16, 32])
def test_rows_that_are_not_finite(block):
    x = torch.randn(20, 128, generator=torch.Generator().manual_seed(3))
    w = torch.randn(300, 128, generator=torch.Generator().manual_seed(4))
    x[4, 100], w[77, 5] = float("nan"), float("inf")
    xq, wq = lp.quantize_fp4(x.cuda(), block), lp.quantize_fp4(w.cuda(), block)
    y = lp.project_fp4(xq[0], xq[1], wq[0], wq[1], block, xq[2], wq[2], workspace=lp.new_head_workspace()).cpu()
    want = torch.zeros(20, 300, dtype=torch.bool)
    want[4], want[:, 77] = True, True
    assert torch.equal(torch.isnan(y), want)


def test_a_graph_and_two_streams():
    c = Case(60, 512, 3000, 16, seed=8)
    want = c.run().clone()
    xs, ws = c.tiles()
    x, w, xr, wr = (t.cuda() for t in (c.x, c.w, c.xr, c.wr))
    spaces = [lp.new_head_workspace() for _ in range(2)]
    outs = [torch.zeros(60, 3000, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, space, out in zip(streams, spaces, outs):
            lp.project_fp4(x, xs, w, ws, 16, xr, wr, out=out, workspace=space, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.project_fp4(x, xs, w, ws, 16, xr, wr, out=outs[0], workspace=spaces[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and lp.read_status(spaces[0]) == 0
