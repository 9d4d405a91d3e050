"""Rows in 4 bits (lp_head_quantize4, lp_head_dequantize4) against the 64-bit formulas: both blocks, all
types, widths and row counts round the tiles of scales, strides, ties, extreme and non-finite rows."""

import math

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


def check(x, block, got=None):
    """Codes, scales and row scales of x are those of the formula, exactly."""
    codes, scales, rows = lp.quantize_fp4(x.cuda() if not x.is_cuda else x, block) if got is None else got
    T, H = x.shape
    number, negative, want, want_rows = ref.quantise(x.cpu(), block)
    have, left = ref.scale_values(scales.cpu(), T, H, block)
    assert torch.equal(torch.nan_to_num(have, nan=-1.0), torch.nan_to_num(want, nan=-1.0))
    assert int(left.sum()) == 0
    if block == 16:
        assert torch.equal(torch.nan_to_num(rows.double().cpu(), nan=-1.0), torch.nan_to_num(want_rows, nan=-1.0))
    else:
        assert rows is None
    n, s = ref.unpack(codes.cpu())
    fine = torch.isfinite(want).repeat_interleave(block, 1)
    assert torch.equal(n[fine], number[fine])
    assert torch.equal((s & (n > 0))[fine], (negative & (number > 0))[fine])
    return codes, scales, rows


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 4096), (3, 96), (5, 160), (33, 64), (127, 32), (128, 1024), (129, 1056),
                                 (130, 128), (300, 224), (2, 8192), (2, 8224), (1, 32768)])
def test_sizes(T, H, dtype, block):
    g = torch.Generator().manual_seed(T * 1000 + H)
    x = (torch.randn(T, H, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(dtype)
    check(x, block)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_ties_go_to_the_even_code(dtype, block):
    # every half of a step, with the block's scale set by a largest element of 6 (or 4 for blocks of 32)
    halves = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 6.0])
    x = torch.stack([torch.cat([halves, -halves]) * 2.0 ** e for e in range(-9, 9)])
    check(x.to(dtype), block)


@pytest.mark.parametrize("block", [16, 32])
def test_scales_next_to_their_borders(block):
    # maxima round powers of two, round 2688 times them, and round the middles of e4m3's steps
    tops = []
    for e in (-20, -3, 0, 5):
        for m in (1.0, 1.3125, 1.5, 1.75, 1.9921875, 4.0 / 3, 1.0625 * 1.5, 1.1875 * 0.75 * 2):
            v = torch.tensor(m * 2.0 ** e, dtype=F32)
            tops += [v, torch.nextafter(v, torch.tensor(0.0)), torch.nextafter(v, torch.tensor(1e9))]
    x = torch.zeros(len(tops), 64)
    x[:, 5] = torch.stack(tops)
    x[:, 40] = x[:, 5] / 37
    check(x, block)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_rows(dtype, block):
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.zeros(9, 64)
    x[1, 3], x[2, 3], x[3, 3] = big, small, small / 64
    x[4] = small / 128
    x[5, :32], x[5, 32:] = big, small
    x[6, 0], x[6, 63] = 2.0 ** -95, -(2.0 ** -100)
    x[7] = -0.0
    x[8] = torch.linspace(-1e-30, 1e30, 64)
    check(x.to(dtype), block)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite(dtype, block, bad):
    x = torch.randn(4, 1056, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[1, 500] = bad
    x[3, 0] = bad
    codes, scales, rows = check(x, block)
    v = lp.dequantize_fp4(codes, scales, rows, block, out_dtype=F32).cpu()
    hit = torch.isnan(v)
    want = torch.zeros_like(hit)
    if block == 16:
        want[1] = want[3] = True
    else:
        want[1, 480:512] = want[3, :32] = True
    assert torch.equal(hit, want)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift,extra", [(0, 8), (1, 0), (3, 5), (0, 1)])
def test_strides_and_places(dtype, block, shift, extra):
    T, H = 7, 96
    g = torch.Generator().manual_seed(2)
    flat = torch.randn(T * (H + extra) + shift + 8, generator=g).to(dtype).cuda()
    x = flat[shift:shift + T * (H + extra)].view(T, H + extra)[:, :H]
    codes = torch.full((T, 80), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((lp.fp4_scale_bytes(T, H, block) + 32,), 0x55, dtype=torch.uint8, device="cuda")
    inner = scales[16:-16]
    rows = torch.zeros(T, device="cuda") if block == 16 else None
    got = lp.quantize_fp4(x, block, out=codes[:, :H // 2], out_scales=inner, out_row_scale=rows)
    assert got[0].data_ptr() == codes.data_ptr() and got[1].data_ptr() == inner.data_ptr()
    check(x, block, got)
    assert bool((codes[:, H // 2:] == 0xAA).all())             # nothing behind the rows
    assert bool((scales[:16] == 0x55).all()) and bool((scales[-16:] == 0x55).all())
    out = torch.full((T * (H + extra) + shift + 8,), 77.0, dtype=dtype, device="cuda")
    view = out[shift:shift + T * (H + extra)].view(T, H + extra)[:, :H]
    lp.dequantize_fp4(got[0], got[1], got[2], block, out=view)
    n, s = ref.unpack(got[0].cpu())
    want = ref.values(n, s, ref.scale_values(inner.cpu(), T, H, block)[0], None if rows is None else rows.cpu(), block)
    assert torch.equal(view.double().cpu(), want.to(dtype).double())
    view.fill_(77.0)
    assert bool((out == 77.0).all())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,H", [(1, 32), (130, 96), (300, 4128)])
def test_values_of_any_rows(V, H, out_dtype, block):
    codes, scale, rs = ref.random_rows(V, H, block, seed=V + H)
    tiles = lp.tile_fp4_scales(ref.scale_bytes(scale, block)).cuda()
    n, s = ref.unpack(codes)
    want = ref.values(n, s, scale, rs, block)
    c = lambda t: None if t is None else t.cuda()
    got = lp.dequantize_fp4(c(codes), tiles, c(rs), block, out_dtype=out_dtype)
    # rounded at the product with the row scale (f32) and at the end
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[out_dtype]
    room = want.abs() * (half + 2.0 ** -24) + (2.0 ** -25 if out_dtype == F16 else 0.0)
    assert bool(((got.double().cpu() - want).abs() <= room).all())
    pick = torch.tensor([V - 1, 0, V // 2, 0], dtype=torch.int32)
    ws = lp.new_head_workspace()
    some = lp.dequantize_fp4(c(codes), tiles, c(rs), block, rows=pick.cuda(), out_dtype=out_dtype, workspace=ws)
    assert torch.equal(some, got[pick.long().cuda()]) and lp.read_status(ws) == 0


def test_smallest_and_missing_scales():
    # e8m0: 2^-127 and NaN; e4m3: 0, its smallest, NaN
    codes = torch.full((1, 48), 0x77, dtype=torch.uint8, device="cuda")
    tiles = lp.tile_fp4_scales(torch.tensor([[0, 255, 254]], dtype=torch.uint8)).cuda()
    v = lp.dequantize_fp4(codes, tiles, block=32, out_dtype=F32).cpu()[0]
    assert bool((v[:32] == 6 * 2.0 ** -127).all()) and bool(torch.isnan(v[32:64]).all()) and bool(torch.isinf(v[64:]).all())
    tiles = lp.tile_fp4_scales(torch.tensor([[0, 1, 0x7F, 0x7E, 0x38, 0x08]], dtype=torch.uint8)).cuda()
    v = lp.dequantize_fp4(codes, tiles, block=16, out_dtype=F32).cpu()[0].view(6, 16)
    assert v[:, 0].tolist()[:2] == [0.0, 6 * 2.0 ** -9] and math.isnan(v[2, 0])
    assert v[3:, 0].tolist() == [6 * 448.0, 6.0, 6 * 2.0 ** -6]


def test_rows_past_the_last_are_nan_and_reported():
    codes, scale, rs = ref.random_rows(40, 64, 16, seed=9)
    tiles = lp.tile_fp4_scales(ref.scale_bytes(scale, 16)).cuda()
    ws = lp.new_head_workspace()
    rows = torch.tensor([3, 40, -1, 39], dtype=torch.int32, device="cuda")
    v = lp.dequantize_fp4(codes.cuda(), tiles, rs.cuda(), 16, rows=rows, out_dtype=F32, workspace=ws).cpu()
    assert torch.isnan(v).all(1).tolist() == [False, True, True, False] and not bool(torch.isnan(v[[0, 3]]).any())
    assert lp.read_status(ws) == 1 << 4  # LP_ERR_OFFSETS
    lp.clear_status(ws)
    assert lp.read_status(ws) == 0


def test_a_lookup_past_32_bits():
    # codes of more than 2^32 bytes: rows at the very end
    V, H = 270000, 32768
    codes = torch.zeros(V, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((lp.fp4_scale_bytes(V, H, 32),), 127, dtype=torch.uint8, device="cuda")
    codes[V - 1, :] = 0x72
    codes[V - 2, -1] = 0x51
    ws = lp.new_head_workspace()
    rows = torch.tensor([V - 2, V - 1], dtype=torch.int32, device="cuda")
    v = lp.dequantize_fp4(codes, scales, block=32, rows=rows, out_dtype=F32, workspace=ws).cpu()
    assert v[0, -2:].tolist() == [0.5, 3.0] and float(v[0].sum()) == 3.5
    assert v[1].view(-1, 2)[:, 0].unique().tolist() == [1.0] and v[1].view(-1, 2)[:, 1].unique().tolist() == [6.0]


def test_another_stream_and_a_graph():
    x = torch.randn(50, 512, device="cuda").bfloat16()
    want = [t.clone() for t in lp.quantize_fp4(x)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lp.quantize_fp4(x, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.zeros(50, 512, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.quantize_fp4(x, 16, *got)
        lp.dequantize_fp4(*got, out=out)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(out, lp.dequantize_fp4(*want))
