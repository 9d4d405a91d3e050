"""Host checks of the 4-bit operators without a GPU: every refusal (nothing is enqueued, no pointer is
dereferenced), the layout of the scales, and the 64-bit forms of the tests against values worked out by hand."""

import pytest
import torch

from tests import fp4_reference as ref
from tests.test_head_host import BF16, DTYPE, E4M3, F32, FAKE, NULL, SHAPE, WORKSPACE, lib  # noqa: F401 (a fixture)


def _quantize(lib, x=FAKE, dtype=BF16, T=4, H=64, xs=64, block=16, codes=FAKE, cs=32, scales=FAKE, row=FAKE):  # noqa: F811
    return lib.lp_head_quantize4(x, dtype, T, H, xs, block, codes, cs, scales, row, None)


def _dequantize(lib, codes=FAKE, cs=32, scales=FAKE, row=FAKE, V=4, H=64, block=16, rows=None, n=4, out=FAKE,  # noqa: F811
                odtype=F32, os_=64, ws=None, wsb=0):
    return lib.lp_head_dequantize4(codes, cs, scales, row, V, H, block, rows, n, out, odtype, os_, ws, wsb, None)


def _project(lib, x=FAKE, xs=32, xsc=FAKE, xr=FAKE, T=4, H=64, block=16, w=FAKE, wst=32, wsc=FAKE, wr=FAKE, V=100,  # noqa: F811
             out=FAKE, odtype=F32, os_=100, ws=FAKE, wsb=256):
    return lib.lp_head_project4(x, xs, xsc, xr, T, H, block, w, wst, wsc, wr, V, out, odtype, os_, ws, wsb, None)


def test_scale_bytes(lib):  # noqa: F811
    f = lib.lp_head_fp4_scale_bytes
    assert f(1, 64, 16) == 512 and f(128, 64, 16) == 512 and f(129, 64, 16) == 1024 and f(1, 96, 16) == 1024
    assert f(1, 128, 32) == 512 and f(1, 160, 32) == 1024 and f(300, 4096, 16) == 3 * 64 * 512
    assert f(1, 64, 8) == 0 and f(1, 64, 0) == 0 and f(0, 64, 16) == 0
    assert f(2 ** 31, 32768, 16) == 2 ** 31 * 2048


def test_quantize_refusals(lib):  # noqa: F811
    for name in ("x", "codes", "scales", "row"):
        assert _quantize(lib, **{name: None}) == NULL
    assert _quantize(lib, block=32) == DTYPE and _quantize(lib, block=64, row=None) == SHAPE
    assert _quantize(lib, dtype=E4M3) == DTYPE and _quantize(lib, dtype=99) == DTYPE
    assert _quantize(lib, T=0, x=None) == SHAPE and _quantize(lib, H=0) == SHAPE
    for H in (16, 48, 65, 32800):
        assert _quantize(lib, H=H, xs=40000, cs=32768) == SHAPE
    assert _quantize(lib, xs=63) == SHAPE and _quantize(lib, cs=16) == SHAPE and _quantize(lib, cs=40) == SHAPE
    assert _quantize(lib, x=FAKE + 1) == SHAPE and _quantize(lib, codes=FAKE + 8) == SHAPE
    assert _quantize(lib, scales=FAKE + 4) == SHAPE and _quantize(lib, row=FAKE + 2) == SHAPE


def test_dequantize_refusals(lib):  # noqa: F811
    for name in ("codes", "scales", "out"):
        assert _dequantize(lib, **{name: None}) == NULL
    assert _dequantize(lib, odtype=E4M3) == DTYPE
    assert _dequantize(lib, V=0, n=0) == SHAPE and _dequantize(lib, n=3) == SHAPE and _dequantize(lib, H=48) == SHAPE
    assert _dequantize(lib, block=8) == SHAPE and _dequantize(lib, cs=24) == SHAPE and _dequantize(lib, os_=63) == SHAPE
    assert _dequantize(lib, rows=FAKE, n=0, ws=FAKE, wsb=256) == SHAPE
    assert _dequantize(lib, out=FAKE + 2) == SHAPE and _dequantize(lib, codes=FAKE + 4) == SHAPE
    assert _dequantize(lib, row=FAKE + 1) == SHAPE and _dequantize(lib, rows=FAKE + 2, ws=FAKE, wsb=256) == SHAPE
    assert _dequantize(lib, rows=FAKE, n=2) == WORKSPACE and _dequantize(lib, rows=FAKE, n=2, ws=FAKE, wsb=255) == WORKSPACE
    assert _dequantize(lib, ws=FAKE + 64, wsb=256) == WORKSPACE


def test_project_refusals(lib):  # noqa: F811
    for name in ("x", "xsc", "w", "wsc", "out"):
        assert _project(lib, **{name: None}) == NULL
    assert _project(lib, odtype=E4M3) == DTYPE and _project(lib, odtype=99) == DTYPE
    for name in ("T", "V", "H"):
        assert _project(lib, **{name: 0}) == SHAPE
    assert _project(lib, H=48) == SHAPE and _project(lib, block=64) == SHAPE
    assert _project(lib, xs=16) == SHAPE and _project(lib, xs=40) == SHAPE and _project(lib, wst=40) == SHAPE
    assert _project(lib, os_=99) == SHAPE
    for name in ("x", "xsc", "w", "wsc"):
        assert _project(lib, **{name: FAKE + 8}) == SHAPE
    for name in ("xr", "wr", "out"):
        assert _project(lib, **{name: FAKE + 2}) == SHAPE
    assert _project(lib, V=2 ** 31 - 512, os_=2 ** 31, H=32768, xs=16384, wst=16384) == SHAPE  # copies' coordinates
    assert _project(lib, ws=None) == WORKSPACE and _project(lib, wsb=255) == WORKSPACE and _project(lib, ws=FAKE + 16) == WORKSPACE


def test_binding_refuses_host_tensors_and_other_blocks(lib):  # noqa: F811
    import ragged_log_probs_gb300 as lp
    x, b = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8)
    ws, s = torch.zeros(256, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: lp.quantize_fp4(x), lambda: lp.quantize_fp4(None), lambda: lp.dequantize_fp4(b, s),
                 lambda: lp.project_fp4(b, s, b, s, workspace=ws)):
        with pytest.raises(TypeError):
            call()
    for block in (8, 64, 0, -16):
        with pytest.raises(ValueError):
            lp.dequantize_fp4(b, s, block=block)
        with pytest.raises(ValueError):
            lp.fp4_scale_bytes(1, 64, block)
    with pytest.raises(ValueError):
        lp.tile_fp4_scales(torch.zeros(4, 4))


@pytest.mark.parametrize("rows,blocks", [(1, 1), (1, 4), (5, 7), (128, 8), (129, 9), (300, 3)])
def test_tiles_of_scales(lib, rows, blocks):  # noqa: F811
    import ragged_log_probs_gb300 as lp
    s = torch.randint(1, 127, (rows, blocks)).to(torch.uint8)
    tiles = lp.tile_fp4_scales(s)
    assert tiles.numel() == lp.fp4_scale_bytes(rows, blocks * 16, 16) == lp.fp4_scale_bytes(rows, blocks * 32, 32)
    got, left = ref.scale_values(tiles, rows, blocks * 32, 32)
    assert torch.equal(got, 2.0 ** (s.double() - 127)) and int(left.sum()) == 0
    assert int(tiles.long().sum()) == int(s.long().sum())


def test_the_reference_by_hand():
    # 0.75 lies between 0.5 and 1: the even code, 1; 2.5 between 2 and 3: 2; 5 between 4 and 6: 4
    assert ref.nearest(torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0, -0.3], dtype=torch.float64)).tolist() \
        == [0, 2, 2, 4, 4, 6, 6, 7, 1]
    assert [ref.e4m3(v) for v in (448.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9)] \
        == [448.0, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8]
    x = torch.zeros(2, 32)
    x[0, 0], x[0, 1], x[1, 20] = 2688.0, 448.0, -2689.0
    number, negative, scales, rows = ref.quantise(x, 16)
    assert rows.tolist() == [1.0, 2.0] and scales.tolist() == [[448.0, 0.0], [0.0, 224.0]]
    assert number[0, :2].tolist() == [7, 2] and number[1, 20] == 7 and bool(negative[1, 20])
    number, _, scales, rows = ref.quantise(torch.tensor([[7.9] + [1.0] * 31, [8.0] + [-3.0] * 31]), 32)
    assert scales.flatten().tolist() == [1.0, 2.0] and number[:, :2].tolist() == [[7, 2], [6, 3]] and rows is None
