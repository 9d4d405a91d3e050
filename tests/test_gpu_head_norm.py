"""Final norm (lp_head_norm) against the 64-bit formula: types, widths, strides, picked
rows, residuals, in place, 8-bit outputs, rows of zeros and of non-finite values."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import head_reference as ref
from tests import parity

pytestmark = pytest.mark.gpu

EPS = 1e-5
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# f32 arithmetic: the sum (1), a sum of squares of at most 32 terms a thread and 10 tree
# steps (halved by the root), rsqrtf (4), three products and a division: below 32 roundings
F32 = 32 * 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


def check(got, want, dtype):
    got, want = got.double().cpu(), want
    smallest = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -126}[dtype]
    bound = want.abs() * (half_step(dtype) + F32) * (1 + F32) + smallest
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    fine = torch.isfinite(want)
    assert ((got - want).abs() <= bound)[fine].all(), float(((got - want).abs() - bound)[fine].max())


def check_e4m3(q, scale, y):
    want = ref.e4m3_scale(y)
    assert ((scale.double().cpu() - want).abs() <= want * F32).all()
    v = y / scale.double().cpu()[:, None]
    q = q.float().double().cpu()
    # half a step of the value: 2^-4 of it, or of the subnormal step 2^-9
    assert ((q - v).abs() <= v.abs() * (2.0 ** -4 + 2 * F32) + 2.0 ** -10).all()


def inputs(T, H, dtype, residual=True, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + H)
    x = (torch.randn(T, H, generator=g) * 3).to(dtype)
    r = (torch.randn(T, H, generator=g) * 5).to(dtype) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)
    return x, r, w


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 7, 8, 64, 255, 256, 1000, 1024, 1032, 4096, 4100, 5001, 8192, 8200, 16384, 32768])
def test_widths_and_types(dtype, H):
    x, r, w = inputs(5, H, dtype)
    xc, rc, wc = cuda(x, r, w)
    h, y = ref.norm(x, w, EPS, r)
    kept = torch.empty_like(xc)
    out = lp.rms_norm(xc, wc, EPS, residual=rc, residual_out=kept)
    assert out.dtype == dtype
    check(out, y, dtype)
    check(kept, h, dtype)
    check(lp.rms_norm(xc, wc, EPS, residual=rc, out_dtype=torch.float32), y, torch.float32)
    q, scale = lp.rms_norm(xc, wc, EPS, residual=rc, out_dtype=torch.float8_e4m3fn)
    check_e4m3(q, scale, y)


@pytest.mark.parametrize("T", [1, 2, 3, 151, 700])
@pytest.mark.parametrize("H", [48, 1024, 2056])
def test_row_counts_without_residual(T, H):
    x, _, w = inputs(T, H, torch.bfloat16, residual=False, seed=T)
    xc, wc = cuda(x, w)
    _, y = ref.norm(x, w, EPS)
    check(lp.rms_norm(xc, wc, EPS), y, torch.bfloat16)
    check_e4m3(*lp.rms_norm(xc, wc, EPS, out_dtype=torch.float8_e4m3fn), y)


def test_f32_weight_for_16_bit_rows():
    x, r, w = inputs(9, 2048, torch.bfloat16)
    w = w.float() * 1.0001
    xc, rc, wc = cuda(x, r, w)
    check(lp.rms_norm(xc, wc, EPS, residual=rc), ref.norm(x, w, EPS, r)[1], torch.bfloat16)


@pytest.mark.parametrize("H", [100, 1536, 4104])
def test_picked_rows(H):
    x, r, w = inputs(50, H, torch.float16)
    rows = [49, 0, 7, 7, 31]
    xc, rc, wc = cuda(x, r, w)
    ws = lp.new_head_workspace()
    rt = torch.tensor(rows, dtype=torch.int32, device="cuda")
    h, y = ref.norm(x, w, EPS, r, rows)
    kept = torch.empty(5, H, dtype=torch.float16, device="cuda")
    check(lp.rms_norm(xc, wc, EPS, residual=rc, rows=rt, residual_out=kept, workspace=ws), y, torch.float16)
    check(kept, h, torch.float16)
    assert lp.read_status(ws) == 0


def test_row_index_past_the_rows_sets_a_bit_and_gives_nan():
    x, r, w = inputs(6, 640, torch.bfloat16)
    xc, rc, wc = cuda(x, r, w)
    ws = lp.new_head_workspace()
    rows = torch.tensor([5, 6, 2, -1], dtype=torch.int32, device="cuda")
    out = lp.rms_norm(xc, wc, EPS, residual=rc, rows=rows, workspace=ws)
    assert lp.read_status(ws) == 1 << 4
    assert torch.isnan(out[[1, 3]]).all()
    check(out[[0, 2]], ref.norm(x, w, EPS, r, [5, 2])[1], torch.bfloat16)
    q, scale = lp.rms_norm(xc, wc, EPS, rows=rows, workspace=ws, out_dtype=torch.float8_e4m3fn)
    assert torch.isnan(scale[[1, 3]]).all() and torch.isnan(q.float()[[1, 3]]).all()
    lp.clear_status(ws)
    assert lp.read_status(ws) == 0


@pytest.mark.parametrize("extra,shift", [(8, 0), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_unaligned_bases(extra, shift, dtype):
    T, H = 7, 1608
    x, r, w = inputs(T, H, dtype)
    buf = torch.full((3, T, H + extra + shift), 9.0, dtype=dtype, device="cuda")
    xv, rv, ov = (buf[i][:, shift:shift + H] for i in range(3))
    xv.copy_(x)
    rv.copy_(r)
    lp.rms_norm(xv, w.cuda(), EPS, residual=rv, out=ov)
    check(ov, ref.norm(x, w, EPS, r)[1], dtype)
    assert (buf[2][:, :shift] == 9).all() and (buf[2][:, shift + H:] == 9).all()


def test_in_place():
    x, r, w = inputs(33, 4096, torch.bfloat16)
    xc, rc, wc = cuda(x, r, w)
    h, y = ref.norm(x, w, EPS, r)
    lp.rms_norm(xc, wc, EPS, residual=rc, out=xc, residual_out=rc)
    check(xc, y, torch.bfloat16)
    check(rc, h, torch.bfloat16)


def test_zero_and_tiny_rows():
    x = torch.zeros(3, 512)
    x[1] = 1e-30
    x[2, 5] = 1e-20
    w = torch.ones(512)
    xc, wc = cuda(x, w)
    out = lp.rms_norm(xc, wc, 0.0, out_dtype=torch.float32)
    assert torch.isnan(out[0]).all()          # 0 / 0 without eps
    out = lp.rms_norm(xc, wc, EPS)
    check(out, ref.norm(x, w, EPS)[1], torch.float32)
    q, scale = lp.rms_norm(xc, wc, EPS, out_dtype=torch.float8_e4m3fn)
    assert float(scale[0]) == 2.0 ** -126 and (q.float()[0] == 0).all()
    check_e4m3(q, scale, ref.norm(x, w, EPS)[1])


@pytest.mark.parametrize("H", [256, 4096])
def test_nan_and_infinity_stay_in_their_rows(H):
    x, r, w = inputs(4, H, torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    xc, rc, wc = cuda(x, r, w)
    out = lp.rms_norm(xc, wc, EPS, residual=rc)
    y = ref.norm(x, w, EPS, r)[1]
    check(out[[0, 3]], y[[0, 3]], torch.bfloat16)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, 5]) and (out[2, :5] == 0).all()
    q, scale = lp.rms_norm(xc, wc, EPS, residual=rc, out_dtype=torch.float8_e4m3fn)
    assert torch.isnan(scale[[1, 2]]).all() and torch.isnan(q.float()[[1, 2]]).all()
    check_e4m3(q[[0, 3]], scale[[0, 3]], y[[0, 3]])


def test_on_another_stream_and_in_a_graph():
    x, r, w = inputs(40, 2048, torch.bfloat16)
    xc, rc, wc = cuda(x, r, w)
    y = ref.norm(x, w, EPS, r)[1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = lp.rms_norm(xc, wc, EPS, residual=rc, stream=s)
    s.synchronize()
    check(out, y, torch.bfloat16)
    out = torch.empty_like(xc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.rms_norm(xc, wc, EPS, residual=rc, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(out, y, torch.bfloat16)


def test_refusals_of_the_binding():
    x, r, w = inputs(4, 64, torch.bfloat16)
    xc, rc, wc = cuda(x, r, w)
    for bad in (dict(residual=rc[:3]), dict(residual=rc.float()), dict(out=torch.empty(4, 65, device="cuda")),
                dict(out=torch.empty(64, 4, device="cuda", dtype=torch.bfloat16).t()), dict(residual=r),
                dict(out=xc, out_dtype=torch.float32), dict(out_scale=torch.empty(3, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            lp.rms_norm(xc, wc, EPS, **bad)
    with pytest.raises(ValueError):
        lp.rms_norm(xc[0], wc, EPS)
    with pytest.raises((ValueError, TypeError)):
        lp.rms_norm(xc, wc[:63], EPS)
    with pytest.raises(lp.LpError):                  # picked rows need a workspace
        lp.rms_norm(xc, wc, EPS, rows=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(lp.LpError):
        lp.rms_norm(xc.int(), wc.int().float(), EPS)


@pytest.mark.parametrize("H", [1025, 1026, 1031, 2049, 4095, 32761, 32767, 32768])
@pytest.mark.parametrize("dtype", DTYPES)
def test_unaligned_rows(H, dtype):
    # rows that begin at every boundary, and each tensor at another one
    T = 9
    x, r, w = inputs(T, H, dtype, seed=3)
    buf = torch.full((4, T, H + 16), 9.0, dtype=dtype, device="cuda")
    xv, rv, ov, kv = (buf[i].flatten()[i:i + T * (H + 5)].view(T, H + 5)[:, :H] for i in range(4))
    xv.copy_(x)
    rv.copy_(r)
    lp.rms_norm(xv, w.cuda(), EPS, residual=rv, out=ov, residual_out=kv)
    h, y = ref.norm(x, w, EPS, r)[:2]
    check(ov, y, dtype)
    check(kv, h, dtype)
    for t in range(T - 1):  # the elements between the rows
        assert (buf[2].flatten()[2 + t * (H + 5) + H:2 + (t + 1) * (H + 5)] == 9).all()
        assert (buf[3].flatten()[3 + t * (H + 5) + H:3 + (t + 1) * (H + 5)] == 9).all()
    q = torch.zeros(T * (H + 3) + 1, dtype=torch.uint8, device="cuda")
    qv = q[1:].view(T, H + 3)[:, :H].view(torch.float8_e4m3fn)
    qv, scale = lp.rms_norm(xv, w.cuda(), EPS, residual=rv, out=qv, out_scale=torch.empty(T, device="cuda"))
    check_e4m3(qv, scale, y)
    assert (q[1:].view(T, H + 3)[:, H:] == 0).all() and q[0] == 0


def test_unaligned_rows_in_place():
    x, r, w = inputs(40, 5003, torch.bfloat16, seed=4)
    xc, rc, wc = cuda(x, r, w)
    lp.rms_norm(xc, wc, EPS, residual=rc, out=xc, residual_out=rc)
    h, y = ref.norm(x, w, EPS, r)[:2]
    check(xc, y, torch.bfloat16)
    check(rc, h, torch.bfloat16)


@pytest.mark.parametrize("H", [64, 1608, 1609])
def test_rows_far_apart(H):
    # the third row begins past 2^32 elements
    T, step = 3, 2 ** 31 + 24
    x, r, w = inputs(T, H, torch.bfloat16, seed=5)
    far = torch.empty(2 * step + H, dtype=torch.bfloat16, device="cuda")
    xv = far.as_strided((T, H), (step, 1))
    xv.copy_(x)
    lp.rms_norm(xv, w.cuda(), EPS, residual=r.cuda(), out=xv)
    check(xv, ref.norm(x, w, EPS, r)[1], torch.bfloat16)
    del far, xv
    torch.cuda.empty_cache()
