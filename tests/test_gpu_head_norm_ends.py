"""The final norm at the ends of float32: rows whose squares, or whose products with the weight,
leave it, while the normed row does not."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import head_reference as ref
from tests import parity
from tests.test_gpu_head_norm import check, check_e4m3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [40, 1000, 4096, 5001])
def test_norm_of_rows_whose_squares_leave_float32(H, dtype):
    # sizes of the rows: h^2 or its sum overflows, or h^2 is below the least number
    sizes = [1e18, 1e20, 3e30, 1e37, 1.0, 1e-18, 1e-23, 1e-30]
    g = torch.Generator().manual_seed(H)
    x = (torch.rand(len(sizes), H, generator=g) + 0.5) * torch.tensor(sizes)[:, None]
    x = (x * torch.where(torch.rand(len(sizes), H, generator=g) < 0.5, -1.0, 1.0)).to(dtype)
    r = (x.float() * 0.25).to(dtype)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)
    for eps in (0.0, 1e-30, 1e-5):
        h, y = ref.norm(x, w, eps, r)
        kept = torch.empty_like(x.cuda())
        args = dict(eps=eps, residual=r.cuda())
        check(lp.rms_norm(x.cuda(), w.cuda(), residual_out=kept, **args), y, dtype)
        check(kept, h, dtype)
        check(lp.rms_norm(x.cuda(), w.cuda(), out_dtype=torch.float32, **args), y, torch.float32)
        q, scale = lp.rms_norm(x.cuda(), w.cuda(), out_dtype=torch.float8_e4m3fn, **args)
        check_e4m3(q, scale, y)


def test_norm_of_large_rows_with_weights_at_the_ends():
    # |h w| leaves float32 at either end, y does not
    H = 2048
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, H, generator=g) * torch.tensor([1e25, 1e15, 1e-15, 1e-20])[:, None]
    for size in (1e25, 1e-25):
        w = (1 + torch.rand(H, generator=g)) * size
        _, y = ref.norm(x, w, 0.0)
        check(lp.rms_norm(x.cuda(), w.cuda(), 0.0), y, torch.float32)
        check_e4m3(*lp.rms_norm(x.cuda(), w.cuda(), 0.0, out_dtype=torch.float8_e4m3fn), y)


def test_norm_of_large_rows_in_place():
    x = torch.full((3, 1536), 2e25)
    x[1] = 3.0
    xc, rc = x.cuda(), (-0.5 * x).cuda()
    w = torch.ones(1536)
    h, y = ref.norm(x, w, 1e-5, -0.5 * x)
    lp.rms_norm(xc, w.cuda(), 1e-5, residual=rc, out=xc, residual_out=rc)
    check(xc, y, torch.float32)
    check(rc, h, torch.float32)
