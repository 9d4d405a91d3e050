"""Infinities in adapters' weights and scales: what the formula gives, on every path that the
projection has for adapters."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import parity
from tests.test_gpu_head_project import BF16, E4M3, F16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


# Requests whose 32-row blocks have one adapter or two (the tensor cores' form for pairs of CTAs), or
# many (the epilogue's), on tiles of pairs, and few rows, on tiles of single CTAs.
FORMS = {"one a block": ([0, 64, 256], [0, 1]), "two a block": ([0, 48, 170, 256], [0, 1, -1]),
         "many": (None, [b % 5 for b in range(256)]), "few rows": (None, [b % 2 for b in range(20)])}


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("name", sorted(FORMS))
def test_an_infinite_b_gives_what_the_formula_gives(name, out_dtype, dtype):
    off, ids = FORMS[name]
    T = off[-1] if off else len(ids)
    c = Case(T, 512, 20001, dtype, A=5, rank=16, ids=ids, off=off, seed=31, unit=True,
             lora_dtype=BF16 if dtype == E4M3 else None)
    assert lp.project_cut(T, 512, 20001, dtype, 5, 16)[2] == (T > 128)
    # u[t, 0] one value of 16 bits (1, -2, 0 or 0.5), u[t, 1] another of few bits
    x, la, lb = c.x.clone(), c.la.clone(), c.lb.clone()
    x[:, :2] = torch.tensor([[1.0, 1.5], [-2.0, 1.0], [0.0, -3.0], [0.5, 0.0]]).repeat((T + 3) // 4, 1)[:T].to(dtype)
    la[:, :2] = 0
    la[:, 0, 0], la[:, 1, 1] = 1.0, 1.0
    lb[1, 5, 0], lb[1, 6, 0], lb[1, 19990, 1], lb[1, 19991, 2] = (float(v) for v in ("inf", "-inf", "inf", "inf"))
    out = c.run(out_dtype, x=x.cuda(), lora_a=la.cuda(), lora_b=lb.cuda()).double().cpu()
    xd = x.double() if c.sx is None else x.double() * c.sx.double()[:, None]
    of = list(range(T)) if off is None else [b for b in range(len(ids)) for _ in range(off[b], off[b + 1])]
    assert torch.isfinite(out[[t for t in range(T) if ids[of[t]] != 1]]).all()
    touched = [5, 6, 19990, 19991]
    for t in (t for t in range(T) if ids[of[t]] == 1):
        want = lb[1][touched].double() @ (la[1].double() @ xd[t])
        assert torch.equal(out[t, touched].nan_to_num(7.0, 1e300, -1e300), want.nan_to_num(7.0, 1e300, -1e300)), t
    others = [v for v in range(20001) if v not in touched]
    assert torch.isfinite(out[:, others]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("name", sorted(FORMS))
def test_an_infinite_u_gives_what_the_formula_gives(name, dtype):
    # one adapter's scale is infinite: its rows' u are infinities of either sign, the others' are finite
    off, ids = FORMS[name]
    T = off[-1] if off else len(ids)
    c = Case(T, 256, 20001, dtype, A=5, rank=1, ids=ids, off=off, seed=32, unit=True)
    la, lb = torch.zeros(5, 8, 256, dtype=dtype), torch.zeros(5, 20001, 8, dtype=dtype)
    la[:, :1], lb[:, :, :1] = c.la, c.lb
    la[:, 1:] = c.la          # eight equal columns: infinities of one sign
    lb[:, :, 1:] = c.lb
    c.rank = 8
    assert lp.project_cut(T, 256, 20001, dtype, 5, 8)[2] == (T > 128)
    scale = torch.ones(5)
    scale[1] = float("inf")
    out = c.run(F32, lora_a=la.cuda(), lora_b=lb.cuda(), adapter_scale=scale.cuda()).cpu()
    of = list(range(T)) if off is None else [b for b in range(len(ids)) for _ in range(off[b], off[b + 1])]
    mine = torch.tensor([ids[b] == 1 for b in of])
    assert torch.isfinite(out[~mine]).all()
    want = (c.x.double()[mine] @ c.la[1, 0].double())[:, None] * c.lb[1, :, 0].double()[None] * float("inf")
    got = out[mine].double()
    assert torch.equal(got.nan_to_num(7.0, 1e300, -1e300), want.nan_to_num(7.0, 1e300, -1e300))
