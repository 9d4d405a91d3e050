"""Host checks of the draw without a GPU: every refusal, and the tests' 64-bit form against values worked out
by hand."""

import math

import pytest
import torch

from tests import sample_reference as ref
from tests.test_head_host import DTYPE, E4M3, F32, FAKE, NULL, SHAPE, WORKSPACE, lib  # noqa: F401 (a fixture)


def _sample(lib, x=FAKE, dtype=F32, T=4, V=100, xs=100, u=FAKE, off=None, B=4, tau=FAKE, k=FAKE, p=FAKE, q=FAKE, out=FAKE,  # noqa: F811
            lw=FAKE, ws=FAKE, wsb=4096):
    return lib.lp_head_sample(x, dtype, T, V, xs, u, off, B, tau, k, p, q, out, lw, ws, wsb, None)


def test_refusals(lib):  # noqa: F811
    for name in ("x", "u", "out"):
        assert _sample(lib, **{name: None}) == NULL
    assert _sample(lib, dtype=E4M3) == DTYPE and _sample(lib, dtype=99) == DTYPE
    assert _sample(lib, T=0, x=None, B=0) == SHAPE and _sample(lib, V=0) == SHAPE
    assert _sample(lib, B=3) == SHAPE and _sample(lib, off=FAKE, B=0) == SHAPE
    assert _sample(lib, xs=99) == SHAPE and _sample(lib, V=393217, xs=400000) == SHAPE
    assert _sample(lib, T=2 ** 29, B=2 ** 29) == SHAPE
    for name in ("x", "u", "off", "tau", "k", "p", "q", "out", "lw"):
        for by in (1, 2, 3):
            assert _sample(lib, **{name: FAKE + by}) == SHAPE
    assert _sample(lib, ws=None) == WORKSPACE and _sample(lib, wsb=335) == WORKSPACE and _sample(lib, ws=FAKE + 128) == WORKSPACE


def test_workspace_size(lib):  # noqa: F811
    f = lib.lp_head_sample_workspace_size
    # 16 bytes for a part of 1024 tokens (up to 7 of them before a row's first), 4 for a row's place in the order
    assert f(0, 0) == 256 and f(4, 100) == 256 + 4 * 20 and f(1, 1017) == 256 + 16 + 4 and f(1, 1018) == 256 + 32 + 4
    assert f(2 ** 31, 393216) == 256 + 2 ** 31 * (385 * 16 + 4)


def test_new_error_codes(lib):  # noqa: F811
    import ragged_log_probs_gb300 as lp
    texts = {lib.lp_ragged_strerror(c).decode() for c in range(15)}
    assert len(texts) == 15 and "unknown lp_status" not in texts
    assert lp.STATUS_NAMES[13] == "LP_ERR_SAMPLING" and lp.STATUS_NAMES[14] == "LP_ERR_LOGITS"


def test_binding_refuses_host_tensors(lib):  # noqa: F811
    import ragged_log_probs_gb300 as lp
    with pytest.raises(TypeError):
        lp.sample(torch.zeros(2, 8), torch.zeros(2), workspace=torch.zeros(256, dtype=torch.uint8))


def test_the_reference_by_hand():
    x = torch.tensor([1.0, 0.5, 0.25, 0.25]).log()  # weights 4, 2, 1, 1 of 8
    cuts = {0.0: 0, 0.49: 0, 0.51: 1, 0.74: 1, 0.76: 2, 0.87: 2, 0.88: 3}  # (logarithms in f32: not at the borders)
    assert {u: ref.draw(x, u)[0] for u in cuts} == cuts
    assert abs(ref.draw(x, 0.6)[1] - math.log(0.25)) < 1e-7
    assert ref.draw(x, 0.9, k=2)[0] == 1 and abs(ref.draw(x, 0.9, k=2)[1] - math.log(1 / 3)) < 1e-7
    assert ref.draw(x, 0.99, k=3)[0] == 2                 # of the two alike the lower id
    assert ref.draw(x, 0.99, p=0.45)[0] == 0 and ref.draw(x, 0.99, p=0.55)[0] == 1 and ref.draw(x, 0.99, p=0.8)[0] == 2
    assert ref.draw(x, 0.99, p=0.0)[0] == 0 and ref.draw(x, 0.99, k=2, p=0.7)[0] == 1 and ref.draw(x, 0.99, k=2, p=0.6)[0] == 0
    assert ref.draw(x, 0.99, q=0.3)[0] == 1 and ref.draw(x, 0.99, q=1.0)[0] == 0
    assert ref.draw(x, 0.99, tau=0.0)[0] == 0 and abs(ref.draw(x, 0.0, tau=0.5)[1] - math.log(16 / 22)) < 1e-7
    assert ref.draw(torch.full((3,), -math.inf), 0.5)[0] is None and ref.draw(torch.tensor([0.0, math.nan]), 0.5)[0] is None
