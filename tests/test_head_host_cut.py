"""How the projection's sizes are cut into tiles, without a GPU: what the kernel and the workspace
need of every cut, and which sizes reach the adapters' form on the tensor cores."""

import random

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests.test_head_host import lib  # noqa: F401 (a fixture)

TYPES = [torch.bfloat16, torch.float16, torch.float8_e4m3fn]


def test_every_cut_fits_the_kernel_and_the_workspace(lib):  # noqa: F811
    rng = random.Random(7)
    for _ in range(20000):
        T, V, H = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 19)), 16 * int(2 ** rng.uniform(0, 10))
        adapters = rng.choice([0, 3])
        rank = rng.randint(1, 64) if adapters else 0
        ctas, rows, tensor = lp.project_cut(T, H, V, rng.choice(TYPES), adapters, rank, rng.choice([132, 148, 152, 160]))
        assert ctas in (1, 2) and rows % (16 * ctas) == 0 and 16 <= rows <= 256
        assert not tensor or (ctas == 2 and rank and rank % 8 == 0)
        tiles = -(-T // rows)
        assert (tiles - 1) * rows < T
        if adapters:  # a page of lists for every 32 rows; u's parts in whole 256
            assert tiles <= -(-T // 32) and (tensor == 0 or tiles * rows <= -(-T // 256) * 256)


@pytest.mark.parametrize("sms", [148, 152, 160])
def test_which_sizes_reach_the_tensor_cores(lib, sms):  # noqa: F811
    for dtype in TYPES:
        assert lp.project_cut(256, 2048, 20001, dtype, 3, 16, sms) == (2, 256, True)
        assert lp.project_cut(600, 2048, 20001, dtype, 3, 64, sms)[::2] == (2, True)
        assert lp.project_cut(256, 2048, 20001, dtype, 3, 20, sms)[2] is False
        assert lp.project_cut(20, 2048, 20001, dtype, 3, 16, sms)[0] == 1
        assert lp.project_cut(256, 2048, 20001, dtype, 0, 0, sms)[2] is False


def test_refusals(lib):  # noqa: F811
    for bad in ((0, 64, 64, torch.bfloat16), (4, 64, 64, torch.float32), (4, 64, 64, torch.bfloat16, 1, 65)):
        with pytest.raises(lp.LpError):
            lp.project_cut(*bad, sms=152) if len(bad) == 4 else lp.project_cut(*bad, 152)
