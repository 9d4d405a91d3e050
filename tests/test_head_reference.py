"""The 64-bit forms that the head operators' tests compare with, against values worked out by hand."""

import math

import torch

from tests import head_reference as ref


def test_norm():
    x, r, w = torch.tensor([[3.0, 0.0, 1.0], [0.0, 0.0, 0.0]]), torch.tensor([[0.0, 4.0, -1.0], [0.0, 0.0, 0.0]]), torch.tensor([1.0, 2.0, 5.0])
    h, y = ref.norm(x, w, 0.0, r, rows=[0])
    assert h.tolist() == [[3.0, 4.0, 0.0]]
    rms = math.sqrt(25 / 3)
    assert torch.allclose(y, torch.tensor([[3 / rms, 8 / rms, 0.0]], dtype=torch.float64), rtol=1e-15)
    h, y = ref.norm(x, w, 0.25)
    assert y[1].tolist() == [0.0, 0.0, 0.0]
    assert torch.allclose(y[0], torch.tensor([3.0, 0.0, 5.0], dtype=torch.float64) / math.sqrt(10 / 3 + 0.25), rtol=1e-15)
    assert ref.e4m3_scale(torch.tensor([[-896.0, 4.0], [0.0, 0.0]], dtype=torch.float64)).tolist() == [2.0, 2.0 ** -126]


def test_process():
    x = torch.tensor([[2.0, -2.0, 1.0, 0.0, 5.0]] * 3)
    out, _ = ref.process(x, row_offsets=[0, 2, 3], history=[[0, 0, 1, 2, 2, 9], []], prompt_lens=[2, 0], rep=[2.0, 3.0],
                         freq=[0.5, 1.0], pres=[0.25, 1.0], bias=[{3: 1.5, 4: -1.0}, {}],
                         mask=torch.tensor([[True, True, False, True, True]]), mask_index=[-1, 0, 0])
    # token 0: of the prompt only; 1: once in the output; 2: twice; 9 is past the vocabulary
    assert out[0].tolist() == [1.0, -4.75, 0.5 - 1.0 - 0.25, 1.5, 4.0]
    assert out[1].tolist() == [1.0, -4.75, -math.inf, 1.5, 4.0]
    assert out[2].tolist() == [2.0, -2.0, -math.inf, 0.0, 5.0]


def test_rows_and_masks():
    assert ref.requests_of_rows(4, [0, 1, 1, 4]) == [0, 2, 2, 2] and ref.requests_of_rows(2, None) == [0, 1]
    allowed = torch.zeros(1, 34, dtype=torch.bool)
    allowed[0, [0, 5, 31, 33]] = True
    assert ref.pack_mask(allowed).tolist() == [[1 + 32 - 2 ** 31, 2]]
