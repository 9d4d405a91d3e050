"""Processing of logits with offsets that are wrong: what a row gets does not depend on whether
histories were sorted by slices first, nothing of an earlier call comes back, and the status word
tells."""

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import head_reference as ref
from tests import parity
from tests.test_gpu_head_process import bits, check, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    parity.ensure_built()


# offsets of the requests' histories, and the requests whose own two offsets are wrong
LISTS = {
    "two claim one chunk": ([0, 9000, 4000, 13000], [1]),
    "one over another": ([0, 30000, 10000, 30000], [1]),
    "past the total between": ([0, 10 ** 9, 5000, 13000], [0, 1]),
    "one wrong of many": ([4200 * b if b != 20 else 4200 * 38 for b in range(41)], [20]),
}


@pytest.mark.parametrize("neutral", [False, True])
@pytest.mark.parametrize("name", sorted(LISTS))
def test_decreasing_history_offsets_where_histories_are_sorted(name, neutral):
    off, wrong = LISTS[name]
    B, V = len(off) - 1, 20000
    total = max(o for o in off if o < 10 ** 9)
    assert total // B >= 4096
    g = torch.Generator().manual_seed(41)
    tokens = (V * torch.rand(total, generator=g) ** 3).long().clamp_max(V - 1)
    x = torch.randn(B, V, generator=g) * 3
    rep, freq, pres = [1.25] * B, [0.5] * B, [-0.25] * B
    if neutral:  # a request whose history has no effect does not have it read
        for b in wrong:
            rep[b], freq[b], pres[b] = 1.0, 0.0, 0.0
    args = dict(history=tokens.to(torch.int32).cuda(), repetition=torch.tensor(rep).cuda(),
                frequency=torch.tensor(freq).cuda(), presence=torch.tensor(pres).cuda())
    prompt = [1000 + b for b in range(B)]
    ws = lp.new_head_workspace(requests=B, history=total)
    # an earlier call with good lists in the same workspace
    step = total // B
    lp.process_logits(x.cuda(), history_offsets=i32([step * b for b in range(B + 1)]), workspace=ws, **args)
    assert lp.read_status(ws) == 0
    out = lp.process_logits(x.cuda(), history_offsets=i32(off), prompt_lens=i32(prompt), workspace=ws, **args)
    right = [b for b in range(B) if b not in wrong]
    history = [tokens[off[b]:off[b + 1]].tolist() if b in right else [] for b in range(B)]
    want = ref.process(x, history=history, prompt_lens=prompt, rep=rep, freq=freq, pres=pres)
    if neutral:
        right = list(range(B))
    else:
        assert torch.isnan(out[wrong]).all() and lp.read_status(ws) == bits(4)
    check(out[right], (want[0][right], want[1][right]))


def test_a_refused_call_leaves_nothing_enqueued():
    # more rows times slices than a grid holds: refused on the host before the histories' sort
    B, total = 1, 9000
    ws = lp.new_head_workspace(requests=B, history=total)
    history, off = torch.zeros(total, dtype=torch.int32).cuda(), i32([0, total])
    rep, rows = torch.full((1,), 1.5).cuda(), i32([0, 4])
    rc = lp.load().lp_head_process(0x10000, 0, 0xF0000000, 64, 64, rows.data_ptr(), B, history.data_ptr(), off.data_ptr(),
                                   total, None, rep.data_ptr(), None, None, None, None, None, 0, None, 0, 0, None, 0x20000,
                                   64, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 3 and not ws.any()


@pytest.mark.parametrize("mean", [10, 5000])
@pytest.mark.parametrize("name,off", [("row_offsets", [0, 2, 1, 3]), ("row_offsets", [0, 1, 2, 4]), ("row_offsets", [0, 3, 3, 2]),
                                      ("bias_offsets", [0, 2, 1, 2]), ("bias_offsets", [0, 0, 1, 9]),
                                      ("history_offsets", [0, 2, 1, 3]), ("history_offsets", [0, 1, 2, 4])])
def test_offsets_wrong_anywhere_set_a_bit(name, off, mean):
    # also of requests that have no rows, or whose history has no effect
    B, V, total = 3, 700, 3 * mean
    if name == "history_offsets":
        off = [mean * o for o in off]
    args = dict(history=torch.zeros(total, dtype=torch.int32).cuda(), history_offsets=i32([0, mean, 2 * mean, total]),
                repetition=torch.ones(3).cuda(), bias_tokens=i32([4, 5]), bias_values=torch.zeros(2).cuda(),
                bias_offsets=i32([0, 1, 1, 2]), row_offsets=i32([0, 3, 3, 3]))
    x = torch.randn(3, V).cuda()
    ws = lp.new_head_workspace(requests=B, history=total)
    assert torch.equal(lp.process_logits(x, workspace=ws, **args), x) and lp.read_status(ws) == 0
    lp.process_logits(x, workspace=ws, **dict(args, **{name: i32(off)}))
    assert lp.read_status(ws) == bits(4)
