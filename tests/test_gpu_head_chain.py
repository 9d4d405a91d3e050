"""The head's operators and the logprob rows together, as a serving step runs them
(examples/head_step.py), against the same chain in 64 bits."""

import importlib.util
import os

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import head_reference as ref
from tests import parity

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    parity.ensure_built()
    spec = importlib.util.spec_from_file_location("head_step", os.path.join(ROOT, "examples", "head_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_runs(example, capsys):
    example.main(requests=4, hidden=256, vocab=5000, steps=3)
    assert capsys.readouterr().out.count("step") == 3


def test_a_step_matches_the_chain_in_64_bits(example):
    B, H, V = 5, 512, 3001
    head = example.Head(B, H, V, adapters=2, rank=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, r = (torch.randn(B, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    history = [h.tolist() for h in head.history]
    best, logprobs, tokens = head.step(x, r)
    # from the 8-bit hidden states on (their rounding is tested by itself), in 64 bits
    h = head.hidden8.double().cpu() * head.hidden_scale.double().cpu()[:, None]
    y = h @ (head.weight.double().cpu() * head.weight_scale.double().cpu()[:, None]).t()
    for b, a in enumerate(head.adapter_ids.tolist()):
        if a >= 0:
            y[b] += head.lora_b[a].double().cpu() @ (head.lora_a[a].double().cpu() @ h[b])
    allowed = torch.zeros(1, V, dtype=torch.bool)
    allowed[0, ::2] = True
    want, _ = ref.process(y, history=history, prompt_lens=[len(t) for t in history], rep=head.repetition.double().tolist(),
                          freq=head.frequency.double().tolist(), pres=head.presence.double().tolist(), mask=allowed,
                          mask_index=head.mask_index.tolist())
    want = want - torch.logsumexp(want, 1, keepdim=True)
    K = tokens.shape[1] - 1
    got = logprobs.double().cpu()
    for b in range(B):
        ids = tokens[b].tolist()
        # f32 logits of magnitude below 16 and their logsumexp: errors below 1e-4
        assert (got[b] - want[b, ids]).abs().max() < 1e-4
        assert ids[0] == ids[K] == int(best[b]) and int(best[b]) % 2 == 0 or b > 0
        assert want[b, ids[0]] >= want[b].max() - 1e-4
    assert lp.read_status(head.head_ws) == 0 and lp.read_status(head.rows_ws) == 0


def test_the_chain_in_a_graph(example):
    B, H, V = 7, 256, 4001
    head = example.Head(B, H, V, adapters=3, rank=8)
    x, r = (torch.randn(B, H, device="cuda").bfloat16() for _ in range(2))
    hist = torch.cat(head.history)
    lens = torch.tensor([0] + [h.numel() for h in head.history]).cumsum(0).to(torch.int32).cuda()
    best = torch.zeros(B, dtype=torch.int32, device="cuda")

    def run():
        lp.rms_norm(x, head.gain, 1e-5, residual=r, out=head.hidden8, out_scale=head.hidden_scale)
        lp.project(head.hidden8, head.weight, x_scale=head.hidden_scale, weight_scale=head.weight_scale,
                   lora_a=head.lora_a, lora_b=head.lora_b, adapter_ids=head.adapter_ids, out=head.logits,
                   workspace=head.head_ws)
        lp.process_logits(head.logits, history=hist, history_offsets=lens, prompt_lens=head.prompt_lens,
                          repetition=head.repetition, out=head.logits, workspace=head.head_ws)
        lp.step(head.logits, head.offsets, best, best, head.echo, head.levels, head.out_off, head.out_lp, head.out_tok,
                head.rows_ws)

    run()
    torch.cuda.synchronize()
    want = head.logits.clone(), head.out_lp.clone(), head.out_tok.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    for t in (head.logits, head.out_lp, head.out_tok):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(head.logits, want[0]) and torch.equal(head.out_lp, want[1]) and torch.equal(head.out_tok, want[2])


def test_every_row_leads_with_its_chosen_token(example):
    # the best token is the first of the top and the row's own, in every row; the first row's is even
    B = 6
    head = example.Head(B, 256, 2001, adapters=2, rank=4, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    for _ in range(3):
        x, r = (torch.randn(B, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
        best, logprobs, tokens = head.step(x, r)
        K = tokens.shape[1] - 1
        for b in range(B):
            assert int(tokens[b, 0]) == int(tokens[b, K]) == int(best[b])
            assert float(logprobs[b, 0]) == float(logprobs[b, K])
        assert int(best[0]) % 2 == 0
