"""The 4-bit head, the processing of its logits, the draw, the logprob rows and the lookup of the drawn tokens together,
as a serving step runs them (examples/head_step.py), against the same chain in 64 bits; and in one graph."""

import importlib.util
import os

import pytest
import torch

import ragged_log_probs_gb300 as lp
from tests import fp4_reference as fp4
from tests import head_reference as ref
from tests import parity
from tests import sample_reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    parity.ensure_built()
    spec = importlib.util.spec_from_file_location("head_step", os.path.join(ROOT, "examples", "head_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_the_example_runs(example, capsys, bits, temperature):
    example.main(requests=4, hidden=256, vocab=5000, steps=3, bits=bits, temperature=temperature)
    assert capsys.readouterr().out.count("step") == 3


def values(q):
    codes, scales, rows = (t.cpu() for t in q)
    H = codes.shape[1] * 2
    return fp4.values(*fp4.unpack(codes), fp4.scale_values(scales, codes.shape[0], H, 16)[0], rows, 16)


def test_a_step_matches_the_chain_in_64_bits(example):
    B, H, V = 5, 512, 3001
    head = example.Head(B, H, V, adapters=2, rank=4, bits=4, temperature=0.7)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, r = (torch.randn(B, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    history = [h.tolist() for h in head.history]
    state = head.random.get_state()
    token, logprobs, tokens = head.step(x, r)
    head.random.set_state(state)
    u = torch.rand(B, generator=head.random, device="cuda").tolist()
    # the normed rows in bf16 and their 4 bits are tested by themselves: from those on, in 64 bits
    y = lp.rms_norm(x, head.gain, 1e-5, residual=r)
    number, negative, scales, rows = fp4.quantise(y.cpu(), 16)
    y4, w4 = fp4.values(number, negative, scales, rows, 16), values(head.weight4)
    allowed = torch.zeros(1, V, dtype=torch.bool)
    allowed[0, ::2] = True
    want, _ = ref.process(y4 @ w4.t(), history=history, prompt_lens=[len(t) for t in history],
                          rep=head.repetition.double().tolist(), freq=head.frequency.double().tolist(),
                          pres=head.presence.double().tolist(), mask=allowed, mask_index=head.mask_index.tolist())
    got, K = logprobs.double().cpu(), tokens.shape[1] - 1
    lw = want - torch.logsumexp(want, 1, keepdim=True)
    assert (head.logits.double().cpu() - want)[torch.isfinite(want)].abs().max() < 1e-4
    for b in range(B):
        # the draw, from the logits as they are in f32
        t, _, margin = sample_reference.draw(head.logits[b].cpu(), u[b], torch.tensor(0.7).item(), 50, torch.tensor(0.9).item())
        assert int(token[b]) == t or margin < 2.0 ** -31
        assert int(tokens[b, K]) == int(token[b]) and (got[b] - lw[b, tokens[b].tolist()]).abs().max() < 1e-4
        assert torch.equal(head.embeddings[b].double().cpu(), w4[int(token[b])].bfloat16().double())
    assert int(token[0]) % 2 == 0
    assert lp.read_status(head.head_ws) == 0 and lp.read_status(head.rows_ws) == 0


def test_the_chain_in_a_graph(example):
    B, H, V = 7, 256, 4001
    head = example.Head(B, H, V, adapters=3, rank=8, bits=4, temperature=0.9)
    x, r = (torch.randn(B, H, device="cuda").bfloat16() for _ in range(2))
    u = torch.rand(B, device="cuda")
    w, w_scales, w_row = head.weight4
    y = torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
    codes, scales, row_scale = lp.quantize_fp4(y)

    def run():
        lp.rms_norm(x, head.gain, 1e-5, residual=r, out=y)
        lp.quantize_fp4(y, 16, codes, scales, row_scale)
        lp.project_fp4(codes, scales, w, w_scales, 16, row_scale, w_row, out=head.logits, workspace=head.head_ws)
        lp.sample(head.logits, u, temperature=head.temperature, top_k=head.top_k, top_p=head.top_p, out=head.tokens,
                  workspace=head.head_ws)
        lp.dequantize_fp4(w, w_scales, w_row, rows=head.tokens, out=head.embeddings, workspace=head.head_ws)
        lp.step(head.logits, head.offsets, head.tokens, head.tokens, head.echo, head.levels, head.out_off, head.out_lp,
                head.out_tok, head.rows_ws)

    run()
    torch.cuda.synchronize()
    kept = head.logits, head.tokens, head.embeddings, head.out_lp, head.out_tok
    want = [t.clone() for t in kept]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        run()
    for t in kept:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
