"""One decode step of a served model's head, from the last layer's output to the logprob rows.

    hidden --rms_norm--> e4m3 --project (+ adapters)--> logits --process_logits--> --sample--> --step--> rows

or, with a head in 4 bits, which the next step's embeddings are looked up in as well:

    hidden --rms_norm--> bf16 --quantize_fp4--> --project_fp4--> logits --process_logits--> --sample--> --step--> rows
                                                          --dequantize_fp4--> embeddings of the drawn tokens

Random hidden states and weights of a small head; prints each request's next token (by default
the best of its processed logits) with its logprob, for a few steps in which the chosen tokens join the
histories. Run from the repository's root, after the library has been built:

    python examples/head_step.py [bits of the head: 8 or 4] [temperature]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ragged_log_probs_gb300 as lp  # noqa: E402


class Head:
    """The buffers and weights that a serving program keeps between steps."""

    def __init__(self, requests, hidden, vocab, adapters, rank, levels=3, max_history=512, seed=0, bits=8,
                 temperature=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.B, self.H, self.V, self.levels, self.bits = requests, hidden, vocab, levels, bits
        self.gain = (1.0 + 0.1 * rn(hidden)).bfloat16()
        w = rn(vocab, hidden) * (2.0 / hidden ** 0.5)
        self.weight_scale = w.abs().amax(1) / 448.0          # an 8-bit head, one scale a token
        self.weight = (w / self.weight_scale[:, None]).to(torch.float8_e4m3fn)
        if bits == 4:  # one scale for 16 elements, laid out once; no adapters
            self.weight4 = lp.quantize_fp4(w.bfloat16())
            self.embeddings = torch.empty(requests, hidden, dtype=torch.bfloat16, device="cuda")
        self.lora_a = (rn(adapters, rank, hidden) / hidden ** 0.5).bfloat16()
        self.lora_b = (rn(adapters, vocab, rank) * 0.2).bfloat16()
        self.adapter_ids = (torch.arange(requests, device="cuda") % (adapters + 1) - 1).to(torch.int32)  # -1: none
        self.repetition = torch.full((requests,), 1.2, device="cuda")
        self.frequency = torch.full((requests,), 0.3, device="cuda")
        self.presence = torch.full((requests,), 0.1, device="cuda")
        # a grammar for the first request: only even tokens
        words = (vocab + 31) // 32
        self.mask = torch.full((1, words), 0x55555555, dtype=torch.int32, device="cuda")
        self.mask_index = torch.full((requests,), -1, dtype=torch.int32, device="cuda")
        self.mask_index[0] = 0
        self.history = [torch.randint(0, vocab, (5 + 3 * b,), generator=g, device="cuda", dtype=torch.int32)
                        for b in range(requests)]
        self.prompt_lens = torch.tensor([h.numel() for h in self.history], dtype=torch.int32, device="cuda")
        # how the tokens are drawn: temperature 0 takes the best
        self.random = g
        self.temperature = torch.full((requests,), temperature, device="cuda")
        self.top_k = torch.full((requests,), 50, dtype=torch.int32, device="cuda")
        self.top_p = torch.full((requests,), 0.9, device="cuda")
        self.tokens = torch.empty(requests, dtype=torch.int32, device="cuda")
        # what the logprob rows need: one row a request
        self.offsets = torch.arange(requests + 1, dtype=torch.int32, device="cuda")
        self.echo = torch.zeros(requests, dtype=torch.uint8, device="cuda")
        W = lp.out_per_token(levels)
        self.hidden8 = torch.empty(requests, hidden, dtype=torch.float8_e4m3fn, device="cuda")
        self.hidden_scale = torch.empty(requests, device="cuda")
        self.logits = torch.empty(requests, vocab, device="cuda")
        self.out_off = torch.empty(requests + 1, dtype=torch.int32, device="cuda")
        self.out_lp = torch.empty(requests, W, device="cuda")
        self.out_tok = torch.empty(requests, W, dtype=torch.int32, device="cuda")
        self.head_ws = lp.new_head_workspace(requests, rank, requests, requests * max_history, draws=requests,
                                             vocab=vocab)
        self.rows_ws = lp.new_workspace(requests, requests, vocab, levels)

    def step(self, x, residual):
        """Logits of the last layer's output, processed; its logprob rows; the token drawn for each."""
        if self.bits == 4:
            y = lp.rms_norm(x, self.gain, 1e-5, residual=residual)
            codes, scales, row_scale = lp.quantize_fp4(y)
            w, w_scales, w_row = self.weight4
            lp.project_fp4(codes, scales, w, w_scales, x_row_scale=row_scale, weight_row_scale=w_row, out=self.logits,
                           workspace=self.head_ws)
        else:
            lp.rms_norm(x, self.gain, 1e-5, residual=residual, out=self.hidden8, out_scale=self.hidden_scale)
            lp.project(self.hidden8, self.weight, x_scale=self.hidden_scale, weight_scale=self.weight_scale,
                       lora_a=self.lora_a, lora_b=self.lora_b, adapter_ids=self.adapter_ids, out=self.logits,
                       workspace=self.head_ws)
        lens = torch.tensor([0] + [h.numel() for h in self.history]).cumsum(0).to(torch.int32).cuda()
        lp.process_logits(self.logits, history=torch.cat(self.history), history_offsets=lens,
                          prompt_lens=self.prompt_lens, repetition=self.repetition, frequency=self.frequency,
                          presence=self.presence, mask=self.mask, mask_index=self.mask_index, out=self.logits,
                          workspace=self.head_ws)
        # the row's own token is the one just drawn
        uniform = torch.rand(self.B, generator=self.random, device="cuda")
        best = lp.sample(self.logits, uniform, temperature=self.temperature, top_k=self.top_k, top_p=self.top_p,
                         out=self.tokens, workspace=self.head_ws).clone()
        if self.bits == 4:
            w, w_scales, w_row = self.weight4
            lp.dequantize_fp4(w, w_scales, w_row, rows=best, out=self.embeddings, workspace=self.head_ws)
        lp.step(self.logits, self.offsets, best, best, self.echo, self.levels, self.out_off, self.out_lp, self.out_tok,
                self.rows_ws)
        self.history = [torch.cat([h, best[b:b + 1]]) for b, h in enumerate(self.history)]
        return best, self.out_lp, self.out_tok


def main(requests=6, hidden=1024, vocab=32000, steps=4, bits=8, temperature=0.0):
    head = Head(requests, hidden, vocab, adapters=3, rank=8, bits=bits, temperature=temperature)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for n in range(steps):
        x, residual = (torch.randn(requests, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
        best, logprobs, tokens = head.step(x, residual)
        K = tokens.shape[1] - 1
        print(f"step {n}: " + "  ".join(f"{int(t)} ({float(l):.2f})" for t, l in zip(best, logprobs[:, K])))
    status = lp.read_status(head.head_ws) | lp.read_status(head.rows_ws)
    if status:
        raise SystemExit(f"status {status:#x}")
    return head


if __name__ == "__main__":
    main(bits=int(sys.argv[1]) if len(sys.argv) > 1 else 8, temperature=float(sys.argv[2]) if len(sys.argv) > 2 else 0.0)
