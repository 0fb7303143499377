"""One serving step over several requests, from the library's entry points.

A block of a ternary model with adapters and drafted tokens: the rows of a
step are a few drafted tokens each of several requests, and every request may
have a low-rank adapter of its own.

    x      = rms(r) * w1                               pq2_rmsnorm
    gu     = gate/up projection of x                   pq2_matmul
    gu    += adapter on gate/up                        pq2_lora_add (in place)
    y      = down projection of silu(gate) * up        pq2_mlp_down_swiglu
    r', x' = r + alpha * rms(y) * w2, rms(r') * w3     pq2_norm_residual
    logits = lm_head of x'                             pq2_matmul
    kept drafts and the next token of each request     pq2_verify_drafts

Random weights stand in for a checkpoint.  Run it as

    python examples/serving_step.py [--requests 4] [--drafts 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gemm_pq2_ternary_gb300 import binding as pq2  # noqa: E402
from gemm_pq2_ternary_gb300 import inputs  # noqa: E402

EPS = 1e-6
ALPHA = 1.0


class Block:
    """Weights and buffers for steps of up to `rows` token rows."""

    def __init__(self, rows, hidden, inner, vocab, adapters, rank, requests, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.rows, self.hidden, self.inner, self.vocab = rows, hidden, inner, vocab
        self.requests = requests

        def projection(N, K):
            tern = inputs.draw_ternary_torch(N, K, "p343", gen, device)
            return pq2.pack(tern, inputs.draw_ws_torch(N, K, gen, device))

        def randn(*shape):
            return torch.randn(shape, generator=gen, device=device)

        self.gate_up = projection(2 * inner, hidden)
        self.down = projection(hidden, inner)
        self.lm_head = projection(vocab, hidden)
        self.w1, self.w2, self.w3 = (1.0 + 0.1 * randn(hidden) for _ in range(3))
        self.A = (randn(adapters, rank, hidden) * hidden ** -0.5).half()
        self.B = (randn(adapters, 2 * inner, rank) * 0.1).half()
        self.scales = torch.full((adapters,), 0.5, device=device)

        def workspace(op, N, K):
            return pq2.alloc_workspace(op, rows, N, K, device)

        self.ws_gate_up = workspace(pq2.PQ2_OP_MATMUL, 2 * inner, hidden)
        self.ws_down = workspace(pq2.PQ2_OP_SWIGLU_DOWN, hidden, inner)
        self.ws_head = workspace(pq2.PQ2_OP_MATMUL, vocab, hidden)
        self.ws_lora = pq2.alloc_lora_workspace(rows, 2 * inner, hidden, adapters, rank, device)
        self.ws_verify = pq2.alloc_verify_workspace(requests, rows, vocab, device)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        self.x = empty(rows, hidden, dtype=torch.float16)
        self.gu = empty(rows, 2 * inner)
        self.y = empty(rows, hidden)
        self.r_out = empty(rows, hidden)
        self.x_out = empty(rows, hidden, dtype=torch.float16)
        self.logits = empty(rows, vocab)
        self.accepted = empty(requests, dtype=torch.int32)
        self.tokens = empty(rows, dtype=torch.int32)

    def step(self, r, ids, row_start, drafts, u, e, temperature):
        """r fp32 [rows, hidden]; ids int32 [rows], each row's adapter (-1:
        none); row_start int32 [requests + 1]; drafts int32 [rows], each row's
        drafted next token (the drafter was certain of it); u [rows] and
        e [requests, vocab] the random numbers; temperature [requests]."""
        pq2.pq2_rmsnorm(r, self.w1, self.x, EPS)
        pq2.pq2_matmul(self.x, *self.gate_up, self.gu, self.ws_gate_up)
        pq2.pq2_lora_add(self.x, self.A, self.B, ids, self.gu, self.gu, self.ws_lora,
                         scales=self.scales)
        pq2.pq2_mlp_down_swiglu(self.gu, *self.down, self.y, self.ws_down)
        pq2.pq2_norm_residual(self.y, r, self.r_out, w_post=self.w2, w_next=self.w3, x=self.x_out,
                              eps=EPS, alpha=ALPHA)
        pq2.pq2_matmul(self.x_out, *self.lm_head, self.logits, self.ws_head)
        pq2.pq2_verify_drafts(self.logits, row_start, drafts, None, u, e, temperature, self.accepted,
                              self.tokens, self.ws_verify)
        return self.accepted, self.tokens


def random_step(block, drafts, adapters, seed=0, device="cuda"):
    """Arguments of Block.step for requests with `drafts` drafts each."""
    gen = torch.Generator(device=device).manual_seed(seed)
    n, rows = block.requests, block.rows
    assert rows == n * (drafts + 1)
    row_start = torch.arange(0, rows + 1, drafts + 1, dtype=torch.int32, device=device)
    request = torch.arange(rows, device=device) // (drafts + 1)
    ids = (request % (adapters + 1) - 1).to(torch.int32)      # every so many without one
    return dict(r=torch.randn((rows, block.hidden), generator=gen, device=device), ids=ids,
                row_start=row_start,
                drafts=torch.randint(0, block.vocab, (rows,), generator=gen, device=device,
                                     dtype=torch.int32),
                u=torch.rand(rows, generator=gen, device=device),
                e=torch.empty((n, block.vocab), device=device).exponential_(generator=gen),
                temperature=torch.full((n,), 0.8, device=device))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inner", type=int, default=17408)
    ap.add_argument("--vocab", type=int, default=248320)
    ap.add_argument("--adapters", type=int, default=3)
    ap.add_argument("--rank", type=int, default=16)
    a = ap.parse_args()
    block = Block(a.requests * (a.drafts + 1), a.hidden, a.inner, a.vocab, a.adapters, a.rank, a.requests)
    args = random_step(block, a.drafts, a.adapters)
    for _ in range(3):
        accepted, tokens = block.step(**args)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        block.step(**args)
    end.record()
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    print("accepted", accepted.tolist())
    print("tokens  ", tokens.view(a.requests, -1).tolist())
    print(f"{start.elapsed_time(end) / 20 * 1e3:.1f} us per step")


if __name__ == "__main__":
    main()
