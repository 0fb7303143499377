"""One serving step over several requests, from the library's entry points.

A block of a ternary model with adapters and drafted tokens: the rows of a
step are a few drafted tokens each of several requests, and every request may
have a low-rank adapter of its own.

    pages for the step's tokens, refused drafts' given back   pq2_pages_update, pq2_pages_copy
    q, k, v = projection of rms(r)                     pq2_rmsnorm, pq2_matmul
    q turned, k turned and v into the 4-bit cache      pq2_cache4_append
    a      = attention over the cache                  pq2_cache4_attend
    r     += output projection of a                    pq2_matmul, pq2_norm_residual
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


class Attention:
    """Weights, cache and buffers of the attention before a Block: `q_heads` query
    heads share `heads` key/value heads of `dim`."""

    def __init__(self, block, q_heads, heads, dim, length, page=32, seed=1, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.block, self.q_heads, self.heads, self.dim, self.page = block, q_heads, heads, dim, page
        rows, B = block.rows, block.requests
        wide = q_heads + 2 * heads

        def projection(N, K):
            tern = inputs.draw_ternary_torch(N, K, "p343", gen, device)
            return pq2.pack(tern, inputs.draw_ws_torch(N, K, gen, device))

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        self.qkv = projection(wide * dim, block.hidden)
        self.out = projection(block.hidden, q_heads * dim)
        self.ws_qkv = pq2.alloc_workspace(pq2.PQ2_OP_MATMUL, rows, wide * dim, block.hidden, device)
        self.ws_out = pq2.alloc_workspace(pq2.PQ2_OP_MATMUL, rows, block.hidden, q_heads * dim, device)
        W = -(-length // page)
        self.pool = pq2.alloc_cache4(B * (W + 1), heads, dim, page, device=device)
        self.pages = torch.full((2, B, W), -1, dtype=torch.int32, device=device)
        self.refs = torch.zeros((2, B * (W + 1)), dtype=torch.int32, device=device)
        self.turn = 0                                   # which of the two is in use
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.source = torch.arange(B, dtype=torch.int32, device=device)
        self.copies = empty(B, 2, dtype=torch.int32)
        self.info = empty(2, dtype=torch.int32)
        self.ws_pages = pq2.alloc_pages_workspace(B, B * (W + 1), device)
        self.ws_attend = pq2.alloc_attend_workspace(rows, q_heads, heads, dim, device)
        self.angles = empty(W * page, dim // 2, 2)
        pq2.pq2_rope_table(self.angles, 1e6)
        self.x = empty(rows, block.hidden, dtype=torch.float16)
        self.rows = empty(rows, wide, dim)
        self.q, self.a = (empty(rows, q_heads, dim, dtype=torch.float16) for _ in range(2))
        self.y, self.r_out = (empty(rows, block.hidden) for _ in range(2))

    def step(self, r, row_start, keep, max_rows=0):
        """r fp32 [rows, hidden] with row_start int32 [requests + 1]; keep int32
        [requests]: tokens of the cache that still hold (refused drafts do not);
        max_rows: rows of any request at most, where the host knows (0: all)."""
        b, now = self.block, self.turn
        after = keep + (row_start[1:] - row_start[:-1])
        pq2.pq2_pages_update(self.pages[now], self.refs[now], self.lens, self.source, keep, after, self.page,
                             self.pages[1 - now], self.refs[1 - now], self.copies, self.info, self.ws_pages)
        pq2.pq2_pages_copy(self.pool, self.copies)
        self.turn, self.lens = 1 - now, after
        pages = self.pages[self.turn]
        pq2.pq2_rmsnorm(r, b.w1, self.x, EPS)
        pq2.pq2_matmul(self.x, *self.qkv, self.rows.view(b.rows, -1), self.ws_qkv)
        h = self.q_heads
        pq2.pq2_cache4_append(self.rows[:, h:h + self.heads], self.rows[:, h + self.heads:], self.pool, pages, row_start,
                              after, q=self.rows[:, :h], q_out=self.q, table=self.angles)
        pq2.pq2_cache4_attend(self.q, self.pool, pages, row_start, after, self.a, self.ws_attend,
                              max_rows=max_rows)
        pq2.pq2_matmul(self.a.view(b.rows, -1), *self.out, self.y, self.ws_out)
        pq2.pq2_norm_residual(self.y, r, self.r_out, w_post=b.w2, eps=EPS, alpha=ALPHA)
        return self.r_out


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
    ap.add_argument("--query-heads", type=int, default=24)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--head-dim", type=int, default=256)
    a = ap.parse_args()
    block = Block(a.requests * (a.drafts + 1), a.hidden, a.inner, a.vocab, a.adapters, a.rank, a.requests)
    args = random_step(block, a.drafts, a.adapters)
    attention = Attention(block, a.query_heads, a.heads, a.head_dim, 32 * (a.drafts + 1))
    keep = torch.zeros(a.requests, dtype=torch.int32, device="cuda")

    def step():
        nonlocal keep
        r = attention.step(args["r"], args["row_start"], keep, a.drafts + 1)
        accepted, tokens = block.step(**{**args, "r": r})
        keep = keep + accepted + 1      # the drafts kept and the token before them
        return accepted, tokens

    for _ in range(3):
        accepted, tokens = step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        step()
    end.record()
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    print("accepted", accepted.tolist())
    print("tokens  ", tokens.view(a.requests, -1).tolist())
    print(f"{start.elapsed_time(end) / 20 * 1e3:.1f} us per step")


if __name__ == "__main__":
    main()
