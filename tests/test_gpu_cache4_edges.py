"""The 4-bit cache at the edges of what a call may hold: tokens without a place,
groups of many heads, numbers of rows on both sides of a change of kernel."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_gpu_cache4 import Cache, _attend, _check, _dev, _np, _q

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


@pytest.mark.parametrize("D,out", [(64, torch.float16), (128, torch.float32), (256, torch.bfloat16)])
@pytest.mark.parametrize("angles", ["none", "places", "positions"])
def test_queries_of_tokens_without_a_place(pq2, D, out, angles):
    # before the first position or behind the table's last: the whole token is skipped; a
    # page outside the pool: its queries are written all the same
    H, Hq, T, W = 1, 3, 16, 2
    c = Cache(pq2, 1, W, H, D, T)
    pages = c.pages.copy()
    pages[0, 1] = 10 ** 6
    g = torch.Generator(device=DEV).manual_seed(D)
    for n, ln, there in ((4, 2, [False, False, True, True]),          # positions -2 .. 1
                         (3, 34, [True, False, False]),               # 31 (no page), 32, 33
                         (2, 40, [False, False]), (2, 18, [True, True])):
        x = torch.randn((n, Hq + 2, D), generator=g, device=DEV)
        kw = {}
        if angles != "none":
            kw["table"] = torch.empty((64, D // 2, 2), device=DEV)
            pq2.pq2_rope_table(kw["table"], 1e4)
        if angles == "positions":
            kw["positions"] = _dev(np.arange(n))
        q_out = torch.full((n, Hq, D), 9.0, dtype=out, device=DEV)
        pq2.pq2_cache4_append(x[:, Hq:Hq + 1], x[:, Hq + 1:], c.pool, _dev(pages), _dev([0, n]), _dev([ln]), q=x[:, :Hq],
                              q_out=q_out, **kw)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
        written = (q_out != 9.0).any(-1).any(-1).tolist()
        assert written == there, (n, ln)


@pytest.mark.parametrize("G", [25, 33, 48, 64])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 7])
def test_groups_of_many_heads(pq2, G, D, n):
    lens = [n, 40, 131]
    c = Cache(pq2, 3, 9, 1, D, 16, seed=G)
    pool = c.fill(lens)
    q = _q(3 * n, G, D, "f16")
    got = _attend(pq2, c, q, [n] * 3, lens, max_rows=n)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, pool, c, [n] * 3, lens)


@pytest.mark.parametrize("D,G,n", [(64, 1, [47, 48, 49, 50, 2]), (128, 3, [15, 16, 17, 1, 0]), (128, 1, [49, 48, 0, 49, 1]),
                                   (256, 1, [31, 32, 33, 34, 1]), (256, 4, [9, 8, 7, 9, 0])])
@pytest.mark.parametrize("window", [0, 37])
def test_rows_on_both_sides_of_the_change_of_kernel(pq2, D, G, n, window):
    # sequences with just as many rows as the one kernel takes, and with one more, in one call
    lens = [max(k, 20 + 30 * i) for i, k in enumerate(n)]
    c = Cache(pq2, len(n), -(-max(lens) // 16), 1, D, 16, seed=D)
    pool = c.fill(lens)
    q = _q(sum(n) + 1, G, D, "bf16")
    for max_rows in (0, max(n)):
        got = _attend(pq2, c, q, n, lens, window, max_rows=max_rows)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        _check(got, q, pool, c, n, lens, window, dtype="bf16")
        assert torch.all(got[sum(n):] == 7.0)
    for n0 in sorted(set(n)):                  # and alone
        if n0 == 0:
            continue
        b = n.index(n0)
        r0 = sum(n[:b])
        one = Cache.__new__(Cache)
        one.T, one.D, one.H, one.pool, one.pages, one.dev = 16, D, 1, c.pool, c.pages[b:b + 1], c.dev[b:b + 1].contiguous()
        alone = _attend(pq2, one, q[r0:r0 + n0].contiguous(), [n0], [lens[b]], window)
        _check(alone, q[r0:r0 + n0], pool, one, [n0], [lens[b]], window, dtype="bf16")


VALUES = 1 << 16   # withheld pieces of values, with many rows


@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (256, 1), (64, 20), (128, 20), (256, 20)])
@pytest.mark.parametrize("stage", [1, 2, 3, 4, VALUES, VALUES + 1, VALUES + 2, VALUES + 3])
def test_a_piece_that_never_comes(pq2, D, n, stage):
    # 24 tiles and more for each warp, or CTA; few rows have no pieces of values
    ln, W, G = 60000, 200, 6
    pool = torch.zeros((2, 1, 16 * (D + 8) * 20), dtype=torch.uint8, device=DEV)
    pages = _dev(np.arange(64 * W).reshape(64, W) % 2)
    q = _q(64 * n, G, D, "f16")
    out = torch.empty_like(q)
    ws = pq2.alloc_attend_workspace(64 * n, G, 1, D)
    start, lens = _dev(n * np.arange(65)), _dev(np.full(64, ln))

    def run():
        pq2.pq2_cache4_attend(q, pool, pages, start, lens, out, ws, max_rows=n)
        return pq2.pq2_last_device_error()

    assert run() == pq2.PQ2_OK and torch.all(out == 0)
    try:
        pq2.pq2_debug_set_wait_limit_ns(20_000_000)
        pq2.pq2_debug_skip_stage(stage)
        assert run() == (pq2.PQ2_OK if n == 1 and stage >= VALUES else pq2.PQ2_ERR_TIMEOUT)
    finally:
        pq2.pq2_debug_skip_stage(-1)
        pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
    assert run() == pq2.PQ2_OK and torch.all(out == 0)


@pytest.mark.parametrize("drafts", [0, 7])
def test_steps_of_the_serving_example_that_know_their_rows(pq2, drafts):
    import serving_step
    B, q_heads, heads, dim = 9, 4, 1, 128
    block = serving_step.Block(B * (drafts + 1), 512, 640, 1000, 2, 16, B)
    args = serving_step.random_step(block, drafts, 2)
    at = serving_step.Attention(block, q_heads, heads, dim, 40 * (drafts + 1), page=16)
    keep = torch.zeros(B, dtype=torch.int32, device=DEV)
    for step in range(3):
        at.step(args["r"] * (1 + step), args["row_start"], keep, max_rows=drafts + 1)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        want, tol = ref.attend(_np(at.q), at.pool.cpu().numpy(), at.pages[at.turn].cpu().numpy(),
                               args["row_start"].cpu().numpy(), at.lens.cpu().numpy(), 16, dim ** -0.5, 0)
        err = np.abs(at.a.double().cpu().numpy() - want)
        assert np.all(err <= tol + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
        keep = keep + drafts + 1


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 5, 60])
def test_heads_before_tokens(pq2, D, n):
    # all arrays laid out [heads, tokens, values], the first token of the call a sequence of none
    Hq, H, T, ln = 4, 2, 16, 75
    g = torch.Generator(device=DEV).manual_seed(D + n)
    table = torch.empty((128, D // 2, 2), device=DEV)
    pq2.pq2_rope_table(table, 1e4)

    def across(heads, dtype=torch.float16):
        return torch.randn((heads, n + 2, D), generator=g, device=DEV).to(dtype).transpose(0, 1)
    c, plain = (Cache(pq2, 1, -(-ln // T), H, D, T, seed=D) for _ in range(2))
    pool = c.fill([ln])
    plain.pool.copy_(c.pool)
    q, k, v = across(Hq), across(H), across(H)
    outs = []
    for cache, lay in ((c, lambda t: t), (plain, lambda t: t.contiguous())):
        q_out, out, kr, vr = (torch.full((h, n + 2, D), 7.0, dtype=torch.float16, device=DEV).transpose(0, 1) for h in (Hq, Hq, H, H))
        q_out, out, kr, vr = lay(q_out), lay(out), lay(kr), lay(vr)
        args = (cache.pool, cache.dev, _dev([1, 1 + n]), _dev([ln]))
        pq2.pq2_cache4_append(lay(k), lay(v), *args, q=lay(q), q_out=q_out, table=table)
        pq2.pq2_cache4_read(*args, kr, vr)
        pq2.pq2_cache4_attend(q_out, *args, out, pq2.alloc_attend_workspace(n + 2, Hq, H, D))
        turned = lay(torch.full((Hq, n + 2, D), 7.0, dtype=torch.float16, device=DEV).transpose(0, 1))
        pq2.pq2_rope(lay(q), table, _dev(np.arange(n + 2)), turned)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        outs.append([t.clone() for t in (q_out, out, kr, vr, turned, cache.pool)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for t in outs[0][:4]:                      # rows of no sequence are left as they were
        assert torch.all(t[0] == 7.0) and torch.all(t[n + 1] == 7.0)
    want, tol = ref.attend(_np(outs[0][0][1:1 + n]), c.pool.cpu().numpy(), c.pages, [0, n], [ln], T, D ** -0.5)
    err = np.abs(outs[0][1][1:1 + n].double().cpu().numpy() - want)
    assert np.all(err <= tol + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
    assert pool is not None


@pytest.mark.parametrize("H,D,n", [(1024, 64, 1), (1000, 128, 2), (300, 64, 60)])
def test_many_key_value_heads(pq2, H, D, n):
    ln, T = 70, 16
    c = Cache(pq2, 2, 5, H, D, T, spare=0)
    g = torch.Generator(device=DEV).manual_seed(H)
    x = torch.randn((2, ln, 2 * H, D), generator=g, device=DEV).flatten(0, 1)
    pq2.pq2_cache4_append(x[:, :H], x[:, H:], c.pool, c.dev, _dev([0, ln, 2 * ln]), _dev([ln, ln]))
    q = _q(2 * n, H, D, "f16")
    got = _attend(pq2, c, q, [n, n], [ln, ln], max_rows=n)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    pool = c.pool.cpu().numpy()
    for h in (0, 1, H // 2, H - 1):
        want, tol = ref.attend(_np(q[:, h:h + 1]), pool[:, h:h + 1], c.pages, [0, n, 2 * n], [ln, ln], T, D ** -0.5)
        err = np.abs(got[:, h:h + 1].double().cpu().numpy() - want)
        assert np.all(err <= tol + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)


@pytest.mark.parametrize("D,T,n", [(64, 1024, 1), (128, 1008, 3), (256, 1024, 40), (128, 1024, 70)])
def test_large_pages(pq2, D, T, n):
    lens = [1100, 2017, 16]
    rows = [n, n, min(n, 16)]
    c = Cache(pq2, 3, 3, 1, D, T, spare=1)
    pool = c.fill(lens)
    q = _q(sum(rows), 2, D, "bf16")
    got = _attend(pq2, c, q, rows, lens)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, pool, c, rows, lens, dtype="bf16")


@pytest.mark.parametrize("n", [1, 60])
def test_a_captured_step_over_changing_lengths(pq2, n):
    # one graph, replayed after the lengths, the pages and the queries have changed
    Hq, H, D, T, B = 4, 2, 128, 16, 3
    c = Cache(pq2, B, 20, H, D, T)
    pool = c.fill([320] * B)
    q, out = _q(B * n, Hq, D, "f16"), torch.empty((B * n, Hq, D), dtype=torch.float16, device=DEV)
    start, lens = _dev(n * np.arange(B + 1)), _dev([n] * B)
    ws = pq2.alloc_attend_workspace(B * n, Hq, H, D)
    pq2.pq2_cache4_attend(q, c.pool, c.dev, start, lens, out, ws, max_rows=n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq2.pq2_cache4_attend(q, c.pool, c.dev, start, lens, out, ws, max_rows=n)
    rng = np.random.default_rng(1)
    for step in range(4):
        now = rng.integers(n, 321, B)
        c.pages = c.pages[rng.permutation(B)]
        c.dev.copy_(_dev(c.pages))
        lens.copy_(_dev(now))
        q.copy_(_q(B * n, Hq, D, "f16", seed=step))
        g.replay()
        _check(out, q, pool, c, [n] * B, now)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
