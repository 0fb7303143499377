"""What the attention over the 4-bit cache does at its limits: a tile that never
comes, stores outside a buffer in the bounds-checked build, keys far from
zero, and a step of the serving example with it."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle.step import TINY, UNIT
from test_gpu_cache4 import Cache, _attend, _check, _dev, _np, _q, _starts

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAD = 64
SENTINEL = 123.0


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


@pytest.mark.parametrize("Hq,H,D,n", [(4, 2, 64, 1), (6, 1, 128, 5), (6, 1, 256, 1),        # few rows
                                      (2, 2, 64, 70), (6, 1, 128, 9), (6, 1, 128, 60), (6, 1, 256, 30)])
@pytest.mark.parametrize("stage", [0, 1])
def test_a_tile_that_never_comes(pq2, Hq, H, D, n, stage):
    # (tile or half of a tile `stage` of every ring is withheld; of 1500 tokens a
    # warp, or a CTA, may have one tile and no second one)
    reaches = stage == 0
    ln = 1500
    c = Cache(pq2, 1, -(-ln // 64), H, D, 64)
    pool = c.fill([ln])
    q = _q(n, Hq, D, "f16")
    want = _attend(pq2, c, q, [n], [ln])
    _check(want, q, pool, c, [n], [ln])
    try:
        pq2.pq2_debug_set_wait_limit_ns(20_000_000)
        pq2.pq2_debug_skip_stage(stage)
        got = _attend(pq2, c, q, [n], [ln])
        error = pq2.pq2_last_device_error()
        assert error == pq2.PQ2_ERR_TIMEOUT or (not reaches and error == pq2.PQ2_OK and torch.equal(got, want))
    finally:
        pq2.pq2_debug_skip_stage(-1)
        pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
    assert torch.equal(_attend(pq2, c, q, [n], [ln]), want)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("stage", [1, 2])
def test_a_later_tile_that_never_comes(pq2, stage, n):
    # 24 tiles and more for each warp, or CTA
    ln, W = 60000, 200
    pool = torch.zeros((2, 1, 16 * 136 * 20), dtype=torch.uint8, device=DEV)
    pages = _dev(np.arange(64 * W).reshape(64, W) % 2)
    q = _q(64 * n, 6, 128, "f16")
    out = torch.empty_like(q)
    ws = pq2.alloc_attend_workspace(64 * n, 6, 1, 128)
    start, lens = _dev(n * np.arange(65)), _dev(np.full(64, ln))

    def run():
        pq2.pq2_cache4_attend(q, pool, pages, start, lens, out, ws, max_rows=n)
        return pq2.pq2_last_device_error()

    assert run() == pq2.PQ2_OK and torch.all(out == 0)
    try:
        pq2.pq2_debug_set_wait_limit_ns(20_000_000)
        pq2.pq2_debug_skip_stage(stage)
        assert run() == pq2.PQ2_ERR_TIMEOUT
    finally:
        pq2.pq2_debug_skip_stage(-1)
        pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
    assert run() == pq2.PQ2_OK and torch.all(out == 0)


@pytest.mark.parametrize("n", [1, 6, 60])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_far_from_zero(pq2, D, n):
    # scores that are small differences of z sum(q): weights tell how well both are kept
    ln, H, G = 96, 1, 2
    c = Cache(pq2, 1, 6, H, D, 16)
    g = torch.Generator(device=DEV).manual_seed(D + n)
    k = 8.0 + torch.randn((ln, H, D), generator=g, device=DEV)
    v = torch.randn((ln, H, D), generator=g, device=DEV)
    pq2.pq2_cache4_append(k, v, c.pool, c.dev, _dev([0, ln]), _dev([ln]))
    q = (0.5 + 0.1 * torch.randn((n, H * G, D), generator=g, device=DEV)).half()
    got = _attend(pq2, c, q, [n], [ln])
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, c.pool.cpu().numpy(), c, [n], [ln])


@pytest.mark.parametrize("Hq,H,D,n", [(10, 2, 128, 5), (10, 2, 128, 200), (6, 1, 256, 100), (1, 1, 64, 300)])
def test_rows_of_different_lengths_share_the_work(pq2, Hq, H, D, n):
    # long sequences next to many short ones: parts of items and whole ones in one CTA
    lens = [2000] + [n + 3 * i for i in range(12)] + [1, 0]
    rows = [n] + [n] * 12 + [1, 0]
    c = Cache(pq2, len(lens), -(-max(lens) // 16), H, D, 16, seed=3)
    pool = c.fill(lens)
    q = _q(sum(rows), Hq, D, "bf16")
    got = _attend(pq2, c, q, rows, lens)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    b = 0
    for i in (0, 1, 12, 13):  # (some of them against the definition)
        r0 = int(_starts(rows)[i])
        sub = _Part(c, i)
        _check(got[r0:r0 + rows[i]], q[r0:r0 + rows[i]], pool, sub, [rows[i]], [lens[i]], dtype="bf16")
        b += 1
    assert torch.equal(got, _attend(pq2, c, q, rows, lens))


class _Part:
    """One sequence of a cache."""

    def __init__(self, c, b):
        self.T, self.D, self.H, self.pages = c.T, c.D, c.H, c.pages[b:b + 1]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n", [(64, 70), (128, 5), (128, 70), (256, 40)])
def test_rows_with_infinities_stay_among_themselves(pq2, D, n, dtype):
    ln, G = 200, 2
    c = Cache(pq2, 1, 13, 1, D, 16)
    pool = c.fill([ln])
    q = _q(n, G, D, dtype)
    bad = q.clone()
    bad[1, 0, 3] = float("inf")
    bad[2, 1, D - 1] = float("nan")
    bad[n - 1, 0, 0] = float("-inf")
    got = _attend(pq2, c, bad, [n], [ln])
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    for i, h in ((1, 0), (2, 1), (n - 1, 0)):
        got[i, h] = 0.0
    want, tol = ref.attend(_np(q), pool, c.pages, _starts([n]), [ln], 16, D ** -0.5, 0)
    for i, h in ((1, 0), (2, 1), (n - 1, 0)):
        want[i, h] = 0.0
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol + np.abs(want) * UNIT[dtype] + TINY[dtype])


@pytest.mark.parametrize("D,n", [(64, 70), (128, 70), (256, 40)])
def test_rows_of_very_different_size(pq2, D, n):
    # bf16 rows from 2^-60 to 2^60: small ones count as what they are next to the largest
    ln = 100
    c = Cache(pq2, 1, 7, 1, D, 16)
    pool = c.fill([ln], spread=1e-3)
    q = _q(n, 2, D, "bf16")
    q = (q.float() * torch.exp2(torch.arange(n, device=DEV).float()[:, None, None] * (120.0 / n) - 60.0)).bfloat16()
    got = _attend(pq2, c, q, [n], [ln], scale=2.0 ** -58)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    want, tol = ref.attend(_np(q), pool, c.pages, _starts([n]), [ln], 16, 2.0 ** -58, 0)
    # a value of q is off by up to 2^-22 of the largest, so a score by D k 2^-22 times the scale
    kmax = max(np.abs(ref.read_rows(pool, c.pages[0], ln, 0, 16, D)[1].astype(np.float64)).max() * 16, 1e-30)
    off = 2.0 ** -22 * float(q.float().abs().max()) * 2.0 ** -58 * D * kmax
    vmax = np.abs(want).max() + 1e-2
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol + np.abs(want) * UNIT["bf16"] + TINY["bf16"] + 2 * off * vmax)


@pytest.mark.parametrize("D,T,n", [(128, 16, 1), (128, 16, 9), (64, 16, 70), (128, 32, 60), (256, 64, 40)])
def test_pages_before_a_window_may_be_gone(pq2, D, T, n):
    ln, window = 700, 50
    c = Cache(pq2, 1, -(-ln // T), 1, D, T)
    pool = c.fill([ln])
    q = _q(n, 2, D, "f16")
    want = _attend(pq2, c, q, [n], [ln], window=window)
    _check(want, q, pool, c, [n], [ln], window=window)
    c.dev[0, :(ln - n - window + 1) // T] = -1
    got = _attend(pq2, c, q, [n], [ln], window=window)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    assert torch.equal(got, want)


@pytest.mark.parametrize("Hq,H,D", [(6, 2, 64), (5, 1, 128), (4, 1, 256)])
@pytest.mark.parametrize("window", [0, 30])
def test_prompts_around_many_decoding_sequences(pq2, Hq, H, D, window):
    # more sequences than a walk looks at at once, empty ones among them, in both kernels' shares
    n = [90] + [1, 0, 1, 2] * 20 + [300] + [1] * 5 + [0] * 40 + [33]
    lens = [95] + [17, 0, 33, 5] * 20 + [310] + [64] * 5 + [9] * 40 + [40]
    c = Cache(pq2, len(n), -(-max(lens) // 16), H, D, 16, seed=5)
    pool = c.fill(lens)
    q = _q(sum(n) + 1, Hq, D, "f16")
    got = _attend(pq2, c, q, n, lens, window=window)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, pool, c, n, lens, window=window)
    assert torch.all(got[sum(n):] == 7.0)


# --- the bounds-checked build ---------------------------------------------
@pytest.fixture(scope="module")
def libs():
    from gemm_pq2_ternary_gb300 import _build, binding
    release = binding._lib
    debug = binding.load_library(_build.build(debug=True))
    yield binding, release, debug
    binding._lib = release
    debug.pq2_debug_shrink_bounds(0)


def _padded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((2 * PAD + n,), SENTINEL, dtype=dtype, device=DEV)
    return buf, buf[PAD:PAD + n].view(shape)


def _rope(pq2, D, rot):
    g = torch.Generator(device=DEV).manual_seed(D)
    table = torch.empty((64, rot // 2, 2), device=DEV)
    pq2.pq2_rope_table(table, 1e4)
    q = torch.randn((9, 3, D), generator=g, device=DEV)
    b, o = _padded((9, 3, D), torch.float16)
    pq2.pq2_rope(q, table, _dev(np.arange(9)), o)
    return [(b, o)]


def _append(pq2, D):
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn((5, 4, D), generator=g, device=DEV)
    nbytes = pq2.pq2_cache4_page_bytes(1, D, 16)
    pb, flat = _padded((1, nbytes), torch.uint8)
    qb, q = _padded((5, 2, D), torch.float16)
    table = torch.empty((64, D // 2, 2), device=DEV)
    pq2.pq2_rope_table(table, 1e4)
    # (the last token of the page, whose pair of values is the pool's last word)
    pq2.pq2_cache4_append(x[:, 2:3], x[:, 3:], flat.unflatten(1, (1, nbytes)), _dev([[0]]), _dev([0, 5]), _dev([16]),
                          q=x[:, :2], q_out=q, table=table)
    return [(pb, flat), (qb, q)]


def _read(pq2, D):
    c = Cache(pq2, 1, 2, 2, D, 16)
    c.fill([20])
    kb, k = _padded((20, 2, D), torch.float32)
    vb, v = _padded((20, 2, D), torch.float32)
    pq2.pq2_cache4_read(c.pool, c.dev, _dev([0, 20]), _dev([20]), k, v)
    return [(kb, k), (vb, v)]


def _attention(pq2, Hq, H, D, n, ln):
    c = Cache(pq2, 1, -(-ln // 64), H, D, 64)
    c.fill([ln])
    q = _q(n, Hq, D, "f16")
    b, o = _padded((n, Hq, D), torch.float16)
    _attend(pq2, c, q, [n], [ln], out=o)
    return [(b, o)]


CASES = {
    "rope_64": lambda p: _rope(p, 64, 64), "rope_any": lambda p: _rope(p, 80, 40), "append_64": lambda p: _append(p, 64),
    "append_256": lambda p: _append(p, 256), "read": lambda p: _read(p, 128),
    "few_rows": lambda p: _attention(p, 8, 1, 128, 1, 20), "few_rows_256": lambda p: _attention(p, 8, 1, 256, 1, 900),
    "many_rows": lambda p: _attention(p, 8, 1, 128, 64, 100), "many_rows_64": lambda p: _attention(p, 1, 1, 64, 400, 900),
    "many_rows_256": lambda p: _attention(p, 4, 1, 256, 64, 900),
}


def _run(pq2, lib, name):
    pq2._lib = lib
    outs = CASES[name](pq2)
    torch.cuda.synchronize()
    return outs


def _untouched(outs):
    return all(bool((b[:PAD] == SENTINEL).all()) and bool((b[PAD + o.numel():] == SENTINEL).all()) for b, o in outs)


@pytest.mark.parametrize("name", CASES)
def test_checked_build_matches_and_reports_nothing(libs, name):
    pq2, release, debug = libs
    try:
        want = _run(pq2, release, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        got = _run(pq2, debug, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    finally:
        pq2._lib = release
    assert all(torch.equal(w, g) for (_, w), (_, g) in zip(want, got))
    assert _untouched(want) and _untouched(got)


@pytest.mark.parametrize("name", CASES)
def test_checked_build_reports_a_store_outside(libs, name):
    pq2, release, debug = libs
    pq2._lib = debug
    try:
        debug.pq2_debug_shrink_bounds(1)
        outs = _run(pq2, debug, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_BOUNDS
    finally:
        debug.pq2_debug_shrink_bounds(0)
        pq2._lib = release
    assert _untouched(outs)


# --- the serving example ----------------------------------------------------
@pytest.mark.parametrize("q_heads,heads,dim,drafts", [(6, 2, 64, 3), (12, 2, 128, 0), (4, 1, 256, 9)])
def test_steps_of_the_serving_example(pq2, q_heads, heads, dim, drafts):
    import serving_step
    B = 3
    block = serving_step.Block(B * (drafts + 1), 512, 640, 1000, 2, 16, B)
    args = serving_step.random_step(block, drafts, 2)
    at = serving_step.Attention(block, q_heads, heads, dim, 40 * (drafts + 1), page=16)
    keep = torch.zeros(B, dtype=torch.int32, device=DEV)
    for step in range(4):
        r = at.step(args["r"] * (1 + step), args["row_start"], keep)
        assert torch.isfinite(r).all() and pq2.pq2_last_device_error() == pq2.PQ2_OK and int(at.info[1]) == 0
        lens = at.lens.cpu().numpy()
        assert np.array_equal(lens, keep.cpu().numpy() + drafts + 1)
        # the attention's rows against the definition on what the cache holds
        pages = at.pages[at.turn].cpu().numpy()
        want, tol = ref.attend(_np(at.q), at.pool.cpu().numpy(), pages, args["row_start"].cpu().numpy(), lens, 16, dim ** -0.5, 0)
        err = np.abs(at.a.double().cpu().numpy() - want)
        assert np.all(err <= tol + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
        accepted, _ = block.step(**{**args, "r": r})
        keep = keep + accepted + 1
