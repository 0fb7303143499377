"""The steps around a projection in the bounds-checked build: the same bits as
the normal build and no report; and, with the last element of every checked
buffer treated as outside, a report, a skipped store and nothing written
around the outputs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAD = 64
SENTINEL = 123.0


@pytest.fixture(scope="module")
def libs():
    from gemm_pq2_ternary_gb300 import _build, binding
    release = binding._lib
    debug = binding.load_library(_build.build(debug=True))
    yield binding, release, debug
    binding._lib = release
    debug.pq2_debug_shrink_bounds(0)


def _out(M, N, dtype=torch.float32):
    buf = torch.full((2 * PAD + M * N,), SENTINEL, dtype=dtype, device=DEV)
    return buf, buf[PAD:PAD + M * N].view(M, N)


def _norm(pq2, M, H, before=False, gate=True):
    g = torch.Generator(device=DEV).manual_seed(M + H)
    r = torch.randn((M, H), generator=g, device=DEV)
    y = torch.randn((M, H), generator=g, device=DEV)
    xb, x = _out(M, H, torch.float16)
    if before:
        pq2.pq2_rmsnorm(r, None, x)
        return [(xb, x)]
    rb, ro = _out(M, H)
    pq2.pq2_norm_residual(y, r, ro, gate=y if gate else None, x=x, flags=pq2.PQ2_GATE_SIGMOID if gate else 0)
    return [(rb, ro), (xb, x)]


def _lora(pq2, M, N, R, y_type=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(M + N)
    L, K = 3, 640
    x = torch.randn((M, K), generator=g, device=DEV).half()
    A = (torch.randn((L, R, K), generator=g, device=DEV) * 0.04).half()
    B = (torch.randn((L, N, R), generator=g, device=DEV) * 0.2).half()
    ids = (torch.arange(M, device=DEV) % L).to(torch.int32)
    y = torch.randn((M, N), generator=g, device=DEV).to(y_type)
    b, o = _out(M, N, y_type)
    ws = pq2.alloc_lora_workspace(M, N, K, L, R)
    ws.zero_()
    pq2.pq2_lora_add(x, A, B, ids, y, o, ws)
    return [(b, o)]


def _verify(pq2, greedy):
    rng = np.random.default_rng(3)
    lens, V = [3, 1, 4], 5003
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(start[-1])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    ab, acc = _out(1, len(lens), torch.int32)
    tb, tok = _out(1, rows, torch.int32)
    ws = pq2.alloc_verify_workspace(len(lens), rows, V)
    ws.zero_()
    pq2.pq2_verify_drafts(t(rng.standard_normal((rows, V)).astype(np.float32)), t(start),
                          t(rng.integers(0, V, rows).astype(np.int32)), None,
                          t(rng.random(rows).astype(np.float32)),
                          t(rng.exponential(size=(len(lens), V)).astype(np.float32)),
                          t(np.full(len(lens), 0.0 if greedy else 0.7, np.float32)), acc.view(-1),
                          tok.view(-1), ws)
    return [(ab, acc), (tb, tok)]


CASES = {
    "norm_warp_rows": lambda p: _norm(p, 19, 256), "norm_vectors": lambda p: _norm(p, 5, 1024),
    "norm_ring": lambda p: _norm(p, 700, 1032), "norm_ring_no_gate": lambda p: _norm(p, 650, 2048, gate=False),
    "norm_odd": lambda p: _norm(p, 5, 777), "norm_odd_warp_rows": lambda p: _norm(p, 5, 77),
    "norm_wide": lambda p: _norm(p, 3, 9001), "before_vectors": lambda p: _norm(p, 4, 5120, before=True),
    "before_ring": lambda p: _norm(p, 640, 1024, before=True), "before_wide": lambda p: _norm(p, 2, 12000, before=True),
    "lora_one": lambda p: _lora(p, 1, 300, 16), "lora_few": lambda p: _lora(p, 60, 301, 40),
    "lora_few_bf16": lambda p: _lora(p, 60, 301, 16, torch.bfloat16),
    "lora_ring": lambda p: _lora(p, 150, 300, 16), "lora_ring_64": lambda p: _lora(p, 150, 300, 256),
    "lora_ring_values": lambda p: _lora(p, 150, 301, 24), "lora_ring_bf16": lambda p: _lora(p, 150, 304, 24, torch.bfloat16),
    "lora_tiles_bf16": lambda p: _lora(p, 150, 301, 24, torch.bfloat16),
    "verify": lambda p: _verify(p, False), "verify_greedy": lambda p: _verify(p, True),
}


def _run(pq2, lib, name):
    pq2._lib = lib
    outs = CASES[name](pq2)
    torch.cuda.synchronize()
    return outs


def _guards(outs):
    return all(bool((b[:PAD] == SENTINEL).all()) and bool((b[PAD + o.numel():] == SENTINEL).all())
               for b, o in outs)


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
    assert _guards(want) and _guards(got)


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
    assert _guards(outs)
    assert all(b[PAD + o.numel() - 1].item() == SENTINEL for b, o in outs)
