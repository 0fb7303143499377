"""GPU parity of the low-rank adapters (pq2_lora_add) against the float64
oracle.

Tolerance (u = 2^-24; tensor accumulation counted as truncating, 2 u an
addition).  v = A x: chains of 16 products of 16 terms, then fp32 sums over
K / 256 chains, 8 warps and 32 splits: n_v = 32 + K/256 + 40 additions, error
<= 2 u n_v sum |A x|.  v enters the second product to 2^-22 of the token's
largest |v| (fp16) or of itself (bf16).  That product adds 2 (3 for bf16)
terms of R ranks in instructions of 16: n_e = 3 R / 16 + 16, error <=
2 u n_e sum |B v|.  Scale and the final sum: 4 u; one rounding to y's type."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAD = 64
SENTINEL = 55.0


def _np(t):
    return t.double().cpu().numpy()


def _problem(M, K, N, R, L, ty, y_type, seed, ids="mixed", ranks=True, scales=True, ld_x=None,
             ld_y=None, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    p = {"M": M, "K": K, "N": N, "R": R, "L": L, "ty": ty, "y_type": y_type}
    x = torch.randn((M, K if ld_x is None else ld_x), generator=g, device=DEV)
    p["x"] = x.to(T[ty])[:, :K]
    p["A"] = (torch.randn((L, R, K), generator=g, device=DEV) * K ** -0.5).to(T[ty])
    p["B"] = (torch.randn((L, N, R), generator=g, device=DEV) * 0.3).to(T[ty])
    if isinstance(ids, str):
        ids = torch.randint(-1, L, (M,), generator=h) if ids == "mixed" else torch.sort(
            torch.randint(0, L, (M,), generator=h)).values
    p["ids"] = torch.as_tensor(ids, dtype=torch.int32).to(DEV)
    p["ranks"] = p["scales"] = None
    if ranks:
        rk = torch.randint(0, R + 1, (L,), generator=h, dtype=torch.int32)
        rk[0] = R
        p["ranks"] = rk.to(DEV)
        for l in range(L):      # what lies past an adapter's rank may be anything
            p["A"][l, int(rk[l]):] = float("nan")
            p["B"][l, :, int(rk[l]):] = float("inf")
    if scales:
        p["scales"] = (torch.rand(L, generator=g, device=DEV) * 4 - 2)
    ld = N if ld_y is None else ld_y
    p["y"] = torch.randn((M, ld), generator=g, device=DEV).to(T[y_type])[:, :N]
    p["buf"] = torch.full((2 * PAD + offset + M * ld,), SENTINEL, dtype=T[y_type], device=DEV)
    p["out"] = p["buf"][PAD + offset:PAD + offset + M * ld].view(M, ld)[:, :N]
    return p


def _call(pq2, p, out=None, y=None, stream=None):
    ws = pq2.alloc_lora_workspace(p["M"], p["N"], p["K"], p["L"], p["R"])
    ws.fill_(0xA5)              # the workspace comes with any content
    pq2.pq2_lora_add(p["x"], p["A"], p["B"], p["ids"], p["y"] if y is None else y,
                     p["out"] if out is None else out, ws, ranks=p["ranks"], scales=p["scales"],
                     stream=stream)


def _tolerance(p, want, bounds):
    bv, bs, bm = bounds
    u, K, R = step.U32, p["K"], p["R"]
    t = 2 * u * (32 + K / 256 + 40) * bv + 2 * u * (3 * R / 16 + 16) * bm
    t += 2.0 ** -22 * bs + 4 * u * (np.abs(want) + bm)
    return t + step.UNIT[p["y_type"]] * np.abs(want) * 1.01


def _check(pq2, p, out):
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    rk = None if p["ranks"] is None else p["ranks"].cpu().numpy()
    sc = None if p["scales"] is None else p["scales"].cpu().numpy()
    # the unused ranks are sliced off before any arithmetic
    want, bounds = step.lora(_np(p["x"]), _np(p["A"]), _np(p["B"]), p["ids"].cpu().numpy(), rk, sc,
                             _np(p["y"]))
    got = _np(out)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    tol = _tolerance(p, want, bounds)
    assert np.all(err <= tol), f"max {(err - tol).max()} over, at {np.argmax(err - tol)}"
    none = (p["ids"] < 0).cpu().numpy()
    assert np.array_equal(got[none], _np(p["y"])[none])
    mask = torch.ones_like(p["buf"], dtype=torch.bool)
    mask.as_strided(p["out"].shape, p["out"].stride(), p["out"].storage_offset()).fill_(False)
    assert bool((p["buf"][mask].float() == SENTINEL).all()), "wrote outside y"


SHAPES = [
    # M, K, N, R, L, x type, y type, kwargs
    (1, 5120, 1000, 16, 4, "f16", "f32", {}),
    (1, 640, 1001, 8, 1, "bf16", "bf16", dict(ranks=False)),
    (2, 128, 5, 8, 3, "f16", "f32", {}),
    (8, 8, 3, 8, 2, "bf16", "f32", {}),
    (7, 1664, 333, 64, 2, "f16", "f32", dict(ld_x=1672, ld_y=336)),
    (9, 1024, 256, 128, 9, "bf16", "f32", {}),
    (32, 640, 300, 256, 5, "f16", "bf16", {}),
    (32, 640, 300, 256, 40, "bf16", "f32", dict(scales=False)),
    (17, 1000, 129, 24, 17, "f16", "f32", dict(ld_y=131)),
    (33, 640, 300, 16, 3, "f16", "f32", {}),
    (48, 1664, 513, 32, 32, "bf16", "f32", {}),
    (65, 640, 261, 72, 2, "f16", "bf16", dict(ranks=False)),
    (130, 17408, 128, 64, 3, "f16", "f32", {}),
    (200, 384, 1002, 256, 4, "bf16", "bf16", dict(ld_y=1003, offset=1)),
    (333, 1024, 640, 128, 200, "f16", "f32", {}),
    (700, 256, 515, 8, 2, "bf16", "f32", dict(ids="runs", offset=3)),
    (1500, 512, 384, 40, 700, "f16", "f32", {}),
    (2100, 128, 130, 16, 5, "f16", "f32", dict(ids="runs")),
    (128, 640, 301, 16, 3, "f16", "f32", {}),
    (128, 128, 40, 8, 128, "f16", "f32", {}),
    (100, 1664, 260, 40, 2, "bf16", "f32", dict(ids="runs")),
    (129, 640, 300, 16, 3, "f16", "f32", {}),
    (150, 8, 40, 16, 3, "f16", "f32", {}),
    (150, 24, 260, 40, 3, "bf16", "f32", {}),
    (4097, 64, 36, 8, 3, "f16", "f32", {}),
    (9000, 64, 36, 8, 1000, "f16", "f32", {}),
    # whole 16-byte rows of y and more than 128 tokens: the copy ring
    (40, 5120, 5120, 32, 30, "bf16", "f32", {}),
    (140, 5120, 5120, 32, 30, "bf16", "f32", {}),
    (200, 2048, 1000, 256, 4, "bf16", "bf16", {}),
    (197, 640, 2056, 136, 3, "f16", "bf16", dict(ld_y=2064)),
    (197, 640, 2052, 136, 3, "f16", "f32", dict(ld_y=2060)),
    (300, 72, 4, 8, 2, "f16", "f32", {}),
    (1025, 1000, 1028, 48, 2, "bf16", "f32", dict(ranks=False, ids="runs")),
    (129, 6144, 700, 64, 1, "f16", "f32", dict(scales=False)),
    (4000, 256, 264, 128, 64, "f16", "bf16", {}),
    # clusters of 16 with each count of ranks
    (140, 17408, 130, 256, 2, "f16", "f32", {}),
    (131, 17400, 260, 136, 3, "bf16", "f32", dict(ids="runs")),
    (135, 17408, 132, 96, 2, "bf16", "f32", {}),
    (200, 17408, 132, 24, 2, "f16", "f32", {}),
    # few tokens an adapter
    (70, 64, 5120, 256, 40, "f16", "f32", {}),
    (127, 64, 5120, 256, 50, "f16", "f32", {}),
    (90, 64, 5124, 256, 37, "bf16", "bf16", {}),
    (300, 512, 1028, 128, 40, "f16", "f32", {}),
    (300, 256, 1025, 24, 60, "bf16", "f32", dict(ld_y=1027)),
    (500, 256, 2052, 192, 100, "f16", "f32", {}),
    (640, 256, 1032, 64, 80, "bf16", "bf16", dict(ids="runs")),
    (600, 256, 2600, 40, 90, "bf16", "f32", dict(ids="runs")),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(v) for v in s[:7]))
def test_lora_add(shape):
    from gemm_pq2_ternary_gb300 import binding as pq2
    M, K, N, R, L, ty, y_type, kw = shape
    p = _problem(M, K, N, R, L, ty, y_type, seed=M + K, **kw)
    _call(pq2, p)
    _check(pq2, p, p["out"])


@pytest.mark.parametrize("N", [301, 516])
@pytest.mark.parametrize("M", [1, 20, 64, 400])
def test_in_place_equals_out_of_place(M, N):
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(M, 640, N, 24, 5, "f16", "f32", seed=M)
    _call(pq2, p)
    y = p["y"].clone()
    _call(pq2, p, out=y, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, p["out"])


@pytest.mark.parametrize("L", [1, 31, 33, 200, 1023, 1100, 3000])
def test_in_place_with_any_number_of_adapters(L):
    # in place, expand's items end where the tokens without an adapter begin:
    # a count that the plan takes from that bin's own thread, in another warp
    # than the last one's for some of these L
    from gemm_pq2_ternary_gb300 import binding as pq2
    for M in (400, 2000):
        ids = [-1 if m % 7 == 3 else m * 5 % L for m in range(M)]
        p = _problem(M, 64, 260, 8, L, "f16", "f32", seed=M + L, ids=ids)
        _call(pq2, p)
        y = p["y"].clone()
        _call(pq2, p, out=y, y=y)
        _check(pq2, p, y)
        assert torch.equal(y, p["out"])


@pytest.mark.parametrize("N", [77, 160])
@pytest.mark.parametrize("M", [1, 31, 32, 33, 128, 129, 300])
def test_a_batch_without_adapters_is_a_copy(M, N):
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(M, 256, N, 8, 2, "f16", "f32", seed=1, ids=[-1] * M)
    p["y"][0, 0] = float("inf")
    _call(pq2, p)
    torch.cuda.synchronize()
    assert torch.equal(p["out"], p["y"])


@pytest.mark.parametrize("N", [77, 160])
@pytest.mark.parametrize("M", [3, 90, 200])
def test_every_rank_zero_is_a_copy(M, N):
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(M, 256, N, 8, 2, "bf16", "bf16", seed=1, ids=[0] * M)
    p["ranks"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    _call(pq2, p)
    torch.cuda.synchronize()
    assert torch.equal(p["out"], p["y"])


@pytest.mark.parametrize("M", [5, 100, 300])
def test_an_id_past_the_adapters_is_reported_and_passes_through(M):
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(M, 256, 64, 8, 2, "f16", "f32", seed=2, ids=[m % 3 for m in range(M)])
    _call(pq2, p)
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    assert torch.equal(p["out"][2::3], p["y"][2::3])
    p["ids"][2::3] = -1
    _check(pq2, p, p["out"])


@pytest.mark.parametrize("M", [8, 32, 64, 1000])
def test_the_same_bits_whatever_the_token_order(M):
    # a token's result depends on its adapter and its x alone; only the
    # number of tokens, which sizes the K splits, is the same here
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(M, 640, 200, 24, 3, "f16", "f32", seed=9)
    _call(pq2, p)
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(0)).to(DEV)
    q = dict(p, x=p["x"][perm].contiguous(), ids=p["ids"][perm].contiguous(),
             y=p["y"][perm].contiguous(), out=torch.empty_like(p["out"]))
    _call(pq2, q)
    torch.cuda.synchronize()
    assert torch.equal(q["out"], p["out"][perm])


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 20])
def test_small_and_large_intermediates(ty, scale):
    # v far outside fp16's range of 16-bit terms: the token's power of two
    from gemm_pq2_ternary_gb300 import binding as pq2
    for M in (2, 70, 140):
        p = _problem(M, 512, 96, 16, 2, ty, "f32", seed=4, ranks=False)
        p["A"] = (p["A"].float() * (scale if ty == "bf16" else min(scale, 2.0 ** 12))).to(T[ty])
        if ty == "f16" and scale > 1:
            p["x"] = (p["x"].float() * 2.0 ** 8).to(T[ty])
        p["y"].zero_()
        _call(pq2, p)
        _check(pq2, p, p["out"])


def test_on_another_stream_after_a_producer():
    from gemm_pq2_ternary_gb300 import binding as pq2
    for M in (4, 100, 228):
        p = _problem(M, 640, 256, 16, 3, "f16", "f32", seed=8)
        _call(pq2, p)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        out = torch.empty_like(p["out"])
        with torch.cuda.stream(s):
            y = p["y"] * 1.0
            q = dict(p, x=p["x"] * 1)
            _call(pq2, q, out=out, y=y)
        torch.cuda.synchronize()
        assert torch.equal(out, p["out"])


def test_repeated_calls_give_the_same_bits():
    from gemm_pq2_ternary_gb300 import binding as pq2
    for M in (16, 500):
        p = _problem(M, 5120, 256, 32, 4, "f16", "f32", seed=3)
        outs = [torch.empty_like(p["out"]) for _ in range(10)]
        for o in outs:
            _call(pq2, p, out=o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_the_copy_ring_reports_a_stage_that_never_comes():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(200, 640, 2048, 32, 3, "f16", "f32", seed=21)
    try:
        pq2.pq2_debug_set_wait_limit_ns(20_000_000)
        pq2.pq2_debug_skip_stage(0)
        _call(pq2, p)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_TIMEOUT
    finally:
        pq2.pq2_debug_skip_stage(-1)
        pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
    _call(pq2, p)
    _check(pq2, p, p["out"])


def test_a_workspace_for_many_tokens_serves_fewer():
    from gemm_pq2_ternary_gb300 import binding as pq2
    K, N, R, L = 5120, 640, 32, 3
    ws = pq2.alloc_lora_workspace(500, N, K, L, R)
    for M in (500, 129, 128, 17, 1):
        p = _problem(M, K, N, R, L, "f16", "f32", seed=M)
        pq2.pq2_lora_add(p["x"], p["A"], p["B"], p["ids"], p["y"], p["out"], ws,
                         ranks=p["ranks"], scales=p["scales"])
        _check(pq2, p, p["out"])


def test_offsets_past_32_bits():
    # adapter 9 of a stack with more than 2^31 elements
    from gemm_pq2_ternary_gb300 import binding as pq2
    L, R, K, N = 10, 64, 8, (1 << 22) + 3
    M = 2
    B = torch.zeros((L, N, R), dtype=torch.float16, device=DEV)
    assert B.numel() > 1 << 31
    A = torch.zeros((L, R, K), dtype=torch.float16, device=DEV)
    A[9, 0, 0] = 1.0
    B[9, N - 1, 0] = 2.0
    x = torch.ones((M, K), dtype=torch.float16, device=DEV)
    y = torch.zeros((M, N), device=DEV)
    ids = torch.tensor([9, -1], dtype=torch.int32, device=DEV)
    pq2.pq2_lora_add(x, A, B, ids, y, y, pq2.alloc_lora_workspace(M, N, K, L, R))
    torch.cuda.synchronize()
    assert y[0, N - 1].item() == 2.0 and int(torch.count_nonzero(y)) == 1


def test_binding_refuses():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem(4, 64, 32, 8, 2, "f16", "f32", seed=1)
    ws = pq2.alloc_lora_workspace(4, 32, 64, 2, 8)
    good = [p["x"], p["A"], p["B"], p["ids"], p["y"], p["out"], ws]

    def bad(i, v, match):
        a = list(good)
        a[i] = v
        with pytest.raises((ValueError, pq2.PQ2Error), match=match):
            pq2.pq2_lora_add(*a)

    bad(1, p["A"][:, :, :32].contiguous(), "shapes")
    bad(1, p["A"].bfloat16(), "x's type")
    bad(3, p["ids"].long(), "int32")
    bad(4, p["y"][:, :31], "y_in")
    bad(5, p["out"].bfloat16(), "type")
    bad(6, ws[:16], "workspace")
    bad(6, None, "workspace")
    with pytest.raises(pq2.PQ2Error, match="shape"):
        pq2.alloc_lora_workspace(4, 32, 64, 2, 12)


@pytest.mark.parametrize("L", [12000, 14512, 16384])
@pytest.mark.parametrize("M", [200, 3000])
def test_as_many_adapters_as_are_allowed(M, L):
    from gemm_pq2_ternary_gb300 import binding as pq2
    assert L <= pq2.PQ2_LORA_MAX_L
    ids = [-1 if m % 11 == 5 else (m * 977 + L - 1) % L for m in range(M)]
    p = _problem(M, 64, 36, 8, L, "f16", "f32", seed=L, ids=ids, ranks=False)
    p["ranks"] = (torch.arange(L, device=DEV) * 5 % 9).to(torch.int32)
    _call(pq2, p)
    _check(pq2, p, p["out"])
    y = p["y"].clone()
    _call(pq2, p, out=y, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, p["out"])


# (M, K, N, R, L, y type, kernel whose stage is withheld: the other has none
# of that number)
STAGES = [
    (200, 640, 64, 32, 3, "f32", "shrink, mma.sync"),
    (200, 1280, 64, 64, 3, "f32", "shrink, tcgen05"),
    (200, 1280, 64, 200, 3, "f32", "shrink, tcgen05, two accumulators"),
    (200, 64, 10240, 64, 3, "f32", "expand, tcgen05"),
    (200, 64, 10241, 64, 3, "f32", "expand, tcgen05, y by values"),
    (200, 64, 5120, 16, 20, "f32", "expand, tcgen05, tiles of 16"),
    (200, 64, 5121, 16, 20, "f32", "expand, tcgen05, tiles of 16, y by values"),
    (200, 64, 10240, 64, 3, "bf16", "expand, mma.sync, bf16 y"),
    (200, 64, 5120, 256, 3, "f32", "expand, mma.sync"),
    (200, 64, 5121, 256, 3, "f32", "expand, mma.sync, y by values"),
]


@pytest.mark.parametrize("case", STAGES, ids=lambda c: c[-1])
def test_every_ring_reports_a_stage_that_never_comes(case):
    from gemm_pq2_ternary_gb300 import binding as pq2
    M, K, N, R, L, y_type, _ = case
    p = _problem(M, K, N, R, L, "f16", y_type, seed=R, ranks=False)
    _call(pq2, p)
    _check(pq2, p, p["out"])
    want = p["out"].clone()
    for stage in (1, 2):
        try:
            pq2.pq2_debug_set_wait_limit_ns(20_000_000)
            pq2.pq2_debug_skip_stage(stage)
            _call(pq2, p)
            assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_TIMEOUT
        finally:
            pq2.pq2_debug_skip_stage(-1)
            pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
        _call(pq2, p)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        assert torch.equal(p["out"], want)
