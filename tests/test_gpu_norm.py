"""GPU parity of the norms around a block (pq2_rmsnorm, pq2_norm_residual)
against the float64 oracle.

Tolerance, from the kernel's operations (all fp32, u = 2^-24).  A sum of
squares adds at most 16 values a thread (48 for the widest rows), 5 shuffle
steps and 32 warp sums, all positive: relative error below 96 u, half of that
in the root; rsqrt (2 ulp) and the products add less than 12 u.  The gate's
exponential is within 2 + 1.2 |g| ulp, |g| < 8: 24 u.  So
  |add| error   <= 96 u |add|
  r' error      <= 96 u |add| + 2 u (|r| + |add|) + one rounding to r's type
  x' error      <= 64 u |x'| + (|w| / rms) (r' error before its rounding)
                   + one rounding to x's type."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
PAD = 64
SENTINEL = 77.0


def _np(t):
    return t.double().cpu().numpy()


def _rows(gen, M, H, dtype, ld=None, scale=1.0, offset=0):
    """[M, H] with row stride ld inside a larger buffer of sentinels (offset
    in elements shifts the alignment) -> (buffer, view)."""
    ld = H if ld is None else ld
    buf = torch.full((2 * PAD + offset + M * ld,), SENTINEL, dtype=T[dtype], device=DEV)
    view = buf[PAD + offset:PAD + offset + M * ld].view(M, ld)[:, :H]
    if scale:
        view.copy_((torch.randn((M, H), generator=gen, device=DEV) * scale).to(T[dtype]))
    return buf, view


def _outside_untouched(buf, view):
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[mask].float() == SENTINEL).all())


def _round(v, dtype):
    return step.UNIT[dtype] * np.abs(v) * 1.01 + step.TINY[dtype]


# (M, H, y, r, weights, gate, x, act, post, next, ld_extra, offset)
CASES = [
    (1, 5120, "f32", "bf16", "f32", None, "f16", None, True, True, 0, 0),
    (3, 5120, "f32", "f32", "bf16", "bf16", "bf16", "sigmoid", True, True, 5120, 0),
    (700, 1024, "f32", "f16", "f32", "vector", "f16", None, True, True, 0, 0),
    (5, 6144, "bf16", "bf16", "f16", "f16", "f32", "silu", True, True, 8, 0),
    (2, 8192, "f32", "f32", "f32", "f32", "f16", "sigmoid", False, True, 0, 0),
    (33, 512, "f32", "bf16", "f32", "bf16", "f16", "silu", True, True, 0, 0),     # a warp a row
    (2000, 128, "f16", "f16", "f32", None, "bf16", None, True, True, 0, 0),
    (9, 24, "f32", "f32", "f32", None, "f16", None, True, True, 8, 0),
    (7, 1001, "f32", "bf16", "f32", "bf16", "f16", "sigmoid", True, True, 0, 0),  # odd width
    (4, 1024, "f32", "f16", "f32", "f16", "f16", "silu", True, True, 3, 0),       # odd stride
    (4, 1024, "f32", "f16", "f32", "f16", "f16", None, True, True, 0, 1),         # odd start
    (11, 1, "f32", "f32", "f32", None, "f32", None, True, True, 0, 0),
    (3, 200, "f32", "f32", None, None, "f16", None, False, True, 0, 0),
    (2, 4097, "bf16", "f16", "f16", "vector", "bf16", "silu", True, True, 0, 0),  # shared memory
    (3, 20000, "f32", "bf16", "bf16", "bf16", "f16", "sigmoid", True, True, 0, 0),
    (1, 49152, "f32", "f32", "f32", None, "f16", None, True, True, 0, 0),
    (6, 5120, "f32", "bf16", "f32", None, None, None, True, False, 0, 0),         # no next norm
    (6, 777, "f32", "bf16", "f32", "f32", None, "silu", False, False, 0, 0),
    (300, 2560, "f32", "f32", "f32", None, None, None, False, False, 0, 0),
    # many rows: the copy ring (a few rows per SM and more)
    (1300, 5120, "f32", "bf16", "f32", "bf16", "f16", "sigmoid", True, True, 5120, 0),
    (2048, 520, "f32", "f32", "bf16", "vector", "bf16", "silu", True, True, 0, 0),
    (700, 8192, "f32", "bf16", "f32", None, "f16", None, True, True, 0, 0),
    (700, 8192, "f32", "f32", "f32", "f32", "f16", "silu", True, True, 0, 0),  # too wide for it
    (901, 1024, "bf16", "f16", None, "f16", None, "sigmoid", True, False, 8, 0),
    (613, 6144, "f32", "f32", "f32", None, "f16", None, False, True, 0, 0),
    (777, 2048, "f16", "f32", "f32", "f32", None, None, False, False, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[2]}-{c[3]}-{c[5]}-{c[6]}")
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_residual(case, in_place):
    from gemm_pq2_ternary_gb300 import binding as pq2
    M, H, ty, tr, tw, gate, tx, act, post, nxt, extra, offset = case
    gen = torch.Generator(device=DEV).manual_seed(M * 100003 + H)
    ld = H + extra
    _, y = _rows(gen, M, H, ty, ld, 3.0, offset)
    rbuf, r = _rows(gen, M, H, tr, ld, 2.0, offset)
    w_post = w_next = None
    if tw:
        w_post = (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(T[tw])
        w_next = (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(T[tw])
    g = None
    if gate == "vector":
        g = torch.randn(H, generator=gen, device=DEV).clamp(-7, 7)
    elif gate:
        _, g = _rows(gen, M, H, gate, ld, 1.5, offset)
        g.clamp_(-7, 7)
    obuf, out = (rbuf, r) if in_place else _rows(gen, M, H, tr, ld, 0, offset)
    xbuf, x = _rows(gen, M, H, tx, ld, 0, offset) if nxt else (None, None)
    alpha = 0.6
    want_r, want_x, add = step.norm_residual(
        _np(y), _np(r), None if w_post is None else _np(w_post), None if g is None else _np(g), act,
        None if w_next is None else _np(w_next), EPS, alpha, post)
    r0 = _np(r)
    flags = 0 if post else pq2.PQ2_NORM_NO_POST
    flags |= {"sigmoid": pq2.PQ2_GATE_SIGMOID, "silu": pq2.PQ2_GATE_SILU}.get(act, 0)
    pq2.pq2_norm_residual(y, r, out, w_post=w_post, gate=g, w_next=w_next, x=x, eps=EPS, alpha=alpha,
                          flags=flags)
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    u = step.U32
    err_r = 96 * u * add + 2 * u * (np.abs(r0) + add)
    assert np.all(np.abs(_np(out) - want_r) <= err_r + _round(want_r, tr))
    assert _outside_untouched(obuf, out)
    if nxt:
        rms = np.sqrt((want_r ** 2).mean(axis=1, keepdims=True) + EPS)
        w = 1.0 if w_next is None else np.abs(_np(w_next))
        err_x = 64 * u * np.abs(want_x) + w / rms * err_r
        # the row's own rms moves with r': a second-order share of err_r
        err_x += np.abs(want_x) * np.sqrt((err_r ** 2).mean(axis=1, keepdims=True)) / rms
        assert np.all(np.abs(_np(x) - want_x) <= err_x + _round(want_x, tx))
        assert _outside_untouched(xbuf, x)


@pytest.mark.parametrize("M,H,tr,tx,tw,extra,offset", [
    (1, 5120, "bf16", "f16", "f32", 0, 0), (4096, 64, "f32", "f16", "f32", 0, 0),
    (65, 1001, "f16", "bf16", "bf16", 0, 0), (5, 6144, "f32", "f16", None, 16, 0),
    (3, 9000, "bf16", "f32", "f32", 0, 0), (40, 300, "f16", "f16", "f16", 0, 1),
    (500, 8, "f32", "bf16", "f32", 0, 0), (1999, 5120, "bf16", "f16", "f32", 0, 0),
    (3000, 600, "f32", "bf16", "f16", 8, 0)])
def test_rmsnorm(M, H, tr, tx, tw, extra, offset):
    from gemm_pq2_ternary_gb300 import binding as pq2
    gen = torch.Generator(device=DEV).manual_seed(H)
    _, r = _rows(gen, M, H, tr, H + extra, 2.0, offset)
    w = None if tw is None else (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(T[tw])
    xbuf, x = _rows(gen, M, H, tx, H + extra, 0, offset)
    pq2.pq2_rmsnorm(r, w, x, EPS)
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    want = step.rmsnorm(_np(r), None if w is None else _np(w), EPS)
    assert np.all(np.abs(_np(x) - want) <= 64 * step.U32 * np.abs(want) + _round(want, tx))
    assert _outside_untouched(xbuf, x)


def test_unit_offset_and_static_weights_give_the_same_rows():
    from gemm_pq2_ternary_gb300 import binding as pq2
    gen = torch.Generator(device=DEV).manual_seed(5)
    r = torch.randn((17, 1024), generator=gen, device=DEV)
    # 1 + w exact in fp32 for w a multiple of 2^-10
    w = torch.randint(-512, 512, (1024,), generator=gen, device=DEV).float() / 1024
    x0, x1, x2 = (torch.empty((17, 1024), dtype=torch.float16, device=DEV) for _ in range(3))
    pq2.pq2_rmsnorm(r, w + 1, x0, EPS)
    pq2.pq2_rmsnorm(r, w, x1, EPS, pq2.PQ2_NORM_UNIT_OFFSET)
    pq2.pq2_rmsnorm(r, w + 1, x2, EPS, pq2.PQ2_WEIGHTS_STATIC)
    torch.cuda.synchronize()
    assert torch.equal(x0, x1) and torch.equal(x0, x2)


def test_a_row_of_zeros_and_values_past_fp16():
    from gemm_pq2_ternary_gb300 import binding as pq2
    r = torch.zeros((2, 256), device=DEV)
    r[1, 0] = 1e30                          # its square overflows no sum that matters
    r[1, 0] = 3e4
    w = torch.full((256,), 2e4, device=DEV)
    x = torch.empty((2, 256), dtype=torch.float16, device=DEV)
    pq2.pq2_rmsnorm(r, w, x, EPS)
    torch.cuda.synchronize()
    assert torch.all(x[0] == 0)             # eps keeps the quotient finite
    assert torch.isinf(x[1, 0]) and torch.all(x[1, 1:] == 0)


def test_same_bits_on_another_stream_and_after_a_producer():
    from gemm_pq2_ternary_gb300 import binding as pq2
    gen = torch.Generator(device=DEV).manual_seed(6)
    y = torch.randn((64, 5120), generator=gen, device=DEV)
    r = torch.randn((64, 5120), generator=gen, device=DEV).bfloat16()
    w = torch.ones(5120, device=DEV)
    outs = []
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        x = torch.empty((64, 5120), dtype=torch.float16, device=DEV)
        o = torch.empty_like(r)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            y2 = y * 1.0                     # produced on the same stream just before
            pq2.pq2_norm_residual(y2, r, o, w_post=w, w_next=w, x=x, eps=EPS)
        torch.cuda.synchronize()
        outs.append((o, x))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_the_copy_ring_reports_a_stage_that_never_comes():
    # each CTA's producer withholds a row; the rows' groups give up after the
    # limit and the host reads the timeout; the next call is right
    from gemm_pq2_ternary_gb300 import binding as pq2
    gen = torch.Generator(device=DEV).manual_seed(7)
    for M, H in ((1300, 1024), (2000, 5120)):
        r = torch.randn((M, H), generator=gen, device=DEV)
        x = torch.empty((M, H), dtype=torch.float16, device=DEV)
        try:
            pq2.pq2_debug_set_wait_limit_ns(20_000_000)
            pq2.pq2_debug_skip_stage(1)
            pq2.pq2_norm_residual(r, r, torch.empty_like(r), x=x, eps=EPS)
            assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_TIMEOUT
        finally:
            pq2.pq2_debug_skip_stage(-1)
            pq2.pq2_debug_set_wait_limit_ns(2_000_000_000)
        pq2.pq2_rmsnorm(r, None, x, EPS)
        torch.cuda.synchronize()
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        want = step.rmsnorm(_np(r), None, EPS)
        assert np.all(np.abs(_np(x) - want) <= 64 * step.U32 * np.abs(want) + _round(want, "f16"))


def test_binding_refuses():
    from gemm_pq2_ternary_gb300 import binding as pq2
    r = torch.zeros((4, 64), device=DEV)
    x = torch.zeros((4, 64), dtype=torch.float16, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        pq2.pq2_rmsnorm(r, None, x[:3])
    with pytest.raises(ValueError, match="contiguous"):
        pq2.pq2_rmsnorm(r, None, torch.zeros((64, 4), dtype=torch.float16, device=DEV).T)
    with pytest.raises(ValueError, match="w: expected"):
        pq2.pq2_rmsnorm(r, torch.zeros(63, device=DEV), x)
    with pytest.raises(ValueError, match="expected float32"):
        pq2.pq2_rmsnorm(r.int(), None, x)
    with pytest.raises(ValueError, match="r_out"):
        pq2.pq2_norm_residual(r, r, x)
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_rmsnorm(r, None, x, flags=1 << 20)


# widths a few columns past what whole warps of 16 values a thread hold
@pytest.mark.parametrize("H", [520, 1032, 2056, 5128, 7688])
@pytest.mark.parametrize("M", [1, 6, 70])
def test_widths_just_past_whole_warps(M, H):
    test_norm_residual((M, H, "f32", "bf16", "f32", "bf16", "f16", "sigmoid", True, True, 0, 0), False)
    test_norm_residual((M, H, "f32", "f32", "f32", None, "f16", None, False, True, 8, 0), False)
    test_rmsnorm(M, H, "f32", "f16", "f32", 0, 0)


def test_a_width_just_past_whole_warps_that_is_too_wide_for_the_ring():
    test_norm_residual((700, 7688, "f32", "f32", "f32", "f32", "f16", "silu", True, True, 0, 0), False)


@pytest.mark.parametrize("M,H", [(5, 1024), (700, 1024), (700, 5120)])
def test_static_weights_do_not_cover_the_gate(M, H):
    # a gate vector that a projection writes directly before, a new one each
    # call: the flag lets the norm weights be read early, the gate not
    from gemm_pq2_ternary_gb300 import binding as pq2
    gen = torch.Generator(device=DEV).manual_seed(H)
    y = torch.randn((M, H), generator=gen, device=DEV)
    r = torch.randn((M, H), generator=gen, device=DEV)
    w = 1 + 0.2 * torch.randn(H, generator=gen, device=DEV)
    wg = (torch.randn((H, 4096), generator=gen, device=DEV) / 64).bfloat16()
    xg = torch.randn((20, 1, 4096), generator=gen, device=DEV).bfloat16()
    gate = torch.full((1, H), 50.0, dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty_like(r) for _ in range(20)]
    big = torch.zeros(1 << 26, device=DEV)
    torch.cuda.synchronize()
    for x, out in zip(xg, outs):
        big.add_(1)              # both calls are queued before the first starts
        pq2.pq2_gemm_bf16_splitk(x, wg, gate)
        pq2.pq2_norm_residual(y, r, out, w_post=w, gate=gate[0], flags=pq2.PQ2_WEIGHTS_STATIC)
    torch.cuda.synchronize()
    for x, out in zip(xg, outs):
        pq2.pq2_gemm_bf16_splitk(x, wg, gate)
        torch.cuda.synchronize()
        want = torch.empty_like(r)
        pq2.pq2_norm_residual(y, r, want, w_post=w, gate=gate[0])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
