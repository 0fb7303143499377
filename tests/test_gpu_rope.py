"""Rotary positions on the GPU: tables against 64-bit angles, turned heads
against the same 32-bit steps in numpy (to the bit), and against rotations in
64 bits."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


def _np(t):
    return t.detach().float().cpu().numpy()


@pytest.mark.parametrize("kind,extra", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("ramp", dict(factor=4.0, old_len=32768.0, low=1.0, high=32.0)),
    ("ramp", dict(factor=2.0, old_len=100.0, low=1.0, high=1.0000001)),
    ("bands", dict(factor=8.0, old_len=8192.0, low=1.0, high=4.0))])
@pytest.mark.parametrize("rot,first,count", [(64, 0, 300), (128, 262000, 77), (6, 2 ** 31 - 9, 9), (256, 1000003, 5)])
def test_tables(pq2, kind, extra, rot, first, count):
    t = torch.full((count + 2, rot // 2, 2), 7.0, device=DEV)
    code = {"plain": pq2.PQ2_ROPE_PLAIN, "linear": pq2.PQ2_ROPE_LINEAR, "base": pq2.PQ2_ROPE_BASE,
            "ramp": pq2.PQ2_ROPE_RAMP, "bands": pq2.PQ2_ROPE_BANDS}[kind]
    pq2.pq2_rope_table(t[:count], 1e6, first=first, kind=code, magnitude=1.25, **extra)
    want = ref.table(first, count, ref.frequencies(rot, 1e6, kind, **extra), 1.25)
    # one rounding to fp32, and angles: 64-bit frequencies off by about 4 roundings, times the position
    tol = 2.0 ** -24 * np.abs(want) + 8 * 2.0 ** -53 * (first + count) + 1e-12
    assert np.all(np.abs(t[:count].double().cpu().numpy() - want) <= tol)
    assert torch.all(t[count:] == 7.0)


def _inputs(M, H, D, seed, wide=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((M, H + wide, D + 2 * wide), generator=g, device=DEV).to(dtype)
    return x[:, wide:, wide:wide + D] if wide else x


def _table(rows, rot, seed=5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.rand((rows, rot // 2), generator=g, device=DEV, dtype=torch.float64) * 1e4
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float().contiguous()


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 6), (128, 128), (128, 64), (128, 8), (128, 74), (256, 256),
                                   (256, 64), (256, 16), (256, 250), (96, 96), (80, 20), (1, 0), (2, 2), (512, 512),
                                   (100, 34), (128, 0)])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("xt,yt", [("f32", "f16"), ("bf16", "bf16"), ("f16", "f32")])
def test_turned_to_the_bit(pq2, D, rot, near, xt, yt):
    for M, H, H2, wide in ((1, 1, 0, 0), (5, 3, 2, 0), (37, 5, 1, 8), (3, 2, 1, 1)):
        x = _inputs(M, H, D, M + D, wide, TYPES[xt])
        x2 = _inputs(M, H2, D, M + rot, 0, TYPES[xt]) if H2 else None
        t = _table(50, rot) if rot else None
        pos = torch.randint(0, 50, (M,), device=DEV, dtype=torch.int32)
        out = torch.full((M, H, D + 2 * wide), 9.0, dtype=TYPES[yt], device=DEV)
        y = out[..., wide:wide + D]
        y2 = torch.empty((M, H2, D), dtype=TYPES[yt], device=DEV) if H2 else None
        pq2.pq2_rope(x, t, pos, y, x2, y2, flags=pq2.PQ2_ROPE_NEIGHBOURS if near else 0)
        cs = t[pos.long()].cpu().numpy() if rot else np.zeros((M, 0, 2), np.float32)
        for a, b in ((x, y), (x2, y2)):
            if a is None:
                continue
            want = torch.from_numpy(ref.turn(_np(a), cs, rot, near)).to(TYPES[yt])
            assert torch.equal(b.cpu(), want)
        if wide:  # nothing around the heads is written
            assert torch.all(out[..., :wide] == 9.0) and torch.all(out[..., wide + D:] == 9.0)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK


@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (128, 36), (96, 48)])
@pytest.mark.parametrize("near", [False, True])
def test_in_place_and_back(pq2, D, rot, near):
    M, H = 67, 6
    x = _inputs(M, H, D, 3)
    t, pos = _table(100, rot), torch.randint(0, 100, (M,), device=DEV, dtype=torch.int32)
    flags = pq2.PQ2_ROPE_NEIGHBOURS if near else 0
    want = torch.empty_like(x)
    pq2.pq2_rope(x, t, pos, want, flags=flags)
    y = x.clone()
    pq2.pq2_rope(y, t, pos, y, flags=flags)
    assert torch.equal(y, want)
    pq2.pq2_rope(y, t, pos, y, flags=flags | pq2.PQ2_ROPE_INVERSE)
    # two turns: 3 roundings each, cos^2 + sin^2 off by 2 roundings of the table
    assert torch.all((y - x).abs() <= 10 * 2.0 ** -24 * x.abs().amax(-1, keepdim=True) * 2)


def test_gradient(pq2):
    # of sum(out * w): the inverse turn of w; against differences (the operator is linear)
    M, H, D, rot = 5, 2, 64, 48
    t, pos = _table(9, rot), torch.arange(M, device=DEV, dtype=torch.int32)
    x, w, d = (_inputs(M, H, D, s) for s in (1, 2, 3))
    grad, y0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    pq2.pq2_rope(w, t, pos, grad, flags=pq2.PQ2_ROPE_INVERSE)
    pq2.pq2_rope(x, t, pos, y0)
    pq2.pq2_rope(x + d, t, pos, y1)
    change = float(((y1 - y0).double() * w.double()).sum())
    assert abs(change - float((grad.double() * d.double()).sum())) <= 1e-4


def test_positions_outside_the_table(pq2):
    M, H, D = 6, 3, 128
    t = _table(10, D)
    x = _inputs(M, H, D, 1)
    pos = torch.tensor([0, -1, 9, 10, 2 ** 31 - 1, 3], dtype=torch.int32, device=DEV)
    y = torch.full_like(x, 5.0)
    pq2.pq2_rope(x, t, pos, y)
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    assert torch.all(y[[1, 3, 4]] == 5.0)
    want = ref.turn(_np(x), t[pos.clamp(0, 9).long()].cpu().numpy(), D, False)
    assert np.array_equal(_np(y)[[0, 2, 5]], want[[0, 2, 5]])


def test_streams_and_graphs(pq2):
    M, H, D = 33, 4, 128
    x, t = _inputs(M, H, D, 1), _table(64, D)
    pos = torch.arange(M, device=DEV, dtype=torch.int32)
    y, z = torch.empty_like(x), torch.empty_like(x)
    pq2.pq2_rope(x, t, pos, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pq2.pq2_rope(x, t, pos, z, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq2.pq2_rope(x, t, pos, z)
    x.mul_(2.0)
    g.replay()
    pq2.pq2_rope(x, t, pos, y)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
