"""Host-side argument checks of the steps around a projection (no GPU: every
call here is refused, or has nothing to do, before any CUDA call)."""
import ctypes

import pytest

from test_abi_host import FAKE, ODD, _p, lib  # noqa: F401  (lib is a fixture)


def _norm_args(b, **kw):
    a = b.NormResidualArgs(FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, 64, 64, 64, 0, 64, b.PQ2_F32,
                           b.PQ2_BF16, b.PQ2_F32, 0, b.PQ2_F16, 1e-6, 1.0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_norm_residual_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    f = lib.pq2_norm_residual
    assert f(None, 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b), -1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b), 1, 0, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, ld_y=1 << 20, ld_r=1 << 20, ld_r_out=1 << 20, ld_x=1 << 20), 1, 49153,
             None) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert f(_norm_args(b), 0, 64, None) == b.PQ2_OK                    # nothing to do
    for name in ("y", "r", "r_out"):
        assert f(_norm_args(b, **{name: None}), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    for name in ("ld_y", "ld_r", "ld_r_out", "ld_x"):
        assert f(_norm_args(b, **{name: 63}), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, gate=FAKE, ld_gate=63), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    for name in ("y_type", "r_type", "w_type", "x_type"):
        assert f(_norm_args(b, **{name: 3}), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, y=FAKE + 2), 1, 64, None) == b.PQ2_ERR_MISALIGNED
    assert f(_norm_args(b, x=FAKE + 1), 1, 64, None) == b.PQ2_ERR_MISALIGNED
    assert f(_norm_args(b, eps=-1.0), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, eps=float("nan")), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, flags=1 << 10), 1, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, flags=b.PQ2_GATE_SIGMOID | b.PQ2_GATE_SILU), 1, 64, None) == \
        b.PQ2_ERR_INVALID_ARG


def test_rmsnorm_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    f, P = lib.pq2_rmsnorm, _p(FAKE)
    ok = [P, b.PQ2_BF16, 64, P, b.PQ2_F32, P, b.PQ2_F16, 64]
    assert f(*ok, 0, 64, 1e-6, 0, None) == b.PQ2_OK
    assert f(*ok, 1, 64, 1e-6, b.PQ2_GATE_SILU, None) == b.PQ2_ERR_INVALID_ARG
    assert f(*ok, 1, 65, 1e-6, 0, None) == b.PQ2_ERR_INVALID_ARG        # row strides below H
    for i in (0, 5):
        bad = list(ok)
        bad[i] = None
        assert f(*bad, 1, 64, 1e-6, 0, None) == b.PQ2_ERR_INVALID_ARG
    bad = list(ok)
    bad[3] = _p(FAKE + 2)
    assert f(*bad, 1, 64, 1e-6, 0, None) == b.PQ2_ERR_MISALIGNED


def _lora(lib, b, **kw):  # noqa: F811
    a = dict(x=_p(FAKE), ld_x=64, A=_p(FAKE), B=_p(FAKE), type=b.PQ2_F16, ids=_p(FAKE), ranks=None,
             scales=None, y_in=_p(FAKE), ld_in=32, y_out=_p(FAKE), ld_out=32, y_type=b.PQ2_F32, M=4,
             N=32, K=64, L=2, R=8, workspace=_p(FAKE), workspace_bytes=0, stream=None)
    a.update(kw)
    return lib.pq2_lora_add(*a.values())


def test_lora_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    assert _lora(lib, b) == b.PQ2_ERR_WORKSPACE
    assert _lora(lib, b, workspace=None, workspace_bytes=1 << 30) == b.PQ2_ERR_WORKSPACE
    for name in ("x", "A", "B", "ids", "y_in", "y_out"):
        assert _lora(lib, b, **{name: None}) == b.PQ2_ERR_INVALID_ARG
    for name in ("x", "A", "B", "workspace"):
        assert _lora(lib, b, **{name: _p(ODD)}) == b.PQ2_ERR_MISALIGNED
    for name in ("ids", "ranks", "scales", "y_in", "y_out"):
        assert _lora(lib, b, **{name: _p(FAKE + 2)}) == b.PQ2_ERR_MISALIGNED
    assert _lora(lib, b, M=-1) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, M=0, workspace=None, x=None) == b.PQ2_OK       # nothing to do
    assert _lora(lib, b, N=0, workspace=None, y_out=None) == b.PQ2_OK
    assert _lora(lib, b, K=60) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, K=72) == b.PQ2_ERR_INVALID_ARG                 # ld_x below K
    assert _lora(lib, b, ld_x=68) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, R=12) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, R=264) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, R=0) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, L=0) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, L=16385) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, M=1048577) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert _lora(lib, b, type=b.PQ2_F32) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, y_type=b.PQ2_F16) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, ld_in=31) == b.PQ2_ERR_INVALID_ARG
    assert _lora(lib, b, ld_out=33) == b.PQ2_ERR_INVALID_ARG            # in place, two strides
    assert b.pq2_lora_workspace_bytes(4, 32, 60, 2, 8) == b.SIZE_MAX
    assert b.pq2_lora_workspace_bytes(0, 32, 64, 2, 8) == 0
    assert 0 < b.pq2_lora_workspace_bytes(4096, 17408, 5120, 16384, 256) < 1 << 30
    # a workspace for many tokens serves fewer
    for N, K, L, R in ((5120, 17408, 64, 64), (17408, 5120, 64, 128), (40, 8, 1, 8), (64, 640, 300, 16)):
        sizes = [b.pq2_lora_workspace_bytes(M, N, K, L, R)
                 for M in (*range(1, 140), 512, 513, 2400, 2401, 5000)]
        assert sizes == sorted(sizes)


def _verify(lib, b, **kw):  # noqa: F811
    P = _p(FAKE)
    a = dict(logits=P, ld_logits=50, row_start=P, drafts=P, q=P, ld_q=50, u=P, e=P, ld_e=50,
             temperature=P, accepted=P, tokens=P, B=2, rows=4, V=50, workspace=P, workspace_bytes=0,
             stream=None)
    a.update(kw)
    return lib.pq2_verify_drafts(*a.values())


def test_verify_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    assert _verify(lib, b) == b.PQ2_ERR_WORKSPACE
    assert _verify(lib, b, workspace=None, workspace_bytes=1 << 20) == b.PQ2_ERR_WORKSPACE
    for name in ("logits", "row_start", "drafts", "u", "e", "temperature", "accepted", "tokens"):
        assert _verify(lib, b, **{name: None}) == b.PQ2_ERR_INVALID_ARG
        assert _verify(lib, b, **{name: _p(FAKE + 2)}) == b.PQ2_ERR_MISALIGNED
    assert _verify(lib, b, workspace=_p(ODD)) == b.PQ2_ERR_MISALIGNED
    for name in ("ld_logits", "ld_q", "ld_e"):
        assert _verify(lib, b, **{name: 49}) == b.PQ2_ERR_INVALID_ARG
    assert _verify(lib, b, V=0) == b.PQ2_ERR_INVALID_ARG
    assert _verify(lib, b, B=-1) == b.PQ2_ERR_INVALID_ARG
    assert _verify(lib, b, rows=-1) == b.PQ2_ERR_INVALID_ARG
    assert _verify(lib, b, B=0, workspace=None) == b.PQ2_OK             # nothing to do
    big = (1 << 30) + 1
    assert _verify(lib, b, V=big, ld_logits=big, ld_q=big, ld_e=big) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    assert b.pq2_verify_workspace_bytes(1 << 24, 1 << 24, 1 << 30) == b.SIZE_MAX
    assert 0 < b.pq2_verify_workspace_bytes(64, 256, 248320) < 1 << 20


def test_bindings_refuse_host_tensors(lib):  # noqa: F811
    import torch
    from gemm_pq2_ternary_gb300 import binding as b
    r = torch.zeros((2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        b.pq2_rmsnorm(r, None, r)
    with pytest.raises(ValueError, match="CUDA"):
        b.pq2_norm_residual(r, r, r)
    with pytest.raises(ValueError, match="CUDA"):
        b.pq2_verify_drafts(r, r, r, None, r, r, r[:, 0], r, r, None)
    with pytest.raises(ValueError, match="CUDA"):
        h = torch.zeros((2, 8), dtype=torch.float16)
        b.pq2_lora_add(h, torch.zeros((1, 8, 8), dtype=torch.float16),
                       torch.zeros((1, 4, 8), dtype=torch.float16),
                       torch.zeros(2, dtype=torch.int32), r, r, None)


def test_packed_arguments_meet_the_same_checks(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    assert lib.pq2_lora_add_packed(None, None) == b.PQ2_ERR_INVALID_ARG
    assert lib.pq2_verify_drafts_packed(None, None) == b.PQ2_ERR_INVALID_ARG
    # each field in its place: only the one that is wrong decides
    ok = dict(x=FAKE, A=FAKE, B=FAKE, ids=FAKE, ranks=0, scales=0, y_in=FAKE, y_out=FAKE, workspace=FAKE,
              ld_x=64, ld_in=32, ld_out=32, M=4, N=32, K=64, L=2, R=8, workspace_bytes=0, type=b.PQ2_F16,
              y_type=b.PQ2_F32)

    def lora(**kw):
        return lib.pq2_lora_add_packed(b._lora_add_args.pack(*{**ok, **kw}.values()), None)
    assert lora() == b.PQ2_ERR_WORKSPACE
    assert lora(M=0) == b.PQ2_OK
    assert lora(K=60) == lora(R=9) == b.PQ2_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=0), dict(B=0), dict(ids=0), dict(y_in=0), dict(y_out=0), dict(ld_x=56),
               dict(ld_in=31), dict(ld_out=31), dict(type=b.PQ2_F32), dict(y_type=b.PQ2_F16),
               dict(L=0), dict(M=-1), dict(N=-1)):
        assert lora(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(A=ODD), dict(workspace=ODD), dict(ranks=FAKE + 2), dict(scales=FAKE + 2)):
        assert lora(**kw) == b.PQ2_ERR_MISALIGNED, kw
    ok2 = dict(logits=FAKE, row_start=FAKE, drafts=FAKE, q=FAKE, u=FAKE, e=FAKE, temperature=FAKE,
               accepted=FAKE, tokens=FAKE, workspace=FAKE, ld_logits=50, ld_q=50, ld_e=50, B=2, rows=4,
               V=50, workspace_bytes=0)

    def verify(**kw):
        return lib.pq2_verify_drafts_packed(b._verify_drafts_args.pack(*{**ok2, **kw}.values()), None)
    assert verify() == b.PQ2_ERR_WORKSPACE
    assert verify(B=0) == b.PQ2_OK
    for kw in (dict(ld_logits=49), dict(ld_q=49), dict(ld_e=49), dict(V=0), dict(rows=-1), dict(logits=0),
               dict(row_start=0), dict(temperature=0), dict(accepted=0)):
        assert verify(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(q=FAKE + 2), dict(e=FAKE + 2), dict(workspace=ODD)):
        assert verify(**kw) == b.PQ2_ERR_MISALIGNED, kw


def test_norms_in_place_need_one_row_stride(lib):  # noqa: F811
    # rows are worked on in any order: with another stride (or type) a row
    # would be written over one that is still to be read
    from gemm_pq2_ternary_gb300 import binding as b
    f = lib.pq2_norm_residual
    wide = dict(x=None, ld_y=64)
    assert f(_norm_args(b, ld_r_out=72, **wide), 2, 64, None) == b.PQ2_ERR_INVALID_ARG
    assert f(_norm_args(b, ld_r=72, **wide), 3, 64, None) == b.PQ2_ERR_INVALID_ARG
    g, P = lib.pq2_rmsnorm, _p(FAKE)

    def before(rt, ld_r, xt, ld_x, M):
        return g(P, rt, ld_r, P, b.PQ2_F32, P, xt, ld_x, M, 64, 1e-6, 0, None)
    assert before(b.PQ2_BF16, 64, b.PQ2_BF16, 72, 2) == b.PQ2_ERR_INVALID_ARG
    assert before(b.PQ2_F16, 72, b.PQ2_F16, 64, 2) == b.PQ2_ERR_INVALID_ARG
    assert before(b.PQ2_F32, 64, b.PQ2_F16, 64, 2) == b.PQ2_ERR_INVALID_ARG
    assert before(b.PQ2_F32, 64, b.PQ2_F16, 64, 1) == b.PQ2_ERR_INVALID_ARG
