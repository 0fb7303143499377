"""Host-side argument checks of the attention side of a step (no GPU: every
call here is refused, or has nothing to do, before any CUDA call)."""
import ctypes

import numpy as np
import pytest

from test_abi_host import FAKE, ODD, _p, lib  # noqa: F401  (lib is a fixture)

NAN, INF = float("nan"), float("inf")


def _caller(fn, packer, ok):
    def call(**kw):
        assert set(kw) <= set(ok), set(kw) - set(ok)
        return fn(packer.pack(*{**ok, **kw}.values()), None)
    return call


CACHE = dict(pool=FAKE, pages=FAKE, row_start=FAKE, lens=FAKE, page_stride=2 * 16 * 136, num_pages=4, ld_pages=3, B=2,
             W=3, heads=2, dim=128, page_tokens=16, cache_reserved=0)


def _cache_cases(call, b, pointers=True):
    big = 1 << 31
    for kw in (dict(B=-1), dict(W=-1), dict(num_pages=-1), dict(heads=0), dict(cache_reserved=1), dict(ld_pages=2),
               dict(page_stride=2 * 16 * 136 - 16)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(heads=1025), dict(dim=96), dict(dim=0), dict(page_tokens=8), dict(page_tokens=24),
               dict(page_tokens=1040), dict(page_stride=2 * 16 * 136 + 8), dict(B=big), dict(W=big, ld_pages=big),
               dict(W=1 << 27, ld_pages=1 << 27), dict(num_pages=big)):
        assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
    for name in ("pool", "pages", "row_start", "lens"):
        assert call(**{name: 0}) == b.PQ2_ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == b.PQ2_ERR_MISALIGNED, name
    assert call(pool=ODD) == b.PQ2_ERR_MISALIGNED
    assert call(B=0, row_start=0, lens=0, pages=0) == b.PQ2_OK            # nothing to do


def test_rope_table_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b

    def call(table=FAKE, first=0, count=4, rot=64, base=1e4, kind=0, magnitude=0.0, factor=1.0, old_len=0.0, low=0.0,
             high=0.0):
        return lib.pq2_rope_table(_p(table), first, count, rot, base,
                                  b._rope_scaling.pack(kind, magnitude, factor, old_len, low, high), None)
    assert call(count=0) == b.PQ2_OK
    assert call(table=0) == b.PQ2_ERR_INVALID_ARG
    assert call(table=ODD) == b.PQ2_ERR_MISALIGNED
    for kw in (dict(first=-1), dict(count=-1), dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=NAN), dict(base=INF),
               dict(kind=5), dict(kind=-1), dict(magnitude=NAN), dict(kind=1, factor=0.5), dict(kind=1, factor=NAN),
               dict(kind=2, factor=2.0, rot=2), dict(kind=3, factor=2.0), dict(kind=3, factor=2.0, old_len=9.0, low=0.0, high=1.0),
               dict(kind=4, factor=2.0, old_len=9.0, low=2.0, high=2.0), dict(kind=4, factor=2.0, old_len=INF, low=1.0, high=2.0)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(rot=514), dict(first=2 ** 31, count=1)):
        assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw


def test_rope_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(x=FAKE, x2=FAKE, out=FAKE + 1024, out2=FAKE + 1024, table=FAKE, positions=FAKE, ld_x=256, hs_x=64, ld_x2=256,
              hs_x2=64, ld_out=256, hs_out=64, ld_out2=256, hs_out2=64, M=0, table_rows=8, heads=4, heads2=2, dim=64,
              rot=64, x_type=b.PQ2_F32, out_type=b.PQ2_F16, flags=0, reserved=0)
    call = _caller(lib.pq2_rope, b._rope_args, ok)
    assert lib.pq2_rope(None, None) == b.PQ2_ERR_INVALID_ARG
    assert call() == call(M=3, heads=0, heads2=0) == b.PQ2_OK
    for kw in (dict(M=-1), dict(heads=-1), dict(heads2=-1), dict(dim=0), dict(rot=-2), dict(rot=66), dict(rot=3),
               dict(table_rows=-1), dict(flags=4), dict(reserved=1), dict(x_type=3), dict(out_type=-1)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(dim=514, rot=0), dict(heads=65536), dict(M=1 << 25)):
        assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=0), dict(x2=0), dict(out=0), dict(out2=0), dict(table=0), dict(positions=0), dict(ld_x=63),
               dict(hs_x=63), dict(hs_out2=0), dict(out=FAKE), dict(out2=FAKE),
               dict(out=FAKE, out_type=b.PQ2_F32, ld_out=320)):
        assert call(M=2, **kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(x=FAKE + 2), dict(out=FAKE + 1), dict(table=ODD), dict(positions=FAKE + 2)):
        assert call(M=2, **kw) == b.PQ2_ERR_MISALIGNED, kw


def test_append_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(**CACHE, k=FAKE, v=FAKE, q=FAKE, q_out=FAKE + 64, table=FAKE, positions=0, ld_k=256, hs_k=128, ld_v=256,
              hs_v=128, ld_q=512, hs_q=128, ld_q_out=512, hs_q_out=128, M=4, table_rows=99, q_heads=4, rot=128,
              x_type=b.PQ2_F32, out_type=b.PQ2_F16, flags=0, reserved=0)
    call = _caller(lib.pq2_cache4_append, b._cache4_append_args, ok)
    assert lib.pq2_cache4_append(None, None) == b.PQ2_ERR_INVALID_ARG
    _cache_cases(call, b)
    assert call(M=0, k=0) == b.PQ2_OK
    for kw in (dict(k=0), dict(v=0), dict(q=0), dict(q_out=0), dict(table=0), dict(M=-1), dict(q_heads=-1), dict(rot=130),
               dict(rot=5), dict(rot=-2), dict(flags=2), dict(x_type=9), dict(out_type=9), dict(ld_k=127), dict(hs_v=127),
               dict(reserved=1), dict(q_out=FAKE), dict(q_out=FAKE, out_type=b.PQ2_F32, hs_q_out=64)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(M=1 << 25), dict(q_heads=70000)):
        assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(k=FAKE + 2), dict(q_out=FAKE + 1), dict(table=ODD), dict(positions=FAKE + 1)):
        assert call(**kw) == b.PQ2_ERR_MISALIGNED, kw


def test_read_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(**CACHE, k_out=FAKE, v_out=FAKE, ld_k=256, hs_k=128, ld_v=256, hs_v=128, M=4, out_type=b.PQ2_F16,
              reserved=0)
    call = _caller(lib.pq2_cache4_read, b._cache4_read_args, ok)
    assert lib.pq2_cache4_read(None, None) == b.PQ2_ERR_INVALID_ARG
    _cache_cases(call, b)
    assert call(M=0) == call(k_out=0, v_out=0) == b.PQ2_OK
    for kw in (dict(M=-1), dict(out_type=3), dict(ld_v=100), dict(hs_k=127), dict(reserved=2)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    assert call(v_out=FAKE + 1) == b.PQ2_ERR_MISALIGNED


def test_attend_checks_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(**CACHE, q=FAKE, out=FAKE, workspace=FAKE, ld_q=512, hs_q=128, ld_out=512, hs_out=128, M=4, max_rows=1,
              window=0, workspace_bytes=0, scale=0.1, q_heads=4, type=b.PQ2_F16, reserved=0)
    call = _caller(lib.pq2_cache4_attend, b._cache4_attend_args, ok)
    assert lib.pq2_cache4_attend(None, None) == b.PQ2_ERR_INVALID_ARG
    _cache_cases(call, b)
    assert call() == call(workspace=0, workspace_bytes=1 << 40) == b.PQ2_ERR_WORKSPACE
    assert call(M=0) == b.PQ2_OK
    for kw in (dict(q=0), dict(out=0), dict(M=-1), dict(max_rows=-1), dict(window=-1), dict(scale=NAN), dict(scale=INF),
               dict(type=b.PQ2_F32), dict(q_heads=3), dict(q_heads=0), dict(ld_q=120), dict(hs_out=120), dict(reserved=1)):
        assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(q_heads=130), dict(M=(1 << 20) + 1)):
        assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(q=ODD), dict(out=ODD), dict(workspace=ODD), dict(ld_q=516), dict(hs_q=132), dict(ld_out=516),
               dict(hs_out=132)):
        assert call(**kw) == b.PQ2_ERR_MISALIGNED, kw
    f = b.pq2_cache4_attend_workspace_bytes
    assert f(4, 3, 2, 128) == f(4, 4, 2, 96) == f(-1, 4, 2, 128) == b.SIZE_MAX and f(0, 4, 2, 128) == 0
    for dim in (64, 128, 256):
        sizes = [f(M, 24, 4, dim) for M in (1, 2, 3, 7, 8, 9, 64, 65, 1000, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[-1] < 1 << 29   # enough for fewer rows too


def test_pages_check_arguments(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(pages=FAKE, lens=FAKE, refs=FAKE, source=FAKE, keep=FAKE, new_lens=FAKE, pages_out=FAKE + 64, refs_out=FAKE,
              copies=FAKE, info=FAKE, workspace=FAKE, ld_pages=4, ld_out=4, B=2, W=4, P=9, T=16, workspace_bytes=0)
    few = {k: v for k, v in ok.items() if k not in ("source", "keep", "new_lens")}
    for fn, packer, args in ((lib.pq2_pages_update, b._pages_update_args, ok),
                             (lib.pq2_pages_compact, b._pages_compact_args, few)):
        call = _caller(fn, packer, args)
        assert fn(None, None) == b.PQ2_ERR_INVALID_ARG
        assert call() == call(workspace=0, workspace_bytes=1 << 40) == b.PQ2_ERR_WORKSPACE
        for name in args:
            if name in ("workspace", "workspace_bytes", "ld_pages", "ld_out", "B", "W", "P", "T"):
                continue
            assert call(**{name: 0}) == b.PQ2_ERR_INVALID_ARG, name
            assert call(**{name: FAKE + 2}) == b.PQ2_ERR_MISALIGNED, name
        for kw in (dict(B=-1), dict(W=0), dict(P=-1), dict(T=0), dict(ld_pages=3), dict(ld_out=3)):
            assert call(**kw) == b.PQ2_ERR_INVALID_ARG, kw
        for kw in (dict(B=(1 << 20) + 1), dict(P=(1 << 28) + 1), dict(T=(1 << 20) + 1),
                   dict(W=1 << 11, T=1 << 20, ld_pages=1 << 11, ld_out=1 << 11)):
            assert call(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
        assert call(workspace=ODD) == b.PQ2_ERR_MISALIGNED
    assert _caller(lib.pq2_pages_update, b._pages_update_args, ok)(pages_out=FAKE) == b.PQ2_ERR_INVALID_ARG
    assert _caller(lib.pq2_pages_compact, b._pages_compact_args, few)(pages_out=FAKE, ld_out=5) == b.PQ2_ERR_INVALID_ARG
    assert b.pq2_pages_workspace_bytes(-1, 4) == b.SIZE_MAX

    def copy(pool=FAKE, page_bytes=32, page_stride=32, P=4, layers=1, layer_stride=0, pairs=FAKE, n=2):
        return lib.pq2_pages_copy(_p(pool), page_bytes, page_stride, P, layers, layer_stride, _p(pairs), n, None)
    assert copy(n=0) == copy(layers=0) == copy(P=0) == copy(page_bytes=0) == b.PQ2_OK
    for kw in (dict(pool=0), dict(pairs=0), dict(page_bytes=-16), dict(page_stride=16), dict(P=-1), dict(layers=-1),
               dict(layer_stride=-16), dict(n=-1)):
        assert copy(**kw) == b.PQ2_ERR_INVALID_ARG, kw
    for kw in (dict(page_bytes=24), dict(page_stride=40), dict(layer_stride=8), dict(layers=65537), dict(n=(1 << 28) + 1)):
        assert copy(**kw) == b.PQ2_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(pool=ODD), dict(pairs=FAKE + 4)):
        assert copy(**kw) == b.PQ2_ERR_MISALIGNED, kw


def test_page_bytes(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    f = b.pq2_cache4_page_bytes
    assert f(8, 128, 32) == 8 * 32 * 136
    assert f(0, 128, 32) == f(8, 127, 32) == f(8, 128, 0) == f(8, 128, 40) == f(8, 128, 2048) == 0


def test_bindings_refuse_what_they_cannot_pass(lib):  # noqa: F811
    import torch
    from gemm_pq2_ternary_gb300 import binding as b
    x, i = torch.zeros((2, 4, 64)), torch.zeros(2, dtype=torch.int32)
    pool, pages = torch.zeros((3, 4, 16 * 72), dtype=torch.uint8), torch.zeros((2, 2), dtype=torch.int32)
    for f in (lambda: b.pq2_rope(x, None, i, x), lambda: b.pq2_cache4_append(x, x, pool, pages, i, i),
              lambda: b.pq2_cache4_read(pool, pages, i, i, x, x), lambda: b.pq2_pages_copy(pool, pages),
              lambda: b.pq2_cache4_attend(x, pool, pages, i, i, x, None),
              lambda: b.pq2_pages_compact(pages, i, i, 16, pages, i, pages, i, None)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(b.PQ2Error):
        b.alloc_cache4(2, 4, 96, 16, device="cpu")
    with pytest.raises(b.PQ2Error):
        b.alloc_attend_workspace(4, 3, 2, 128, device="cpu")


def test_oracle_turns_and_quantises():
    # the oracle's own pins: known turns, and codes that stand for their values
    from oracle import attention as ref
    f = ref.frequencies(4, 100.0)
    assert np.allclose(f, [1.0, 0.1])
    cs = ref.table(0, 3, f).astype(np.float32)
    x = np.array([[[1, 2, 3, 4]]], np.float32)
    c, s = np.cos([2, 0.2]), np.sin([2, 0.2])
    want = [1 * c[0] - 3 * s[0], 2 * c[1] - 4 * s[1], 3 * c[0] + 1 * s[0], 4 * c[1] + 2 * s[1]]
    assert np.allclose(ref.turn(x, cs[2:], 4, False)[0, 0], want, rtol=1e-6)
    want = [1 * c[0] - 2 * s[0], 2 * c[0] + 1 * s[0], 3 * c[1] - 4 * s[1], 4 * c[1] + 3 * s[1]]
    assert np.allclose(ref.turn(x, cs[2:], 4, True)[0, 0], want, rtol=1e-6)
    assert np.allclose(ref.frequencies(64, 1e4, "linear", 4.0), ref.frequencies(64, 1e4) / 4)
    bands = ref.frequencies(128, 5e5, "bands", 8.0, 8192.0, 1.0, 4.0)
    plain = ref.frequencies(128, 5e5)
    assert bands[0] == plain[0] and np.isclose(bands[-1], plain[-1] / 8) and np.all(np.diff(bands) < 0)
    ramp = ref.frequencies(128, 1e4, "ramp", 4.0, 4096.0, 1.0, 32.0)
    plain = ref.frequencies(128, 1e4)
    assert ramp[0] == plain[0] and np.isclose(ramp[-1], plain[-1] / 4)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    code, s, z = ref.quantise(x)
    assert np.all(np.abs(ref.dequantise(code, s, z) - x) <= s * 0.51 + 2.0 ** -10 * 15)
    assert code.min() == 0 and code.max() == 15
    code, s, z = ref.quantise(np.full((1, 64), -3.25, np.float32))
    assert np.all(code == 0) and s[0, 0] == 0 and z[0, 0] == -3.25
