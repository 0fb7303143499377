"""Host-side argument checks of the attention side of a step, sizes whose sums
and products do not fit 64 bits (no GPU: every call here is refused)."""

from test_abi_host import FAKE, _p, lib  # noqa: F401  (lib is a fixture)
from test_attention_host import CACHE, _caller


def test_rope_table_refuses_positions_past_64_bits(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    for first, count in ((1 << 62, 1 << 62), ((1 << 63) - 1, 1), (1, (1 << 63) - 1), ((1 << 31) - 3, 4), (0, (1 << 31) + 1)):
        assert lib.pq2_rope_table(_p(FAKE), first, count, 64, 1e4, None, None) == b.PQ2_ERR_UNSUPPORTED_SHAPE, (first, count)


def test_cache_refuses_tables_past_64_bits(lib):  # noqa: F811
    from gemm_pq2_ternary_gb300 import binding as b
    ok = dict(**CACHE, k_out=FAKE, v_out=FAKE, ld_k=256, hs_k=128, ld_v=256, hs_v=128, M=4, out_type=b.PQ2_F16,
              reserved=0)
    call = _caller(lib.pq2_cache4_read, b._cache4_read_args, ok)
    for W in (1 << 59, 1 << 60, (1 << 60) + 1, (1 << 63) - 1):
        assert call(W=W, ld_pages=(1 << 63) - 1) == b.PQ2_ERR_UNSUPPORTED_SHAPE, W
