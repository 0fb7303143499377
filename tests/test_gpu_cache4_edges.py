"""The 4-bit cache at the edges of what a call may hold: tokens without a place,
groups of many heads, numbers of rows on both sides of a change of kernel."""
import numpy as np
import pytest
import torch

from test_gpu_cache4 import Cache, _dev

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
