"""The pages of a cache and rotary tables in the bounds-checked build: the same
results as the normal build and no report at exact sizes; and, with the last
element of every checked buffer treated as outside, a report and nothing
written around the outputs."""
import numpy as np
import pytest
import torch

from test_gpu_cache4 import _dev
from test_gpu_cache4_limits import SENTINEL, _padded, _untouched, libs  # noqa: F401  (libs is a fixture)
from test_gpu_pages import _state

pytestmark = pytest.mark.gpu

DEV = "cuda"
B, W, T, P, WIDE = 5, 7, 16, 41, 9


def _outputs():
    # rows of pages end before the next ones begin
    pb, pages = _padded((B, WIDE), torch.int32)
    return (pb, pages), _padded((P,), torch.int32), _padded((2,), torch.int32)


def _update(pq2):
    rng = np.random.default_rng(3)
    pages, lens, refs = _state(rng, B, W, T, P)
    lens = np.minimum(lens, W * T - 1)
    keep = np.maximum(lens - 5, 0)
    out, ref, info = _outputs()
    copies = _padded((B, 2), torch.int32)
    pq2.pq2_pages_update(_dev(pages), _dev(refs), _dev(lens), _dev((np.arange(B) + 1) % B), _dev(keep), _dev(keep + 1), T,
                         out[1][:, :W], ref[1], copies[1], info[1], pq2.alloc_pages_workspace(B, P))
    return [out, ref, info, copies]


def _compact(pq2):
    rng = np.random.default_rng(4)
    pages, lens, refs = _state(rng, B, W, T, P)
    n = -(-lens[0] // T)
    refs[pages[0, :n]] -= 1
    pages[0], lens[0] = -1, 0
    out, ref, info = _outputs()
    copies = _padded((P // 2, 2), torch.int32)
    pq2.pq2_pages_compact(_dev(pages), _dev(refs), _dev(lens), T, out[1][:, :W], ref[1], copies[1], info[1],
                          pq2.alloc_pages_workspace(B, P))
    return [out, ref, info, copies]


def _copy(pq2, layers):
    nbytes = 2 * 8192 + 48                                  # no multiple of a piece
    buf, pool = _padded((2, 5, nbytes), torch.uint8)
    pool.copy_(torch.arange(pool.numel(), device=DEV).view(pool.shape) % 251)
    pq2.pq2_pages_copy(pool if layers else pool[0], _dev([[0, 4], [-1, 2], [3, 1]]), layers=layers)
    return [(buf, pool)]


def _table(pq2):
    out = _padded((77, 5, 2), torch.float32)
    pq2.pq2_rope_table(out[1], 1e4, first=9)
    return [out]


CASES = {"update": _update, "compact": _compact, "copy": lambda p: _copy(p, False), "copy_layers": lambda p: _copy(p, True),
         "rope_table": _table}


def _run(pq2, lib, name):
    pq2._lib = lib
    outs = CASES[name](pq2)
    torch.cuda.synchronize()
    return outs


def _beside(outs):
    return all(bool((o[:, W:] == SENTINEL).all()) for _, o in outs if o.shape == (B, WIDE))


@pytest.mark.parametrize("name", CASES)
def test_checked_build_matches_and_reports_nothing(libs, name):  # noqa: F811
    pq2, release, debug = libs
    try:
        want = _run(pq2, release, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        got = _run(pq2, debug, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    finally:
        pq2._lib = release
    assert all(torch.equal(w, g) for (_, w), (_, g) in zip(want, got))
    for outs in (want, got):
        assert _untouched(outs) and _beside(outs)


@pytest.mark.parametrize("name", CASES)
def test_checked_build_reports_a_store_outside(libs, name):  # noqa: F811
    pq2, release, debug = libs
    pq2._lib = debug
    try:
        debug.pq2_debug_shrink_bounds(1)
        outs = _run(pq2, debug, name)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_BOUNDS
    finally:
        debug.pq2_debug_shrink_bounds(0)
        pq2._lib = release
    assert _untouched(outs) and _beside(outs)
