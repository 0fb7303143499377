"""The pages of a cache between two steps: updates, compaction and copies
against plain loops (whole numbers, equal)."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _state(rng, B, W, T, P, share=True):
    """A sound table: every sequence its own pages, some first pages shared."""
    lens = rng.integers(0, W * T + 1, B)
    pages = np.full((B, W), -1)
    refs = np.zeros(P, np.int64)
    free = list(rng.permutation(P))
    for b in range(B):
        n = -(-lens[b] // T)
        if n > len(free):
            lens[b] = len(free) * T
            n = len(free)
        pages[b, :n] = [free.pop() for _ in range(n)]
        refs[pages[b, :n]] += 1
    if share:
        for b in range(1, B, 2):
            k = min(lens[b], lens[b - 1]) // T // 2
            refs[pages[b, :k]] -= 1
            pages[b, :k] = pages[b - 1, :k]
            refs[pages[b, :k]] += 1
        for p in rng.integers(0, P, 3):  # kept from outside
            refs[p] += 1
    return pages, lens, refs


def _update(pq2, pages, lens, refs, source, keep, new, T, pad=0, in_place=True):
    B, W = pages.shape
    wide = np.full((B, W + pad), 77)
    wide[:, :W] = pages
    pd = _dev(wide)[:, :W]
    out = torch.full((B, W + pad), 55, dtype=torch.int32, device=DEV)
    r = _dev(refs)
    ro = r if in_place else torch.full_like(r, 99)
    copies = torch.full((B, 2), 88, dtype=torch.int32, device=DEV)
    info = torch.full((2,), 88, dtype=torch.int32, device=DEV)
    ws = pq2.alloc_pages_workspace(B, len(refs)).fill_(0xAB)
    pq2.pq2_pages_update(pd, r, _dev(lens), _dev(source), _dev(keep), _dev(new), T, out[:, :W], ro, copies, info, ws)
    assert pad == 0 or torch.all(out[:, W:] == 55)
    return [t.cpu().numpy() for t in (out[:, :W], ro, copies, info)]


def _same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w), (g, w)


@pytest.mark.parametrize("B,W,T,P", [(1, 1, 16, 1), (3, 5, 16, 11), (40, 9, 32, 300), (7, 64, 16, 500), (300, 3, 64, 700),
                                     (2, 2, 1, 9), (33, 40, 128, 20000), (1, 4, 16, 40000)])
def test_update(pq2, B, W, T, P):
    rng = np.random.default_rng(B + P)
    for trial in range(6):
        pages, lens, refs = _state(rng, B, W, T, P)
        source = np.where(rng.random(B) < 0.6, np.arange(B), rng.integers(-1, B, B))
        keep = np.maximum(lens[source] - rng.integers(0, 2 * T + 2, B), 0)
        if trial % 2:
            keep = rng.integers(0, W * T + 1, B)
        new = np.minimum(keep + rng.integers(0, 2 * T, B), W * T)
        if trial == 4:
            source[:] = 0                       # all fork from one
        if trial == 5:
            source[:], new[:] = -1, 0           # all end
        got = _update(pq2, pages, lens, refs, source, keep, new, T, pad=trial % 3, in_place=trial % 2 == 0)
        _same(got, ref.pages_update(pages, lens, refs, source, keep, new, T))
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        if trial == 5:
            held = np.zeros(P, int)
            np.add.at(held, pages[pages >= 0], 1)
            assert np.array_equal(got[1], np.maximum(refs - held, 0))


def test_update_without_enough_pages(pq2):
    pages, lens, refs = np.array([[2, -1, -1], [0, 1, -1]]), [16, 32], [1, 1, 1, 0]
    args = (pages, lens, np.array(refs), [0, 1], [10, 32], [48, 48], 16)
    got = _update(pq2, *args)
    _same(got, ref.pages_update(*args))
    assert got[3].tolist() == [0, 2] and got[0].tolist() == [[2, 3, -1], [0, 1, -1]]


def test_update_with_values_out_of_range(pq2):
    pages = np.array([[1, 99, -5], [0, 2, 3], [4, 5, 6]])
    args = (pages, [48, 1000, -3], np.ones(9, int), [1, 7, 0], [-2, 10, 40], [16, 9999, 48], 16)
    got = _update(pq2, *args)
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    _same(got, ref.pages_update(*args))


def test_update_of_nothing(pq2):
    z = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    r, e = _dev([3, 0, 0]), torch.zeros(0, dtype=torch.int32, device=DEV)
    info = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    pq2.pq2_pages_update(z, r, e, e, e, e, 16, torch.empty_like(z), r, torch.zeros((0, 2), dtype=torch.int32, device=DEV),
                         info, pq2.alloc_pages_workspace(0, 3))
    assert info.tolist() == [2, 0] and r.tolist() == [3, 0, 0]


@pytest.mark.parametrize("B,W,T,P", [(1, 1, 16, 1), (5, 6, 16, 40), (40, 9, 32, 800), (3, 50, 16, 20000), (1, 3, 16, 2)])
def test_compact(pq2, B, W, T, P):
    rng = np.random.default_rng(B + P)
    for trial in range(4):
        pages, lens, refs = _state(rng, B, W, T, P)
        for b in np.nonzero(rng.random(B) < 0.5)[0]:
            n = -(-lens[b] // T)
            refs[pages[b, :n]] -= 1
            pages[b], lens[b] = -1, 0
        want = ref.pages_compact(pages, lens, refs, T)
        r = _dev(refs)
        ro = r if trial % 2 else torch.full_like(r, 77)
        pd = _dev(pages)
        po = pd if trial == 3 else torch.full_like(pd, 77)
        copies = torch.full((P // 2, 2), 88, dtype=torch.int32, device=DEV)
        info = torch.full((2,), 88, dtype=torch.int32, device=DEV)
        pq2.pq2_pages_compact(pd, r, _dev(lens), T, po, ro, copies, info, pq2.alloc_pages_workspace(B, P).fill_(0xCD))
        _same([t.cpu().numpy() for t in (po, ro, copies, info)], want)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK


@pytest.mark.parametrize("nbytes", [16, 1152, 8192, 8208, 100000])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_copy(pq2, nbytes, layers):
    P, n = 37, 23
    rng = np.random.default_rng(nbytes)
    shape = (max(layers, 1), P + 1, nbytes + 48)
    pool = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).to(DEV)
    view = pool[:, :P, 16:16 + nbytes]
    order = rng.permutation(P)
    pairs = np.full((n, 2), -1)
    pairs[::2] = order[:24].reshape(12, 2)
    pairs[1] = 4, -1
    pairs[3] = -7, 5
    want = pool.clone()
    for a, b in pairs:
        if a >= 0 and b >= 0:
            want[:, b, 16:16 + nbytes] = want[:, a, 16:16 + nbytes]
    if layers:
        pq2.pq2_pages_copy(view, _dev(pairs), layers=True)
    else:
        pq2.pq2_pages_copy(view[0], _dev(pairs))
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    assert torch.equal(pool, want)
    pairs[:, :] = -1
    pairs[5] = 0, P
    pq2.pq2_pages_copy(view[0], _dev(pairs))
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    assert torch.equal(pool, want)


def test_far_pages(pq2):
    # places past 2^31 and 2^32 bytes
    pool = torch.zeros(5 * (1 << 30) + 4096, dtype=torch.uint8, device=DEV)
    view = torch.as_strided(pool, (6, 4096), (1 << 30, 1))
    view[1] = 7
    view[5] = 9
    pq2.pq2_pages_copy(view, _dev([[1, 4], [5, 0]]))
    assert torch.all(view[4] == 7) and torch.all(view[0] == 9) and torch.all(view[3] == 0)


def test_graph_with_another_step(pq2):
    # one workspace, two captured graphs, replayed in turn
    rng = np.random.default_rng(1)
    B, W, T, P = 8, 6, 16, 80
    ws = pq2.alloc_pages_workspace(B, P)
    graphs = []
    for k in range(2):
        pages, lens, refs = _state(rng, B, W, T, P)
        source, keep = np.roll(np.arange(B), k), np.maximum(lens - 3, 0)
        new = np.minimum(keep + 9, W * T)
        d = [_dev(a) for a in (pages, refs, lens, source, keep, new)]
        out = [torch.zeros((B, W), dtype=torch.int32, device=DEV), torch.zeros(P, dtype=torch.int32, device=DEV),
               torch.zeros((B, 2), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)]
        pq2.pq2_pages_update(*d, T, *out, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq2.pq2_pages_update(*d, T, *out, ws)
        graphs.append((g, out, ref.pages_update(pages, lens, refs, source, keep, new, T), d))
    for _ in range(3):
        for g, out, _, _ in graphs:
            for t in out:
                t.fill_(-9)
            g.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in graphs:
            _same([t.cpu().numpy() for t in out], want)
