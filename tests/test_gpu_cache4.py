"""The cache in 4 bits on the GPU: appended rows to the bit, read back to the
bit, and attention over it against float64 within derived bounds."""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle.step import TINY, UNIT

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _np(t):
    return t.detach().float().cpu().numpy()


class Cache:
    """A pool with its table; pages in any order, the unused ones full of
    bytes that no value has (scales that are NaN)."""

    def __init__(self, pq2, B, W, H, D, T, seed=0, spare=2, page_pad=0):
        rng = np.random.default_rng(seed)
        self.T, self.D, self.H = T, D, H
        P = B * W + spare
        nbytes = pq2.pq2_cache4_page_bytes(H, D, T)
        self.raw = torch.full((P, nbytes + page_pad), 0xFF, dtype=torch.uint8, device=DEV)
        self.pool = self.raw[:, :nbytes].unflatten(1, (H, T * (D + 8)))
        self.pages = rng.permutation(P)[:B * W].reshape(B, W).astype(np.int32)
        self.dev = _dev(self.pages)

    def fill(self, lens, seed=1, spread=1.0):
        """Random rows for all tokens of the sequences, written by the oracle."""
        rng = np.random.default_rng(seed)
        pool = self.pool.cpu().numpy().copy()
        for b, ln in enumerate(lens):
            for h in range(self.H):
                if ln <= 0:
                    continue
                x = rng.standard_normal((2, ln, self.D)) * spread + 0.3 * rng.standard_normal((2, 1, self.D))
                x[1] *= rng.uniform(0.2, 3.0, (ln, 1))
                c, s, z = ref.quantise(x.astype(np.float32))
                for t in range(ln):
                    for value in range(2):
                        ref.write_row(pool, self.pages[b, t // self.T], h, t % self.T, self.T, self.D, value,
                                      c[value, t], s[value, t, 0], z[value, t, 0])
        self.pool.copy_(torch.from_numpy(pool).to(DEV))
        return pool


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


@pytest.mark.parametrize("Hq,H,D,T,rot", [(6, 2, 64, 16, 64), (4, 4, 128, 32, 128), (3, 1, 128, 16, 20), (8, 2, 256, 64, 64),
                                          (0, 3, 64, 48, 0), (5, 5, 256, 16, 34)])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("xt,yt", [("f32", "f16"), ("bf16", "bf16")])
def test_append_and_read_to_the_bit(pq2, Hq, H, D, T, rot, near, xt, yt):
    n = [3, 0, 1, 20, 1]
    lens = np.array([3, 5, 17, 40, 16])
    M, W = sum(n) + 3, 4                               # three rows of padding
    g = torch.Generator(device=DEV).manual_seed(D + rot)
    x = (torch.randn((M, Hq + 2 * H, D), generator=g, device=DEV) * 2).to(TYPES[xt])
    x[0, Hq] = 0.0                                     # a row of zeros
    x[1, Hq + H] = 1.5                                 # and one of one value
    x[2, Hq] *= 1e-6
    x[3, Hq + H] *= 3e4
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    c = Cache(pq2, len(n), W, H, D, T, seed=3, page_pad=32)
    before = c.pool.cpu().numpy().copy()
    table = torch.zeros((50, rot // 2, 2), device=DEV)
    if rot:
        pq2.pq2_rope_table(table, 1e4)
    q_out = torch.full((M, Hq, D), 9.0, dtype=TYPES[yt], device=DEV)
    start = _starts(n)
    args = dict(pages=c.dev, row_start=_dev(start), lens=_dev(lens))
    pq2.pq2_cache4_append(k, v, c.pool, **args, q=q if Hq else None, q_out=q_out if Hq else None,
                          table=table if rot else None, flags=pq2.PQ2_ROPE_NEIGHBOURS if near else 0)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    want = before.copy()
    k_out = torch.full((M, H, D), 8.0, dtype=TYPES[yt], device=DEV)
    v_out = torch.full((M, H, D), 8.0, dtype=TYPES[yt], device=DEV)
    pq2.pq2_cache4_read(c.pool, c.dev, args["row_start"], args["lens"], k_out, v_out)
    for b in range(len(n)):
        for i in range(n[b]):
            m, pos = start[b] + i, lens[b] - n[b] + i
            cs = table[pos:pos + 1].cpu().numpy()
            turned = ref.turn(_np(x[m:m + 1]), cs, rot, near)[0]
            for h in range(Hq):
                assert torch.equal(q_out[m, h].cpu(), torch.from_numpy(turned[h]).to(TYPES[yt]))
            for h in range(H):
                for value, row, out in ((0, turned[Hq + h], k_out), (1, _np(v[m, h]), v_out)):
                    code, s, z = ref.quantise(row)
                    ref.write_row(want, c.pages[b, pos // T], h, pos % T, T, D, value, code, s[0], z[0])
                    assert torch.equal(out[m, h].cpu(), torch.from_numpy(ref.dequantise(code, s, z)).to(TYPES[yt]))
    assert np.array_equal(c.pool.cpu().numpy(), want)
    assert torch.all(c.raw[:, c.raw.shape[1] - 32:] == 0xFF)
    for t in (q_out, k_out, v_out):                    # padding is left as it was
        assert torch.all(t[M - 3:] == (9.0 if t is q_out else 8.0))


def test_append_in_place_with_positions(pq2):
    # the queries turned in place, angles at positions other than the places
    M, Hq, H, D, T = 9, 4, 1, 128, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn((M, Hq + 2 * H, D), generator=g, device=DEV)
    want = x.clone()
    table = torch.zeros((64, D // 2, 2), device=DEV)
    pq2.pq2_rope_table(table, 1e4)
    pos = torch.randint(0, 64, (M,), device=DEV, dtype=torch.int32)
    pq2.pq2_rope(want[:, :Hq + H], table, pos, want[:, :Hq + H])
    c = Cache(pq2, 1, 1, H, D, T)
    q = x[:, :Hq]
    pq2.pq2_cache4_append(x[:, Hq:Hq + H], x[:, Hq + H:], c.pool, c.dev, _dev([0, M]), _dev([M]), q=q, q_out=q,
                          table=table, positions=pos)
    assert torch.equal(x[:, :Hq], want[:, :Hq])
    k = torch.empty((M, H, D), device=DEV)
    pq2.pq2_cache4_read(c.pool, c.dev, _dev([0, M]), _dev([M]), k, None)
    code, s, z = ref.quantise(_np(want[:, Hq:Hq + H]))
    assert np.array_equal(_np(k), ref.dequantise(code, s, z))


def test_append_outside_the_cache(pq2):
    # a page outside the pool, a position below 0 and one behind the table: skipped and reported
    H, D, T, W = 1, 64, 16, 2
    c = Cache(pq2, 3, W, H, D, T)
    pages = c.pages.copy()
    pages[0, 0] = 10 ** 6
    x = torch.randn((6, 1, D), device=DEV)
    before = c.pool.clone()
    for n, lens in (([2, 0, 0], [2, 0, 0]), ([0, 3, 0], [0, 1, 0]), ([0, 0, 2], [0, 0, 33])):
        start = _starts(n)
        c.pool.copy_(before)
        pq2.pq2_cache4_append(x, x, c.pool, _dev(pages), _dev(start), _dev(lens))
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
        written = (c.pool != before).any(-1).any(-1).nonzero().flatten().tolist()
        want = {0: [], 1: [pages[1, 0]], 2: [pages[2, 1]]}[int(np.argmax(n))]
        assert written == want


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def _attend(pq2, c, q, n, lens, window=0, max_rows=0, scale=None, out=None, workspace=None):
    M, Hq, D = q.shape
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    if workspace is None:
        workspace = pq2.alloc_attend_workspace(M, Hq, c.H, D).fill_(0xFF)
    pq2.pq2_cache4_attend(q, c.pool, c.dev, _dev(_starts(n)), _dev(lens), out, workspace, window=window,
                          max_rows=max_rows, scale=scale)
    return out


def _check(got, q, pool, c, n, lens, window=0, scale=None, dtype="f16"):
    want, tol = ref.attend(_np(q), pool, c.pages, _starts(n), lens, c.T, c.D ** -0.5 if scale is None else scale, window)
    M = sum(n)
    err = np.abs(got.double().cpu().numpy() - want)[:M]
    bound = (tol + np.abs(want) * UNIT[dtype] + TINY[dtype])[:M]
    assert np.all(err <= bound), float((err / bound).max())


def _q(M, Hq, D, dtype, seed=0, scale=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((M, Hq, D), generator=g, device=DEV) * scale).to(TYPES[dtype])


LAYOUTS = [(1, 1, 64, 16), (8, 2, 64, 32), (6, 1, 128, 16), (10, 2, 128, 48), (12, 2, 256, 64), (7, 7, 128, 16),
           (24, 1, 64, 16), (16, 1, 256, 128)]


@pytest.mark.parametrize("Hq,H,D,T", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 21])
def test_single_tokens(pq2, Hq, H, D, T, dtype, window):
    lens = [1, 15, 16, 17, 33, 200, 2, 129]
    n = [1] * len(lens)
    c = Cache(pq2, len(lens), -(-max(lens) // T), H, D, T, seed=D)
    pool = c.fill(lens)
    q = _q(len(lens), Hq, D, dtype)
    got = _attend(pq2, c, q, n, lens, window, max_rows=1)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, pool, c, n, lens, window, dtype=dtype)


@pytest.mark.parametrize("Hq,H,D,T", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 21])
def test_ragged_rows(pq2, Hq, H, D, T, dtype, window):
    # no rows, no tokens, fewer tokens than rows (rows that see nothing), and padding
    n = [3, 0, 1, 37, 5, 2, 0]
    lens = [3, 9, 77, 150, 2, 0, 0]
    c = Cache(pq2, len(lens), -(-max(lens) // T), H, D, T, seed=D)
    pool = c.fill(lens)
    q = _q(sum(n) + 2, Hq, D, dtype)
    got = _attend(pq2, c, q, n, lens, window)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    _check(got, q, pool, c, n, lens, window, dtype=dtype)
    assert torch.all(got[sum(n):] == 7.0)
    m = sum(n[:4])
    assert torch.all(got[m:m + 3] == 0.0) and torch.all(got[m + 5:m + 7] == 0.0)


@pytest.mark.parametrize("Hq,H,D,T,n,ln", [(8, 1, 128, 16, 1, 5000), (6, 1, 256, 64, 1, 9001), (2, 2, 64, 16, 3, 4001),
                                           (5, 1, 128, 32, 7, 3001), (4, 1, 64, 16, 130, 2100), (2, 1, 256, 16, 300, 1111),
                                           (12, 2, 128, 32, 64, 640), (40, 2, 64, 16, 33, 500)])
def test_long_ones(pq2, Hq, H, D, T, n, ln):
    c = Cache(pq2, 1, -(-ln // T), H, D, T, seed=D)
    pool = c.fill([ln])
    for dtype in ("f16", "bf16"):
        q = _q(n, Hq, D, dtype)
        _check(_attend(pq2, c, q, [n], [ln], max_rows=n), q, pool, c, [n], [ln], dtype=dtype)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK


@pytest.mark.parametrize("n", [1, 40])
def test_large_and_small_numbers(pq2, n):
    # scores of hundreds (a weight of 1 and the rest 0), tiny values, tiny queries
    c = Cache(pq2, 1, 20, 1, 128, 16)
    for spread, scale in ((30.0, None), (1e-3, None), (1.0, 0.0), (1.0, -0.3), (200.0, 1e-4)):
        pool = c.fill([310], spread=spread)
        q = _q(n, 4, 128, "bf16", scale=8.0)
        _check(_attend(pq2, c, q, [n], [310], scale=scale), q, pool, c, [n], [310], scale=scale, dtype="bf16")
        q = _q(n, 4, 128, "f16", scale=1e-5)
        _check(_attend(pq2, c, q, [n], [310], scale=scale), q, pool, c, [n], [310], scale=scale)


@pytest.mark.parametrize("n", [1, 50])
def test_values_of_one_size(pq2, n):
    # rows of one value (scale 0): the result is their weighted mean, offsets alone
    D, T = 128, 16
    c = Cache(pq2, 1, 8, 1, D, T)
    ln = 100
    x = torch.arange(ln, device=DEV).float()[:, None, None].expand(ln, 1, D).contiguous() / 16
    pq2.pq2_cache4_append(torch.zeros_like(x), x, c.pool, c.dev, _dev([0, ln]), _dev([ln]))
    q = _q(n, 3, D, "f16")
    got = _attend(pq2, c, q, [n], [ln])
    want = [(p / 32) for p in range(ln - n, ln)]
    assert np.allclose(_np(got), np.array(want)[:, None, None], rtol=2.0 ** -10, atol=0)


@pytest.mark.parametrize("n", [1, 30])
def test_strides_and_slices(pq2, n):
    Hq, H, D, T, ln = 6, 2, 128, 32, 90
    c = Cache(pq2, 1, 3, H, D, T, page_pad=64)
    pool = c.fill([ln])
    wide = _q(n, Hq + 3, 2 * D, "f16")
    q = wide[:, 1:1 + Hq, D:]
    out = torch.full((n + 1, Hq + 1, D + 8), 7.0, dtype=torch.float16, device=DEV)
    _attend(pq2, c, q, [n], [ln], out=out[:n, :Hq, :D])
    _check(out[:n, :Hq, :D], q, pool, c, [n], [ln])
    assert torch.all(out[n:] == 7.0) and torch.all(out[:, Hq:] == 7.0) and torch.all(out[..., D:] == 7.0)


def test_pages_far_apart(pq2):
    # places past 2^31 and 2^32 bytes
    Hq, H, D, T = 4, 1, 128, 16
    nbytes = pq2.pq2_cache4_page_bytes(H, D, T)
    raw = torch.zeros(5 * (1 << 30) + nbytes, dtype=torch.uint8, device=DEV)
    c = Cache(pq2, 1, 6, H, D, T, spare=0)
    pool = c.fill([93])
    far = torch.as_strided(raw, (6, H, nbytes), (1 << 30, nbytes, 1))
    far.copy_(c.pool)
    for n in (1, 40):
        q = _q(n, Hq, D, "f16")
        near_out = _attend(pq2, c, q, [n], [93])
        c.pool, keep = far, c.pool
        got = _attend(pq2, c, q, [n], [93])
        c.pool = keep
        assert torch.equal(got, near_out)
        _check(got, q, pool, c, [n], [93])


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_lengths(pq2, n):
    Hq, H, D, T = 4, 2, 64, 16
    lens = [80, 80, 80]
    c = Cache(pq2, 3, 5, H, D, T)
    pool = c.fill(lens)
    q = _q(3 * n, Hq, D, "f16")
    good = _attend(pq2, c, q, [n] * 3, lens, max_rows=n)
    _check(good, q, pool, c, [n] * 3, lens)
    for bad in (-1, 17, 2 ** 31 - 1):
        c.dev[1, 2] = bad
        got = _attend(pq2, c, q, [n] * 3, lens, max_rows=n)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
        for b in (0, 2):                               # the others are as they were
            assert torch.equal(got[b * n:(b + 1) * n], good[b * n:(b + 1) * n])
    c.dev[1, 2] = int(c.pages[1, 2])
    for ln in (81, 2 ** 31 - 1, -5):
        got = _attend(pq2, c, q, [n] * 3, [80, ln, 80], max_rows=n)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
        _check(got[:n], q[:n], pool, c, [n], [80])
    # more rows than max_rows, and rows past M
    c2 = c.dev
    c.dev = c.dev[:2].contiguous()
    got = _attend(pq2, c, q, [n, 2 * n], [80, 80], max_rows=n)
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    _check(got[:n], q[:n], pool, c, [n], [80])
    assert torch.all(got[n:] == 7.0)
    c.dev = c2


@pytest.mark.parametrize("n", [1, 3, 70])
def test_graphs_streams_and_one_workspace(pq2, n):
    Hq, H, D, T = 8, 2, 128, 16
    lens = [300, 41, 128]
    c = Cache(pq2, 3, 19, H, D, T)
    c.fill(lens)
    ws = pq2.alloc_attend_workspace(3 * n, Hq, H, D)
    qs = [_q(3 * n, Hq, D, "f16", seed=s) for s in (1, 2)]
    want = [_attend(pq2, c, q, [n] * 3, lens, max_rows=n) for q in qs]
    start, ld = _dev(_starts([n] * 3)), _dev(lens)
    outs, graphs = [torch.empty_like(q) for q in qs], []
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq2.pq2_cache4_attend(q, c.pool, c.dev, start, ld, o, ws, max_rows=n)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)               # the same bits every time
    side = [torch.cuda.Stream() for _ in range(2)]
    spaces = [pq2.alloc_attend_workspace(3 * n, Hq, H, D) for _ in range(2)]
    torch.cuda.synchronize()
    for s, q, o, w in zip(side, qs, outs, spaces):
        for _ in range(5):
            pq2.pq2_cache4_attend(q, c.pool, c.dev, start, ld, o, w, max_rows=n, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_many_sequences(pq2):
    # more sequences than lanes and CTAs, lengths of all sizes, one of them empty
    Hq, H, D, T, B = 4, 2, 64, 16, 777
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 60, B)
    n = np.minimum(lens, 1)
    c = Cache(pq2, B, 4, H, D, T)
    pool = c.fill(lens)
    q = _q(int(n.sum()), Hq, D, "bf16")
    got = _attend(pq2, c, q, n, lens, max_rows=1)
    _check(got, q, pool, c, n, lens, dtype="bf16")
    n = np.minimum(lens, rng.integers(0, 7, B))
    q = _q(int(n.sum()), Hq, D, "bf16")
    got = _attend(pq2, c, q, n, lens, max_rows=6)
    _check(got, q, pool, c, n, lens, dtype="bf16")


@pytest.mark.parametrize("n", [1, 24])
def test_append_attend_and_cut_back(pq2, n):
    """A run of them together: a prompt, drafts, some refused, a fork, then
    the pages moved together; the attention sees what a plain cache would."""
    Hq, H, D, T, W = 4, 2, 64, 16, 12
    B, P = 3, 40
    pool = pq2.alloc_cache4(P, H, D, T)
    pages = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    lens = np.zeros(B, int)
    hist = [np.zeros((2, 0, H, D), np.float32) for _ in range(B)]
    table = torch.zeros((W * T, D // 2, 2), device=DEV)
    pq2.pq2_rope_table(table, 1e4)
    ws = pq2.alloc_pages_workspace(B, P)
    wa = pq2.alloc_attend_workspace(B * 40, Hq, H, D)
    g = torch.Generator(device=DEV).manual_seed(n)
    steps = [((0, -1, -1), (0, 0, 0), (37, 0, 0)), ((0, 0, -1), (37, 37, 0), (n, n, 5)),
             ((0, 1, 1), (37 + n - 1, 20, 16), (n, n, n)), ((2, -1, 0), None, (2, 1, n))]
    for step, (source, keep, new) in enumerate(steps):
        if keep is None:
            keep = [int(lens[max(s, 0)]) if s >= 0 else 0 for s in source]
        kept = np.array([min(k, lens[s]) if s >= 0 else 0 for s, k in zip(source, keep)])
        after = kept + np.array(new)
        out, ro = torch.empty_like(pages), torch.empty_like(refs)
        copies = torch.empty((B, 2), dtype=torch.int32, device=DEV)
        info = torch.empty(2, dtype=torch.int32, device=DEV)
        pq2.pq2_pages_update(pages, refs, _dev(lens), _dev(source), _dev(keep), _dev(after), T, out, ro, copies, info, ws)
        pq2.pq2_pages_copy(pool, copies)
        assert int(info[1]) == 0
        pages, refs = out, ro
        if step == 3:
            out, ro = torch.empty_like(pages), torch.empty_like(refs)
            moves = torch.empty((P // 2, 2), dtype=torch.int32, device=DEV)
            pq2.pq2_pages_compact(pages, refs, _dev(after), T, out, ro, moves, info, ws)
            pq2.pq2_pages_copy(pool, moves)
            pages, refs = out, ro
            assert int(pages.max()) < int(info[0])
        M = int(sum(new))
        x = torch.randn((M, Hq + 2 * H, D), generator=g, device=DEV)
        q = torch.empty((M, Hq, D), dtype=torch.float16, device=DEV)
        start = _dev(_starts(new))
        pq2.pq2_cache4_append(x[:, Hq:Hq + H], x[:, Hq + H:], pool, pages, start, _dev(after), q=x[:, :Hq], q_out=q,
                              table=table)
        got = torch.empty_like(q)
        pq2.pq2_cache4_attend(q, pool, pages, start, _dev(after), got, wa)
        k, v = (torch.empty((M, H, D), device=DEV) for _ in range(2))
        pq2.pq2_cache4_read(pool, pages, start, _dev(after), k, v)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        rows = np.stack([_np(k), _np(v)])
        s0 = _starts(new)
        hist = [np.concatenate([hist[s][:, :kept[b]] if s >= 0 else np.zeros((2, 0, H, D), np.float32),
                                rows[:, s0[b]:s0[b + 1]]], 1) for b, s in enumerate(source)]
        lens = after
        for b in range(B):
            for i in range(new[b]):
                pos = lens[b] - new[b] + i
                for h in range(Hq):
                    kk, vv = hist[b][0, :pos + 1, h // 2].astype(np.float64), hist[b][1, :pos + 1, h // 2].astype(np.float64)
                    y = kk @ _np(q[s0[b] + i, h]).astype(np.float64) * D ** -0.5
                    w = np.exp(y - y.max())
                    w /= w.sum()
                    want = w @ vv
                    # weights to 2^-11, codes within 8 scales of their middle (at most the row's range), fp16
                    tol = (w @ np.ptp(vv, axis=1)) * 2.0 ** -10 + np.abs(want) * 2.0 ** -11 + 2.0 ** -16
                    assert np.all(np.abs(_np(got[s0[b] + i, h]) - want) <= tol)
