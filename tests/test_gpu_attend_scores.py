"""Attention over the 4-bit cache where scores, or the sizes of queries, lie far
apart: finite inputs of any size have their definition's result."""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle.step import TINY, UNIT
from test_gpu_cache4 import TYPES, Cache, _attend, _dev, _np

pytestmark = pytest.mark.gpu

DEV = "cuda"
G, T = 2, 16
# few rows, and many: heads of D values, rows of one sequence
SIZES = [(64, 1), (128, 5), (256, 3), (64, 70), (128, 60), (128, 300), (256, 40)]


@pytest.fixture(scope="module")
def pq2():
    from gemm_pq2_ternary_gb300 import binding
    return binding


def _cache(pq2, k, v):
    """One sequence of keys and values [tokens, D] (one head)."""
    ln, D = k.shape
    c = Cache(pq2, 1, -(-ln // T), 1, D, T)
    k, v = (torch.from_numpy(np.array(a, np.float32)).to(DEV)[:, None].contiguous() for a in (k, v))
    pq2.pq2_cache4_append(k, v, c.pool, c.dev, _dev([0, ln]), _dev([ln]))
    return c


def _held(c, ln):
    """The values as the cache holds them, their parts around code 8, and the rest."""
    code, pair = ref.read_rows(c.pool.cpu().numpy(), c.pages[0], ln, 0, T, c.D)
    s, z = pair[1, :, :1].astype(np.float64), pair[1, :, 1:].astype(np.float64)
    return code[1] * s + z, np.abs((code[1] - 8.0) * s), np.abs(z + 8 * s)


def _close(got, want, mid, rest, keys, dtype):
    # weights to fp16's 11 bits (of the share around code 8), sums of `keys` keys by tiles of
    # 16 cut off at 24 bits, exponentials and quotients by 2^-21, the output's rounding
    tiles = keys / 16 + 16
    bound = mid * 2.0 ** -11 + (mid + rest) * (tiles * 2.0 ** -23 + 2.0 ** -20) + np.abs(want) * UNIT[dtype] + TINY[dtype]
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("at", [3, 64, 300])
@pytest.mark.parametrize("D,n", SIZES)
def test_a_key_far_above_the_others(pq2, D, n, at, dtype):
    # a score past 2^30 behind scores of 0: that key's value, exactly weighed
    ln = at + n + 6
    rng = np.random.default_rng(D + n)
    k = np.zeros((ln, D))
    k[at] = 60000.0
    c = _cache(pq2, k, rng.standard_normal((ln, D)))
    q = torch.full((n, G, D), 60000.0, dtype=TYPES[dtype], device=DEV)
    got = _attend(pq2, c, q, [n], [ln])
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    v, mid, rest = _held(c, ln)
    _close(got, np.broadcast_to(v[at], got.shape), mid[at], rest[at], ln, dtype)


@pytest.mark.parametrize("size", [30.0, 3e3, 4e4])
@pytest.mark.parametrize("D,n", SIZES)
def test_equal_keys_weigh_the_same(pq2, D, n, size):
    # the same large score for all keys: the mean of the values, whatever 32 bits keep of the score
    ln = n + 290
    rng = np.random.default_rng(D + n)
    c = _cache(pq2, np.broadcast_to(1e3 * rng.standard_normal(D), (ln, D)), rng.standard_normal((ln, D)))
    q = torch.from_numpy(np.clip(size * rng.standard_normal((n, G, D)), -6e4, 6e4)).half().to(DEV)
    got = _attend(pq2, c, q, [n], [ln])
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    seen = np.arange(ln - n, ln) + 1
    v, mid, rest = (np.cumsum(a, 0)[seen - 1] / seen[:, None] for a in _held(c, ln))
    _close(got, np.repeat(v[:, None], G, 1), mid[:, None], rest[:, None], ln, "f16")


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,n", SIZES)
def test_scores_past_any_that_stands_for_nothing_seen(pq2, D, n, sign):
    # scores of about +-2^107, all the same
    ln = n + 40
    rng = np.random.default_rng(D + n)
    c = _cache(pq2, np.full((ln, D), -8.0), rng.standard_normal((ln, D)))
    q = torch.full((n, G, D), sign * 2.0 ** 100, dtype=torch.bfloat16, device=DEV)
    got = _attend(pq2, c, q, [n], [ln])
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    seen = np.arange(ln - n, ln) + 1
    v, mid, rest = (np.cumsum(a, 0)[seen - 1] / seen[:, None] for a in _held(c, ln))
    _close(got, np.repeat(v[:, None], G, 1), mid[:, None], rest[:, None], ln, "bf16")


def _unlike(D, n, dtype):
    """Queries of which every third row is small next to its neighbours, keys
    so large that the small rows' scores spread over several units."""
    rng = np.random.default_rng(D + n)
    low, high, scale = (2.0 ** -10, 2.0 ** 13, D ** -0.5) if dtype == "f16" else (2.0 ** -20, 2.0 ** 20, 2.0 ** 10 * D ** -0.5)
    size = np.array([low, 1.0, high])[(np.arange(n * G) * 2 % 3)].reshape(n, G, 1)
    q = torch.from_numpy(rng.standard_normal((n, G, D)) * size).to(TYPES[dtype])
    ln = n + 60
    k = rng.standard_normal((ln, D)) * (2.0 / (low * scale * D ** 0.5))
    return q, k, rng.standard_normal((ln, D)), scale, (size == low)[..., 0]


def _bound(q, pool, pages, n, ln, scale, dtype):
    want, tol = ref.attend(_np(q), pool, pages, [0, n], [ln], T, scale)
    return want, tol + np.abs(want) * UNIT[dtype] + TINY[dtype]


def _rounded(q, step):
    """q with all values of all rows to whole steps of `step` times the largest."""
    step = step * float(q.float().abs().max())
    return torch.round(q.double() / step) * step


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n", SIZES)
def test_rows_keep_what_they_have_next_to_larger_ones(pq2, D, n, dtype):
    q, k, v, scale, small = _unlike(D, n, dtype)
    c = _cache(pq2, k, v)
    ln = len(k)
    got = _attend(pq2, c, q.to(DEV), [n], [ln], scale=scale).double().cpu().numpy()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    pool = c.pool.cpu().numpy()
    want, bound = _bound(q, pool, c.pages, n, ln, scale, dtype)
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound)[small].max())
    # what one step for all rows would do is far outside the bound of the small ones
    if n > 1:
        coarse, _ = ref.attend(_rounded(q, 2.0 ** -18).numpy(), pool, c.pages, [0, n], [ln], T, scale)
        assert np.any((np.abs(coarse - want) > 4 * bound)[small])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n", [(64, 60), (128, 60), (256, 40)])
def test_a_row_does_not_depend_on_the_rows_after_it(pq2, D, n, dtype):
    # the first rows' queries stay, the others' grow: the same bits for the first
    rng = np.random.default_rng(D)
    ln = n + 70
    c = _cache(pq2, rng.standard_normal((ln, D)), rng.standard_normal((ln, D)))
    q = torch.from_numpy(rng.standard_normal((n, G, D))).to(TYPES[dtype]).to(DEV)
    grown = q.clone()
    grown[n // 3:] *= 2.0 ** 12
    one, two = (_attend(pq2, c, x, [n], [ln]) for x in (q, grown))
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    assert torch.equal(one[:n // 3], two[:n // 3])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n", [(64, 4), (64, 23), (128, 5), (128, 24), (256, 3), (256, 16), (64, 70), (128, 60), (128, 300),
                                 (256, 40)])
@pytest.mark.parametrize("before", [0, 150])
def test_rows_do_not_feel_values_that_they_do_not_see(pq2, D, n, before, dtype):
    # small values, then huge ones from the middle of the rows on: earlier rows keep what they have
    ln = before + n
    cut = before + n // 2
    rng = np.random.default_rng(D + n)
    size = np.where(np.arange(ln) < cut, 2.0 ** -12, 3e5)[:, None]
    c = _cache(pq2, rng.standard_normal((ln, D)), rng.standard_normal((ln, D)) * size)
    q = torch.from_numpy(rng.standard_normal((n, G, D))).to(TYPES[dtype]).to(DEV)
    got = _attend(pq2, c, q, [n], [ln]).double().cpu().numpy()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    want, bound = _bound(q, c.pool.cpu().numpy(), c.pages, n, ln, D ** -0.5, dtype)
    fits = np.abs(want) < (6e4 if dtype == "f16" else 1e30)     # (outputs that the type can hold)
    assert fits[:n // 2].all()
    worst = (np.abs(got - want) / bound)[fits]
    assert np.all(worst <= 1), float(worst.max())


@pytest.mark.parametrize("window", [0, 1, 13, 90])
@pytest.mark.parametrize("size", [1.0, 300.0])
@pytest.mark.parametrize("D,n", [(64, 4), (64, 23), (128, 5), (128, 24), (256, 3), (256, 16), (64, 70), (128, 60), (128, 300),
                                 (256, 40)])
def test_values_of_very_different_size(pq2, D, n, size, window):
    # tokens' values from 2^-14 to 2^12 in any order, behind and among the rows, with windows that leave
    # some of them to some of the rows
    ln = n + 230
    rng = np.random.default_rng(D + n)
    c = _cache(pq2, rng.standard_normal((ln, D)), rng.standard_normal((ln, D)) * 2.0 ** rng.uniform(-14, 12, (ln, 1)))
    q = torch.from_numpy(size * rng.standard_normal((n, G, D))).half().to(DEV)
    got = _attend(pq2, c, q, [n], [ln], window).double().cpu().numpy()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    want, tol = ref.attend(_np(q), c.pool.cpu().numpy(), c.pages, [0, n], [ln], T, D ** -0.5, window)
    bound = tol + np.abs(want) * UNIT["f16"] + TINY["f16"]
    worst = np.abs(got - want) / bound
    assert np.all(worst <= 1), float(worst.max())
