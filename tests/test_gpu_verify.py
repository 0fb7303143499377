"""GPU checks of pq2_verify_drafts against the float64 oracle: whole numbers,
equal.  Every case first checks on the oracle's side that no decision lies
within 1e-5 of a tie, where fp32 may decide otherwise (the kernel's p is
within about 4e-6: 2 ulp of the exponential, its argument's rounding, the
sum); exact ties are tested apart, with exactly representable values."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

DEV = "cuda"
MARGIN = 1e-5
SENTINEL = -77


def _problem(lens, V, seed, q=True, temps=None, masked=(), ld=None):
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows, B = int(start[-1]), len(lens)
    logits = (rng.standard_normal((rows, V)) * 2.0).astype(np.float32)
    for b in masked:
        logits[start[b]:start[b + 1], rng.random(V) < 0.5] = -np.inf
    temp = np.full(B, 0.8, dtype=np.float32) if temps is None else np.asarray(temps, np.float32)
    d = logits + 0.8 * rng.standard_normal((rows, V))
    qp = np.zeros((rows, V), dtype=np.float32)
    for b in range(B):
        for r in range(start[b], start[b + 1]):
            t = temp[b] if temp[b] > 0 else 1.0
            w = np.exp((d[r] - d[r].max()) / t) if np.isfinite(d[r]).any() else np.ones(V)
            qp[r] = (w / w.sum()).astype(np.float32)
    drafts = np.array([rng.choice(V, p=qp[r].astype(np.float64) / qp[r].astype(np.float64).sum())
                       if rng.random() < 0.7 else logits[r].argmax() for r in range(rows)],
                      dtype=np.int32)
    return {"logits": logits, "row_start": start, "drafts": drafts, "q": qp if q else None,
            "u": rng.random(rows).astype(np.float32),
            "e": rng.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-9),
            "temperature": temp, "ld": ld}


def _dev(a, ld=None):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    if ld is None or t.dim() < 2:
        return t
    wide = torch.full((t.shape[0], ld), float("nan"), device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _run(pq2, p):
    B, rows, V = len(p["temperature"]), p["logits"].shape[0], p["logits"].shape[1]
    buf_a = torch.full((B + 32,), SENTINEL, dtype=torch.int32, device=DEV)
    buf_t = torch.full((rows + 32,), SENTINEL, dtype=torch.int32, device=DEV)
    ws = pq2.alloc_verify_workspace(B, rows, V)
    ws.fill_(0xA5)
    pq2.pq2_verify_drafts(_dev(p["logits"], p["ld"]), _dev(p["row_start"]), _dev(p["drafts"]),
                          _dev(p["q"], p["ld"]), _dev(p["u"]), _dev(p["e"], p["ld"]),
                          _dev(p["temperature"]), buf_a[16:16 + B], buf_t[16:16 + rows], ws)
    torch.cuda.synchronize()
    a, t = buf_a.cpu().numpy(), buf_t.cpu().numpy()
    for buf, n in ((a, B), (t, rows)):
        assert np.all(buf[:16] == SENTINEL) and np.all(buf[16 + n:] == SENTINEL)
    return a[16:16 + B], t[16:16 + rows]


def _check(p):
    from gemm_pq2_ternary_gb300 import binding as pq2
    acc, tok, margin = step.verify(p["logits"], p["row_start"], p["drafts"], p["q"], p["u"], p["e"],
                                   p["temperature"])
    assert margin > MARGIN, "choose another seed"
    got_a, got_t = _run(pq2, p)
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK
    assert np.array_equal(got_a, acc)
    assert np.array_equal(got_t, tok)


@pytest.mark.parametrize("lens,V,kw", [
    ([4], 248320, {}),
    ([1], 1, {}),
    ([3, 2], 1, {}),
    ([1, 1, 1], 7, {}),
    ([8] * 5, 4096, {}),
    ([5, 1, 3, 2], 4093, {}),
    ([5, 1, 3, 2], 4097, dict(q=False)),
    ([3] * 9, 32003, dict(masked=(1, 4))),
    ([2, 0, 4, 0, 0, 1], 1001, {}),
    ([30, 17], 513, {}),
    ([4] * 6, 8191, dict(temps=[0.0, 1.0, 0.5, 0.0, 2.0, -1.0])),
    ([4] * 6, 8191, dict(temps=[0.0, 1.0, 0.5, 0.0, 2.0, 0.0], q=False, masked=(0, 2))),
    ([2] * 300, 130, {}),
    ([3] * 4, 5000, dict(ld=5008)),
    ([3] * 4, 5000, dict(ld=5003)),
], ids=lambda v: str(v)[:24])
def test_against_the_oracle(lens, V, kw):
    _check(_problem(lens, V, seed=len(lens) * 1000 + V, **kw))


def test_padding_drafts_end_the_sequence():
    p = _problem([4, 4, 4], 999, seed=5)
    p["drafts"][1] = -1
    p["drafts"][4] = 999
    p["drafts"][8] = 2 ** 31 - 1
    p["u"][:] = 0.0          # every real draft with p > 0 is kept
    _check(p)


def test_masked_rows():
    p = _problem([3, 3, 2, 2], 600, seed=6, temps=[0.7, 0.0, 0.7, 0.0])
    p["logits"][[0, 4, 6]] = -np.inf                  # nothing allowed
    p["logits"][7] = np.finfo(np.float32).min         # all at the lowest value: argmax 0
    p["logits"][8, 1:] = np.finfo(np.float32).min     # one allowed token
    p["logits"][8, 0] = 1.0
    _check(p)


def test_lowest_values_are_as_good_as_masked():
    p = _problem([3, 3], 600, seed=7, temps=[0.5, 0.9])
    low = np.finfo(np.float32).min
    p["logits"][:, ::2] = low
    p["logits"][5] = low                              # uniform over the row
    _check(p)


def test_exact_ties_go_to_the_lowest_index():
    from gemm_pq2_ternary_gb300 import binding as pq2
    V = 9000
    p = _problem([3, 2], V, seed=8, temps=[0.0, 1.0], q=False)
    p["logits"][:] = 0.0
    p["logits"][:, [17, 4500, 8999]] = 2.0
    p["drafts"][:] = [17, 4500, 0, 0, 0]
    p["e"][:] = 1.0
    p["u"][:] = 1.0                                   # refuses row 3's draft
    a, t = _run(pq2, p)
    # greedy: 17 kept, 4500 is not the argmax; sampled: three equal scores
    assert list(a) == [1, 0] and list(t) == [17, 17, -1, 17, -1]


def test_equal_probabilities_fall_back_to_the_target():
    # q = p exactly (uniform over a power of two) and a draft refused by u = 1:
    # the residual is zero everywhere, the token comes from p / e
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem([2], 1024, seed=9, temps=[1.0])
    p["logits"][:] = 0.0
    p["q"][:] = 2.0 ** -10
    p["u"][:] = 1.0
    a, t = _run(pq2, p)
    assert a[0] == 0 and t[0] == int(p["e"][0].argmin())


def test_broken_row_ranges_are_reported_and_skipped():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem([2, 2, 2], 100, seed=10)
    good_a, good_t, _ = step.verify(p["logits"], p["row_start"], p["drafts"], p["q"], p["u"],
                                    p["e"], p["temperature"])
    p["row_start"] = np.array([0, 2, 4, 9], dtype=np.int32)   # past the rows
    a, t = _run(pq2, p)
    assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
    assert a[2] == 0 and np.array_equal(a[:2], good_a[:2])
    assert np.array_equal(t[:4], good_t[:4]) and np.all(t[4:] == SENTINEL)


def test_no_rows_at_all():
    from gemm_pq2_ternary_gb300 import binding as pq2
    a = torch.full((3,), 5, dtype=torch.int32, device=DEV)
    z = torch.zeros((0, 50), device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    pq2.pq2_verify_drafts(z, torch.zeros(4, dtype=torch.int32, device=DEV), i, None,
                          torch.zeros(0, device=DEV), torch.ones((3, 50), device=DEV),
                          torch.ones(3, device=DEV), a, i, pq2.alloc_verify_workspace(3, 0, 50))
    torch.cuda.synchronize()
    assert a.tolist() == [0, 0, 0]


def test_first_token_follows_the_target():
    # 4000 sequences of one draft each: the first token's counts against p
    from gemm_pq2_ternary_gb300 import binding as pq2
    n, V = 4000, 6
    rng = np.random.default_rng(11)
    l = np.repeat((rng.standard_normal((1, V)) * 1.5).astype(np.float32), 2 * n, axis=0)
    q0 = rng.dirichlet(np.ones(V)).astype(np.float32)
    p = {"logits": l, "row_start": np.arange(0, 2 * n + 1, 2, dtype=np.int32),
         "drafts": rng.choice(V, 2 * n, p=q0 / q0.sum(dtype=np.float64)).astype(np.int32),
         "q": np.repeat(q0[None], 2 * n, axis=0), "u": rng.random(2 * n).astype(np.float32),
         "e": rng.exponential(size=(n, V)).astype(np.float32),
         "temperature": np.ones(n, dtype=np.float32), "ld": None}
    _, t = _run(pq2, p)
    want = np.exp(l[0].astype(np.float64))
    want /= want.sum()
    got = np.bincount(t[::2], minlength=V)
    assert ((got - n * want) ** 2 / (n * want)).sum() < 35.9   # 5 degrees of freedom: 1e-6


def test_repeated_calls_and_streams_agree():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem([4] * 8, 20011, seed=12)
    first = _run(pq2, p)
    for _ in range(5):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            again = _run(pq2, p)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("V", [1, 3, 5, 2045, 2046, 2047, 2048, 2049, 4094, 4095, 4099])
@pytest.mark.parametrize("ld", [None, 4101, 4102])
def test_row_edges(V, ld):
    # rows that start and end at each offset from 16 bytes
    p = _problem([3, 1, 0, 5], V, seed=V, masked=(3,), temps=[0.7, 0.0, 1.0, 1.3], ld=ld)
    _check(p)


def test_binding_refuses():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem([2, 2], 64, seed=13)
    d = {k: _dev(v) for k, v in p.items() if isinstance(v, np.ndarray)}
    ws = pq2.alloc_verify_workspace(2, 4, 64)
    acc = torch.zeros(2, dtype=torch.int32, device=DEV)
    tok = torch.zeros(4, dtype=torch.int32, device=DEV)

    def call(**kw):
        a = dict(d, accepted=acc, tokens=tok, workspace=ws)
        a.update(kw)
        pq2.pq2_verify_drafts(**a)

    with pytest.raises(ValueError, match="drafts"):
        call(drafts=d["drafts"].long())
    with pytest.raises(ValueError, match="row_start"):
        call(row_start=d["row_start"][:2])
    with pytest.raises(ValueError, match="float32"):
        call(logits=d["logits"].half())
    with pytest.raises(ValueError, match="e: expected shape"):
        call(e=d["e"][:1])
    with pytest.raises(pq2.PQ2Error, match="workspace"):
        call(workspace=ws[:16])


@pytest.mark.parametrize("q", [True, False])
def test_temperatures_at_the_ends_of_their_range(q):
    # infinite: every allowed value alike; tiny, subnormal ones included: the
    # maximum alone
    big, tiny = np.float32(3e38), np.float32(1e-45)
    temps = [np.inf, 1e-40, tiny, big, np.inf, 1e-30]
    for seed in range(5):
        _check(_problem([4] * 6, 3001, seed=40 + seed, temps=temps, q=q))


def test_infinite_temperature_draws_no_masked_value():
    from gemm_pq2_ternary_gb300 import binding as pq2
    p = _problem([3, 2, 4], 2500, seed=50, temps=[np.inf] * 3)
    p["logits"][:, np.random.default_rng(51).random(2500) < 0.5] = -np.inf
    flat = np.where(np.isfinite(p["logits"]), 0.0, -np.inf)   # the same distribution at 1
    acc, tok, margin = step.verify(flat, p["row_start"], p["drafts"], p["q"], p["u"], p["e"], [1.0] * 3)
    assert margin > MARGIN, "choose another seed"
    a, t = _run(pq2, p)
    assert np.array_equal(a, acc) and np.array_equal(t, tok)


def test_no_rows_behind_the_kernel_that_writes_the_ranges():
    # the ranges (all zero) come from a call directly before; what the buffer
    # held until then breaks every rule
    from gemm_pq2_ternary_gb300 import binding as pq2
    n = 40000
    zeros = torch.zeros((1, n), device=DEV)
    ranges = torch.empty((1, n), device=DEV)
    start = ranges.view(torch.int32)[0]
    a = torch.empty(n - 1, dtype=torch.int32, device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    f = torch.zeros(0, device=DEV)
    e, temp, z = torch.ones((n - 1, 1), device=DEV), torch.ones(n - 1, device=DEV), torch.zeros((0, 1), device=DEV)
    ws = pq2.alloc_verify_workspace(n - 1, 0, 1)
    big = torch.zeros(1 << 28, device=DEV)
    for _ in range(5):
        start.fill_(7)
        a.fill_(5)
        torch.cuda.synchronize()
        big.add_(1)              # both calls are queued before the first starts
        pq2.pq2_rmsnorm(zeros, None, ranges)
        pq2.pq2_verify_drafts(z, start, i, None, f, e, temp, a, i, ws)
        assert pq2.pq2_last_device_error() == pq2.PQ2_OK
        assert int(torch.count_nonzero(a)) == 0


def test_a_broken_range_leaves_the_sequences_after_it_alone():
    from gemm_pq2_ternary_gb300 import binding as pq2
    for seed in range(6):
        p = _problem([4, 4], 300, seed=60 + seed)
        p["temperature"] = np.array([3.0, 7.0, 0.5], dtype=np.float32)
        p["e"] = np.random.default_rng(seed).exponential(size=(3, 300)).astype(np.float32)
        p["u"] *= 0.5                        # some drafts are kept
        p["row_start"] = np.array([0, 100, 4, 8], dtype=np.int32)
        want_a, want_t, margin = step.verify(p["logits"], [4, 8], p["drafts"], p["q"], p["u"], p["e"][2:],
                                             p["temperature"][2:])
        assert margin > MARGIN, "choose another seed"
        a, t = _run(pq2, p)
        assert pq2.pq2_last_device_error() == pq2.PQ2_ERR_INVALID_ARG
        assert list(a) == [0, 0, want_a[0]] and np.array_equal(t[4:], want_t[4:])
        assert np.all(t[:4] == SENTINEL)
