"""The steps around the ternary projections of a serving step, as cases to measure.

Three sets of operators:
  norm    RMS norms before and after a block, with the block's gate, residual
          scale and residual add (pq2_rmsnorm, pq2_norm_residual)
  lora    low-rank adapters of many requests beside a shared projection
          (pq2_lora_add)
  verify  drafted tokens against the target's probabilities, from given
          random numbers (pq2_verify_drafts)

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the library's entry points.  Sizes are those of the library's
projections (5120, 6144, 17408, a vocabulary of 248320) and generic ones.
"""
import torch

own = False

DEV = "cuda"
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6

_pq2 = None


def _lib():
    global _pq2
    if _pq2 is None:
        from gemm_pq2_ternary_gb300 import binding
        _pq2 = binding
    return _pq2


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _norm(M, H, post, next_, gate, r, x, name=None):
    # post: the block's output is normed; next_: the next block's norm follows;
    # gate: "none", "layer" (one [H] vector), "sigmoid" or "silu" (per token,
    # one half of a fused [M, 2H] projection output); r, x: element types
    c = {"op": "norm", "M": M, "H": H, "post": post, "next": next_, "gate": gate, "r": r, "x": x}
    return c if name is None else {"name": name, **c}


def _before(M, H, r, x, name=None):
    c = {"op": "before", "M": M, "H": H, "r": r, "x": x}
    return c if name is None else {"name": name, **c}


def _lora(M, K, N, R, L, order, types, name=None):
    # order: "mixed" (each token its own request's adapter, any order) or
    # "runs" (prompts: consecutive tokens share an adapter)
    c = {"op": "lora", "M": M, "K": K, "N": N, "R": R, "L": L, "order": order, "types": types}
    return c if name is None else {"name": name, **c}


def _verify(B, T, V, q, ragged, greedy, name=None):
    # T: drafts per sequence (at most, if ragged); q: the drafter's
    # probabilities are given; greedy: every third sequence has temperature 0
    c = {"op": "verify", "B": B, "T": T, "V": V, "q": q, "ragged": ragged, "greedy": greedy}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one token of one request between two blocks
        _norm(1, 5120, True, True, "none", "bf16", "f16", "norm_token"),
        # a decode batch whose block output has a per-token gate, residual in fp32
        _norm(64, 5120, True, True, "sigmoid", "f32", "f16", "norm_batch_gated"),
        # a prompt chunk, a learned gate per channel
        _norm(4096, 5120, True, True, "layer", "bf16", "f16", "norm_prompt"),
        # the norm before a block on a ragged batch with an odd width
        _before(1021, 1001, "f16", "bf16", "norm_before_odd"),
        # one token with an adapter on the gate projection
        _lora(1, 5120, 17408, 16, 8, "mixed", "f16", "lora_token"),
        # a decode batch of 48 requests with adapters of their own
        _lora(48, 6144, 5120, 32, 32, "mixed", "bf16", "lora_batch"),
        # a few short prompts and their decode neighbours on the down projection
        _lora(333, 17408, 5120, 64, 8, "runs", "f16", "lora_chunk"),
        # a prompt chunk of several requests on the gate projection
        _lora(4096, 5120, 17408, 64, 6, "runs", "f16", "lora_prompt"),
        # one request with three drafted tokens
        _verify(1, 3, 248320, True, False, False, "verify_one"),
        # a batch of requests with seven drafts each
        _verify(16, 7, 248320, True, False, True, "verify_batch"),
        # deterministic drafts of ragged lengths, a smaller odd vocabulary
        _verify(32, 4, 32003, False, True, True, "verify_ragged"),
        # a full serving batch
        _verify(64, 3, 248320, True, False, False, "verify_full"),
    ]


def _log(rng, lo, hi):
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_KN = [(5120, 17408), (17408, 5120), (6144, 5120), (5120, 6144), (5120, 10240), (1024, 256),
       (640, 1001), (1664, 6083)]


def draw(rng):
    op = rng.choice(["norm", "before", "lora", "lora", "verify"])
    if op in ("norm", "before"):
        M = _log(rng, 1, 4096)
        H = rng.choice([5120, 6144, 1024, 2560, _log(rng, 64, 6144), 2 * _log(rng, 32, 2560) + 1])
        r = rng.choice(["f32", "bf16", "f16"])
        x = rng.choice(["f16", "bf16"])
        if op == "before":
            return _before(M, min(H, 5120) if M > 2048 else H, r, x)
        gate = rng.choice(["none", "layer", "sigmoid", "silu"])
        if M > 1500:  # no more bytes than the largest listed case
            H = min(H, 2560)
        return _norm(M, H, rng.random() < 0.7, rng.random() < 0.8, gate, r, x)
    if op == "lora":
        K, N = rng.choice(_KN)
        M = _log(rng, 1, 4096)
        R = rng.choice([8, 16, 24, 32, 64, 128])
        if M > 1024 and R > 64:
            R = 64
        L = _log(rng, 1, 64)
        if M > 256:  # the plain form's products are over all L * R columns
            L = min(L, max(1, 768 // R))
        return _lora(M, K, N, R, L, rng.choice(["mixed", "runs"]), rng.choice(["f16", "bf16"]))
    V = rng.choice([248320, _log(rng, 1000, 248320), 2 * _log(rng, 500, 100000) + 1])
    B, T = _log(rng, 1, 64), rng.randint(0, 7)
    while B * (T + 1) > 256:
        B //= 2
    return _verify(B, T, V, rng.random() < 0.7, T > 0 and rng.random() < 0.5, rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(c):
    """Drafts of each sequence (the ragged ones go 0, 1, ..., T, 0, ...)."""
    return [b % (c["T"] + 1) if c["ragged"] else c["T"] for b in range(c["B"])]


def _ranks(c):
    """Ranks in use: every other adapter is a smaller one."""
    return [c["R"] if l % 2 == 0 else max(1, c["R"] // 2) for l in range(c["L"])]


def _ids(c, gen):
    """Adapter of each token, on the host: all adapters in turn, with every
    tenth request without one (-1)."""
    M, L = c["M"], c["L"]
    if c["order"] == "runs":  # about 2 L + 1 requests, the prompts of different lengths
        cuts = torch.sort(torch.randint(0, M, (2 * L,), generator=gen)).values
        req = torch.searchsorted(cuts, torch.arange(M), right=True)
    else:
        req = torch.randperm(M, generator=gen)
    ids = req % L
    ids[(req % 10 == 9)] = -1
    return ids.to(torch.int32)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "before"):
        M, H = c["M"], c["H"]
        # the residual stream grows over the blocks and has a few large channels
        big = 1.0 + 20.0 * (torch.rand(H, generator=gen, device=DEV) < 0.01)
        s["r"] = (_randn(gen, M, H) * 2.0 * big).to(F[c["r"]])
        s["w_next"] = 1.0 + 0.1 * _randn(gen, H)
        if c["op"] == "before" or c["next"]:
            s["x"] = torch.empty((M, H), dtype=F[c["x"]], device=DEV)
        if c["op"] == "norm":
            s["y"] = _randn(gen, M, H) * 3.0
            s["w_post"] = 1.0 + 0.1 * _randn(gen, H)
            s["r_out"] = torch.empty_like(s["r"])
            if c["gate"] == "layer":
                s["gate"] = 0.5 + 0.1 * _randn(gen, H)
            elif c["gate"] != "none":
                # the second half of a projection's output, in place
                s["gate"] = _randn(gen, M, 2 * H).to(torch.bfloat16)[:, H:]
        return s
    if c["op"] == "lora":
        M, K, N, R, L = c["M"], c["K"], c["N"], c["R"], c["L"]
        t = F[c["types"]]
        x = _randn(gen, M, K)
        x = torch.where(torch.rand((M, K), generator=gen, device=DEV) < 0.01, x * 20.0, x)
        s["x"] = x.to(t)
        s["A"] = (_randn(gen, L, R, K) * K ** -0.5).to(t)
        s["B"] = (_randn(gen, L, N, R) * 0.1).to(t)
        s["ids"] = _ids(c, host).to(DEV)
        s["ranks"] = torch.tensor(_ranks(c), dtype=torch.int32, device=DEV)
        s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=gen, device=DEV)
        s["y"] = _randn(gen, M, N) * 2.0
        s["out"] = torch.empty_like(s["y"])
        s["workspace"] = None  # made by the first pass, kept by the program
        return s
    B, V = c["B"], c["V"]
    lens = torch.tensor(_lens(c))
    s["row_start"] = torch.cat([torch.zeros(1, dtype=torch.int64), (lens + 1).cumsum(0)])
    rows = int(s["row_start"][-1])
    s["row_start"] = s["row_start"].to(torch.int32).to(DEV)
    seq = torch.repeat_interleave(torch.arange(B), lens + 1).to(DEV)
    logits = _randn(gen, rows, V) * 2.5
    # a constrained sequence: part of the vocabulary is masked out
    masked = (torch.rand(V, generator=gen, device=DEV) < 0.3)
    logits.masked_fill_(masked[None, :] & (seq % 4 == 3)[:, None], float("-inf"))
    temp = 0.6 + 0.4 * torch.rand(B, generator=gen, device=DEV)
    if c["greedy"]:
        temp[::3] = 0.0
    # the drafter: the target's logits with an error of its own
    d = logits + 0.7 * _randn(gen, rows, V)
    tt = torch.where(temp > 0, temp, torch.ones_like(temp))[seq][:, None]
    q = torch.softmax(d / tt, -1)
    if c["q"]:
        noise = torch.empty_like(q).exponential_(generator=gen)
        s["q"] = q
        drafts = torch.where((temp > 0)[seq], (q / noise).argmax(-1), q.argmax(-1))
    else:
        s["q"] = None
        drafts = q.argmax(-1)
    s["logits"], s["drafts"], s["temperature"] = logits, drafts.to(torch.int32), temp
    s["u"] = torch.rand(rows, generator=gen, device=DEV)
    s["e"] = torch.empty((B, V), device=DEV).exponential_(generator=gen).clamp_(min=1e-12)
    s["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["tokens"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    s["workspace"] = None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
ALPHA = 0.7  # residual scale of the norm cases


def _run_own(s):
    pq2, c = _lib(), s["case"]
    if c["op"] == "before":
        pq2.pq2_rmsnorm(s["r"], s["w_next"], s["x"], EPS)
        return {"x": s["x"]}
    if c["op"] == "norm":
        flags = 0 if c["post"] else pq2.PQ2_NORM_NO_POST
        flags |= {"sigmoid": pq2.PQ2_GATE_SIGMOID, "silu": pq2.PQ2_GATE_SILU}.get(c["gate"], 0)
        pq2.pq2_norm_residual(s["y"], s["r"], s["r_out"], w_post=s["w_post"] if c["post"] else None,
                              gate=s.get("gate"), w_next=s["w_next"] if c["next"] else None,
                              x=s.get("x"), eps=EPS, alpha=ALPHA, flags=flags)
        return {"r": s["r_out"], "x": s["x"]} if c["next"] else {"r": s["r_out"]}
    if c["op"] == "lora":
        if s["workspace"] is None:
            s["workspace"] = pq2.alloc_lora_workspace(c["M"], c["N"], c["K"], c["L"], c["R"])
        pq2.pq2_lora_add(s["x"], s["A"], s["B"], s["ids"], s["y"], s["out"], s["workspace"],
                         ranks=s["ranks"], scales=s["scales"])
        return {"y": s["out"]}
    if s["workspace"] is None:
        s["workspace"] = pq2.alloc_verify_workspace(c["B"], s["logits"].shape[0], c["V"])
    pq2.pq2_verify_drafts(s["logits"], s["row_start"], s["drafts"], s["q"], s["u"], s["e"],
                          s["temperature"], s["accepted"], s["tokens"], s["workspace"])
    return {"accepted": s["accepted"], "tokens": s["tokens"]}


def _rms(v, w):
    n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return n if w is None else n * w


def _run_norm(s):
    c = s["case"]
    r = s["r"].float()
    if c["op"] == "before":
        return {"x": _rms(r, s["w_next"]).to(F[c["x"]])}
    n = _rms(s["y"], s["w_post"]) if c["post"] else s["y"]
    if c["gate"] != "none":
        g = s["gate"].float()
        if c["gate"] == "sigmoid":
            g = 1.0 / (1.0 + torch.exp(-g))
        elif c["gate"] == "silu":
            g = g / (1.0 + torch.exp(-g))
        n = n * g
    r = r + ALPHA * n
    out = {"r": r.to(F[c["r"]])}
    if c["next"]:
        out["x"] = _rms(r, s["w_next"]).to(F[c["x"]])
    return out


def _run_lora(s):
    # both products over all adapters' columns at once, each token keeping
    # those of its own adapter
    c = s["case"]
    M, N, R, L = c["M"], c["N"], c["R"], c["L"]
    used = torch.arange(R, device=DEV)[None, :] < s["ranks"][:, None]                      # [L, R]
    keep = (torch.arange(L, device=DEV)[None, :] == s["ids"][:, None])[:, :, None] & used   # [M, L, R]
    v = (s["x"].float() @ s["A"].float().reshape(L * R, -1).T).reshape(M, L, R)
    v = torch.where(keep, v * s["scales"][:, None], torch.zeros_like(v))
    b = torch.where(used[:, None, :], s["B"].float(), torch.zeros((), device=DEV))          # [L, N, R]
    return {"y": s["y"] + v.reshape(M, L * R) @ b.permute(0, 2, 1).reshape(L * R, N)}


def _first(score):
    """Lowest index of each row's maximum."""
    at = torch.arange(score.shape[-1], device=DEV)
    top = score.amax(-1, keepdim=True)
    return torch.where(score == top, at, score.shape[-1]).amin(-1)


def _run_verify(s):
    l, start = s["logits"], s["row_start"].long()
    rows, V = l.shape
    at = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(start, at, right=True) - 1
    temp = s["temperature"][seq]
    greedy = temp == 0
    top = l.amax(-1, keepdim=True)
    p = torch.exp((l - top) / torch.where(greedy, torch.ones_like(temp), temp)[:, None])
    p = p / p.sum(-1, keepdim=True)
    best = _first(l)
    d = s["drafts"].long()
    pd = p.gather(1, d[:, None])[:, 0]
    qd = torch.ones_like(pd) if s["q"] is None else s["q"].gather(1, d[:, None])[:, 0]
    last = at == start[seq + 1] - 1
    taken = ~last & torch.where(greedy, d == best, s["u"] * qd < pd)
    stop = torch.full((start.numel() - 1,), rows, device=DEV).scatter_reduce(
        0, seq, torch.where(taken, rows, at), "amin")
    p, d, refused = p[stop], d[stop], ~last[stop]
    if s["q"] is None:
        q = (torch.arange(V, device=DEV) == d[:, None]).float()
    else:
        q = s["q"][stop]
    rest = torch.where(refused[:, None], torch.clamp(p - q, min=0), p)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    token = torch.where(greedy[stop], best[stop], _first(rest / s["e"]))
    tokens = torch.where(at < stop[seq], s["drafts"].long(),
                         torch.where(at == stop[seq], token[seq], -torch.ones_like(at)))
    return {"accepted": (stop - start[:-1]).to(torch.int32), "tokens": tokens.to(torch.int32)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _run_lora(state) if op == "lora" else _run_verify(state) if op == "verify" else _run_norm(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("norm", "before"):
        n, r, x = c["M"] * c["H"], SIZE[c["r"]], SIZE[c["x"]]
        if c["op"] == "before":
            return {"bytes": n * (r + x) + 4 * c["H"], "flops": 4 * n}
        b = n * (4 + 2 * r + (x if c["next"] else 0) + (2 if c["gate"] in ("sigmoid", "silu") else 0))
        b += 4 * c["H"] * (c["post"] + c["next"] + (c["gate"] == "layer"))
        return {"bytes": b, "flops": n * (3 + 4 * c["post"] + 4 * c["next"])}
    if c["op"] == "lora":
        M, K, N, L = c["M"], c["K"], c["N"], c["L"]
        ranks = sum(_ranks(c)[:min(L, M)])  # adapters in use
        mean = sum(_ranks(c)) / L
        return {"bytes": 2 * M * K + 8 * M * N + 2 * ranks * (K + N), "flops": 2 * 0.9 * M * mean * (K + N)}
    V, B = c["V"], c["B"]
    rows = sum(n + 1 for n in _lens(c))
    drawn = B - len(range(0, B, 3)) if c["greedy"] else B  # sequences that draw from a row
    return {"bytes": 4 * V * (rows + drawn * (2 if c["q"] else 1)), "flops": 4 * rows * V}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "lora":
        y = s["y"].double()
        ids = s["ids"].cpu()
        for l, rank in enumerate(_ranks(c)):
            m = torch.nonzero(ids == l)[:, 0].to(DEV)
            if m.numel() == 0:
                continue
            v = torch.einsum("mk,rk->mr", s["x"][m].double(), s["A"][l, :rank].double())
            y[m] += float(s["scales"][l]) * torch.einsum("mr,nr->mn", v, s["B"][l, :, :rank].double())
        return {"y": y}

    def normed(v, w):
        return v / torch.sqrt(torch.sum(v ** 2, dim=1, keepdim=True) / v.shape[1] + EPS) * w.double()

    r = s["r"].double()
    if c["op"] == "before":
        return {"x": normed(r, s["w_next"])}
    add = s["y"].double()
    if c["post"]:
        add = normed(add, s["w_post"])
    if c["gate"] == "layer":
        add = add * s["gate"].double()
    elif c["gate"] in ("sigmoid", "silu"):
        g = s["gate"].double()
        add = add * torch.sigmoid(g) * (g if c["gate"] == "silu" else 1.0)
    r = r + ALPHA * add
    return {"r": r, "x": normed(r, s["w_next"])} if c["next"] else {"r": r}
