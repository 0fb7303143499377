"""The attention side of a serving step, as cases to measure.

Three sets of operators:
  rope    rotary positions of queries and keys (pq2_rope)
  cache   keys and values held in 4 bits in pages: rotated, quantised and
          appended (pq2_cache4_append, read back with pq2_cache4_read), and
          attended to (pq2_cache4_attend)
  pages   the pages of such a cache: continued, forked, cut back, freed and
          allotted for a step (pq2_pages_update), moved to the front
          (pq2_pages_compact), and copied (pq2_pages_copy)

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the library's entry points.  Head layouts are those of the library's
projections (6144 = 24 x 256 = 48 x 128, 5120 = 40 x 128) and generic ones.

A page holds T tokens of every key/value head.  Its bytes, per head, are T/16
tiles of 16 tokens, each
  16 rows of D/2 bytes   key codes (value 2i in the low half of byte i)
  16 rows of D/2 bytes   value codes
  16 pairs of fp16       scale and offset of each key row
  16 pairs of fp16       scale and offset of each value row
and a code c stands for c * scale + offset.
"""
import torch

own = False

DEV = "cuda"
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
TILE = 16  # tokens of a tile
BASE = 1e6  # of the rotary frequencies

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
def _rope(M, Hq, Hkv, D, rot, far, pairs, x, y, name=None):
    # rot: rotated part of a head; far: positions below this; pairs: "halves"
    # or "neighbours"; x: type of the projection's output, y: of the rotated
    c = {"op": "rope", "M": M, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "far": far, "pairs": pairs,
         "x": x, "y": y}
    return c if name is None else {"name": name, **c}


def _append(B, n, len_, Hq, Hkv, D, rot, T, pairs, x, y, name=None):
    # n new tokens (at most: ragged) of each of B sequences that then have at
    # most len_
    c = {"op": "append", "B": B, "n": n, "len": len_, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "T": T,
         "pairs": pairs, "x": x, "y": y}
    return c if name is None else {"name": name, **c}


def _attend(B, n, len_, ragged, Hq, Hkv, D, T, window, types, name=None):
    # n new tokens of each of B sequences, the last of len_; ragged: both up to
    # that; window: tokens that a token sees (0: all before it)
    c = {"op": "attend", "B": B, "n": n, "len": len_, "ragged": ragged, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T,
         "window": window, "types": types}
    return c if name is None else {"name": name, **c}


def _pages(B, W, T, P, Hkv, D, forks, name=None):
    # a step of B sequences of up to W pages: cut back to the kept drafts,
    # forked, ended, and given pages for the next tokens
    c = {"op": "pages", "B": B, "W": W, "T": T, "P": P, "Hkv": Hkv, "D": D, "forks": forks}
    return c if name is None else {"name": name, **c}


def _compact(B, W, T, P, Hkv, D, name=None):
    c = {"op": "compact", "B": B, "W": W, "T": T, "P": P, "Hkv": Hkv, "D": D}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # queries and keys of a decode batch
        _rope(64, 48, 8, 128, 128, 32768, "halves", "f32", "f16", "rope_batch"),
        # of a prompt chunk far into a long context, a quarter of each head rotated
        _rope(4096, 24, 4, 256, 64, 262144, "neighbours", "f32", "bf16", "rope_prompt"),
        # a decode batch's keys and values into the cache
        _append(64, 1, 8192, 24, 4, 256, 64, 64, "halves", "f32", "bf16", "append_batch"),
        # ragged prompt chunks
        _append(5, 1021, 3000, 48, 8, 128, 128, 16, "halves", "f32", "f16", "append_prompt"),
        # one token of one request
        _attend(1, 1, 1027, False, 24, 4, 256, 16, 0, "bf16", "attend_token"),
        # one token of a request with a very long context
        _attend(1, 1, 131071, False, 24, 4, 256, 64, 0, "f16", "attend_long"),
        # a decode batch of requests of all lengths
        _attend(64, 1, 8192, True, 48, 8, 128, 64, 0, "bf16", "attend_batch"),
        # drafts to verify, with a window
        _attend(24, 5, 5003, True, 40, 8, 128, 32, 4096, "f16", "attend_drafts"),
        # ragged prompt chunks behind a longer context
        _attend(3, 1000, 6000, True, 40, 8, 128, 32, 0, "bf16", "attend_chunks"),
        # a long prompt's last chunk
        _attend(1, 4096, 8192, False, 24, 4, 256, 64, 0, "f16", "attend_prompt"),
        # the pages of a batch between two steps
        _pages(64, 48, 32, 3400, 8, 128, True, "pages_step"),
        # a pool that has come to be full of holes
        _compact(96, 40, 64, 3900, 4, 256, "pages_compact"),
    ]


def _log(rng, lo, hi):
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(24, 4, 256), (48, 8, 128), (40, 8, 128), (16, 2, 64), (8, 8, 64), (12, 4, 128), (7, 1, 128),
          (20, 4, 256), (6, 2, 256), (64, 4, 64)]


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "pages", "compact"])
    Hq, Hkv, D = rng.choice(_HEADS)
    T = rng.choice([16, 32, 64, 128])
    pairs = rng.choice(["halves", "neighbours"])
    x, y = rng.choice(["f32", "f32", "bf16", "f16"]), rng.choice(["f16", "bf16"])
    rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
    if op == "rope":
        M = _log(rng, 1, max(1, min(4096, (4096 * 28 * 256) // ((Hq + Hkv) * D))))
        return _rope(M, Hq, Hkv, D, rot, _log(rng, 2000, 262144), pairs, x, y)
    if op == "append":
        B, n = _log(rng, 1, 64), _log(rng, 1, 1021)
        while B * n * (Hq + 2 * Hkv) * D > 5105 * 64 * 128:
            B, n = (B + 1) // 2, (n + 1) // 2
        return _append(B, n, n + _log(rng, 1, 4000), Hq, Hkv, D, rot, T, pairs, x, y)
    if op == "attend":
        kind = rng.choice(["token", "batch", "drafts", "chunks"])
        B = 1 if kind == "token" else _log(rng, 1, 64) if kind != "chunks" else rng.randint(1, 4)
        n = 1 if kind in ("token", "batch") else rng.randint(2, 8) if kind == "drafts" else _log(rng, 17, 3000)
        ln = n + _log(rng, 1, 100000 if kind == "token" else 8192)
        while B * ln * Hkv * D > 64 * 8192 * 4 * 128 or B * n * ln * Hq * D > 4096 * 6144 * 6144:
            B, n, ln = (B + 1) // 2, (n + 1) // 2 if kind == "chunks" else n, max(n, (ln * 3) // 4)
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return _attend(B, n, ln, rng.random() < 0.7, Hq, Hkv, D, T, window, y)
    B, W = _log(rng, 1, 96), _log(rng, 2, 128)
    Hkv, D = rng.choice([(4, 256), (8, 128), (2, 64)])
    while B * W * T * Hkv * D > 64 * 64 * 32 * 1024:
        B, W = (B + 1) // 2, max(2, W // 2)
    if op == "pages":
        return _pages(B, W, T, B * W + B + rng.randint(8, 500), Hkv, D, rng.random() < 0.6)
    return _compact(B, W, T, B * W + rng.randint(8, 400), Hkv, D)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _spread(count, most, ragged):
    """Lengths of `count` sequences: all `most`, or spread over 1 .. most, the
    first one the longest."""
    return [most if not ragged or b == 0 else 1 + (b * 7919 * 13) % most for b in range(count)]


def _lens(c):
    """(new tokens, length) of each sequence."""
    ragged = c.get("ragged", True)
    n = _spread(c["B"], c["n"], ragged)
    return n, [max(k, m) for k, m in zip(n, _spread(c["B"], c["len"], ragged))]


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _table(positions, rot):
    """cos and sin of each position's angles, computed in 64 bits."""
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float().contiguous()


def _quantised(x):
    """Codes, scale and offset of rows of 32-bit values."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = torch.clamp((hi - lo) * (1.0 / 15.0), max=65504.0).half().float()
    offset = torch.clamp(lo, -65504.0, 65504.0).half().float()
    inverse = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    return torch.clamp(torch.round((x - offset) * inverse), 0.0, 15.0), scale, offset


def _packed(k, v):
    """Pages [P, H, bytes] of key and value rows [P, H, T, D]."""
    P, H, T, D = k.shape
    parts, pairs = [], []
    for x in (k, v):
        code, scale, offset = _quantised(x)
        code = code.to(torch.uint8)
        code = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(P, H, T // TILE, TILE * D // 2)
        pair = torch.cat([scale, offset], -1).half().view(torch.uint8)
        parts.append(code)
        pairs.append(pair.reshape(P, H, T // TILE, TILE * 4))
    return torch.cat(parts + pairs, -1).reshape(P, H, T * (D + 8)).contiguous()


def _held(gen, pages, H, T, D):
    """A pool of that many pages of keys and values as a model makes them: a
    few large key channels, channels with an offset, tokens of unlike size."""
    channel = 1.0 + 3.0 * (torch.rand(D, generator=gen, device=DEV) < 0.03)
    k = _randn(gen, pages, H, T, D) * channel + 0.5 * _randn(gen, D)
    v = _randn(gen, pages, H, T, D) * (0.5 + torch.rand((pages, H, T, 1), generator=gen, device=DEV))
    return _packed(k, v)


def _allotted(host, lens, T, W, spare):
    """Pages in any order: [B, W] on the host, with -1 behind the last."""
    counts = [-(-n // T) for n in lens]
    order = torch.randperm(sum(counts) + spare, generator=host).to(torch.int32)
    table, at = torch.full((len(lens), W), -1, dtype=torch.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(counts) + spare


def _starts(n):
    return torch.tensor([0] + n).cumsum(0).to(torch.int32)


def _prepare_pages(c, s, gen, host):
    B, W, T, P = c["B"], c["W"], c["T"], c["P"]
    most = W * T - 8
    lens = [most] + torch.randint(1, most + 1, (B - 1,), generator=host).tolist() if B > 1 else [most]
    table, used = _allotted(host, lens, T, W, 0)
    order = torch.randperm(P - 1, generator=host).to(torch.int32) + 1  # page 0 is the program's own
    table = torch.where(table >= 0, order[table.clamp(min=0)], table)
    refs = torch.zeros(P, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    refs[0] = 1
    if c["op"] == "pages":
        # every fourth sequence began with another's first pages
        for b in range(3, B, 4):
            share = min(lens[b], lens[b - 1]) // T // 2
            refs[table[b, :share].long()] -= 1
            table[b, :share] = table[b - 1, :share]
            refs[table[b, :share].long()] += 1
        ln = torch.tensor(lens)
        source = torch.arange(B)
        keep = torch.clamp(ln - torch.randint(0, 4, (B,), generator=host), min=1)  # refused drafts
        new = keep + 4
        ended = torch.rand(B, generator=host) < 0.1
        if c["forks"]:  # those continue as further samples of a neighbour
            other = (torch.arange(B) + 1) % B
            source = torch.where(ended, other, source)
            keep = torch.where(ended, ln[other], keep)
            new = torch.where(ended, keep + 4, new)
        else:
            source = torch.where(ended, -torch.ones_like(source), source)
            new = torch.where(ended, torch.zeros_like(new), new)
        s |= {"source": source, "keep": keep, "new": new, "copies": torch.zeros((B, 2))}
    else:
        gone = torch.rand(B, generator=host) < 0.3  # sequences that have ended
        for b in torch.nonzero(gone)[:, 0].tolist():
            refs[table[b, :-(-lens[b] // T)].long()] = 0
            table[b], lens[b] = -1, 0
        s |= {"copies": torch.zeros((P // 2, 2))}
    s |= {"table": table, "refs": refs, "lens": torch.tensor(lens), "table_out": torch.zeros_like(table),
          "refs_out": torch.zeros_like(refs), "info": torch.zeros(2)}
    for k, v in s.items():
        if torch.is_tensor(v):
            s[k] = v.to(torch.int32).to(DEV)
    s["pool"] = torch.randint(0, 256, (P, c["Hkv"], T * (c["D"] + 8)), dtype=torch.uint8, generator=gen, device=DEV)
    s["workspace"] = None
    return s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("pages", "compact"):
        return _prepare_pages(c, s, gen, host)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        M = c["M"]
        s["qkv"] = _randn(gen, M, (Hq + 2 * Hkv) * D).to(F[c["x"]])  # the fused projection's output
        s["positions"] = torch.randint(0, c["far"], (M,), generator=host).to(torch.int32).to(DEV)
        s["table"] = _table(c["far"], c["rot"])
        s["q"] = torch.empty((M, Hq, D), dtype=F[c["y"]], device=DEV)
        s["k"] = torch.empty((M, Hkv, D), dtype=F[c["y"]], device=DEV)
        return s
    n, lens = _lens(c)
    M, T = sum(n), c["T"]
    W = -(-max(lens) // T)
    table, P = _allotted(host, lens, T, W, 3)
    s["pages"], s["row_start"] = table.to(DEV), _starts(n).to(DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["op"] == "append":
        s["pool"] = torch.zeros((P, Hkv, T * (D + 8)), dtype=torch.uint8, device=DEV)
        s["qkv"] = _randn(gen, M, (Hq + 2 * Hkv) * D).to(F[c["x"]])
        s["table"] = _table(max(lens), c["rot"])
        s["q"] = torch.empty((M, Hq, D), dtype=F[c["y"]], device=DEV)
        s["k"] = torch.empty((M, Hkv, D), dtype=F[c["y"]], device=DEV)
        s["v"] = torch.empty((M, Hkv, D), dtype=F[c["y"]], device=DEV)
        return s
    s["pool"] = _held(gen, P, Hkv, T, D)
    s["q"] = (_randn(gen, M, Hq, D) * 1.5).to(F[c["types"]])
    s["out"] = torch.empty((M, Hq, D), dtype=F[c["types"]], device=DEV)
    s["workspace"] = None
    return s


# ---------------------------------------------------------------------------
# One pass: the library
# ---------------------------------------------------------------------------
def _split(s):
    """q, k and v in the fused projection's output."""
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, D)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _run_own(s):
    pq2, c = _lib(), s["case"]
    if c["op"] in ("rope", "append"):
        flags = pq2.PQ2_ROPE_NEIGHBOURS if c["pairs"] == "neighbours" else 0
        q, k, v = _split(s)
    if c["op"] == "rope":
        pq2.pq2_rope(q, s["table"], s["positions"], s["q"], k, s["k"], flags=flags)
        return {"q": s["q"], "k": s["k"]}
    if c["op"] == "append":
        pq2.pq2_cache4_append(k, v, s["pool"], s["pages"], s["row_start"], s["lens"], q=q, q_out=s["q"],
                              table=s["table"], flags=flags)
        pq2.pq2_cache4_read(s["pool"], s["pages"], s["row_start"], s["lens"], s["k"], s["v"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if c["op"] == "attend":
        if s["workspace"] is None:
            s["workspace"] = pq2.alloc_attend_workspace(s["q"].shape[0], c["Hq"], c["Hkv"], c["D"])
        pq2.pq2_cache4_attend(s["q"], s["pool"], s["pages"], s["row_start"], s["lens"], s["out"],
                              s["workspace"], window=c["window"], max_rows=c["n"])
        return {"out": s["out"]}
    if s["workspace"] is None:
        s["workspace"] = pq2.alloc_pages_workspace(c["B"], c["P"])
    if c["op"] == "pages":
        pq2.pq2_pages_update(s["table"], s["refs"], s["lens"], s["source"], s["keep"], s["new"], c["T"],
                             s["table_out"], s["refs_out"], s["copies"], s["info"], s["workspace"])
    else:
        pq2.pq2_pages_compact(s["table"], s["refs"], s["lens"], c["T"], s["table_out"], s["refs_out"],
                              s["copies"], s["info"], s["workspace"])
    pq2.pq2_pages_copy(s["pool"], s["copies"])
    return {"table": s["table_out"], "refs": s["refs_out"], "copies": s["copies"], "info": s["info"],
            "pool": s["pool"].view(torch.int32)}


# ---------------------------------------------------------------------------
# One pass: the plain form
# ---------------------------------------------------------------------------
def _rotated(x, cs, rot, pairs):
    """x [M, H, D] in 32 bits with its first `rot` values turned; cs [M, rot / 2, 2]."""
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    c = s["case"]
    q, k, _ = _split(s)
    cs = s["table"][s["positions"].long()]
    return {"q": _rotated(q.float(), cs, c["rot"], c["pairs"]).to(F[c["y"]]),
            "k": _rotated(k.float(), cs, c["rot"], c["pairs"]).to(F[c["y"]])}


def _at(s):
    """Sequence and position of each row."""
    start, row = s["row_start"].long(), torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(start, row, right=True) - 1
    return seq, s["lens"].long()[seq] - start[seq + 1] + row


def _run_append(s):
    # the rows as the cache holds them, written to their places and read back
    c = s["case"]
    T, D, Hkv = c["T"], c["D"], c["Hkv"]
    q, k, v = _split(s)
    seq, pos = _at(s)
    cs = s["table"][pos]
    page = s["pages"].long()[seq, pos // T]
    out = {"q": _rotated(q.float(), cs, c["rot"], c["pairs"]).to(F[c["y"]])}
    tiles = s["pool"].view(-1, Hkv, T // TILE, TILE * (D + 8))
    tile, row = (pos % T) // TILE, pos % TILE
    at = torch.arange(D // 2, device=DEV)
    quad = torch.arange(4, device=DEV)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    for name, x, first in (("k", _rotated(k.float(), cs, c["rot"], c["pairs"]), 0), ("v", v.float(), 1)):
        code, scale, offset = _quantised(x)
        byte = code.to(torch.uint8)
        byte = byte[..., 0::2] | (byte[..., 1::2] << 4)
        pair = torch.cat([scale, offset], -1).half().view(torch.uint8)
        place = (page[:, None, None], head, tile[:, None, None])
        tiles[(*place, (first * TILE + row)[:, None, None] * (D // 2) + at)] = byte
        tiles[(*place, TILE * D + (first * TILE + row)[:, None, None] * 4 + quad)] = pair
        out[name] = (code * scale + offset).to(F[c["y"]])
    return out


def _values(s):
    """Keys and values [B, H, W * T, D] in 32 bits."""
    c = s["case"]
    T, D, Hkv = c["T"], c["D"], c["Hkv"]
    held = s["pool"][s["pages"].long().clamp(min=0)].view(c["B"], -1, Hkv, T // TILE, TILE * (D + 8))
    out = []
    for first in (0, 1):
        code = held[..., first * TILE * D // 2:(first + 1) * TILE * D // 2]
        pair = held[..., TILE * (D + 4 * first):TILE * (D + 4 * first + 4)].contiguous().view(torch.float16)
        pair = pair.float().unflatten(-1, (TILE, 2))
        code = torch.stack([code & 15, code >> 4], -1).float().unflatten(-2, (TILE, D // 2)).flatten(-2)
        x = code * pair[..., :1] + pair[..., 1:]
        out.append(x.permute(0, 2, 1, 3, 4, 5).reshape(c["B"], Hkv, -1, D))
    return out


def _run_attend(s):
    c = s["case"]
    B, n, Hq, Hkv, D = c["B"], c["n"], c["Hq"], c["Hkv"], c["D"]
    k, v = _values(s)
    start, lens = s["row_start"].long(), s["lens"].long()
    i = torch.arange(n, device=DEV)
    rows = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                     # [B, n]
    q = s["q"].float()[rows].view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    pos = lens[:, None] - (start[1:] - start[:-1])[:, None] + i                      # [B, n]
    at = torch.arange(k.shape[2], device=DEV)
    sees = at <= pos[..., None]
    if c["window"]:
        sees &= at > pos[..., None] - c["window"]
    sees = sees[:, None, None].expand(B, Hkv, Hq // Hkv, n, -1).reshape(B, Hkv, -1, k.shape[2])
    w = torch.where(sees, q @ k.transpose(-1, -2) * D ** -0.5, float("-inf"))
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    out = (w @ v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    row = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(start, row, right=True) - 1
    return {"out": out[seq, row - start[seq]].to(F[c["types"]])}


def _count(at, mask, P):
    """How often each page stands in `at` where `mask` is true."""
    return torch.zeros(P + 1, dtype=torch.int64, device=DEV).scatter_add(
        0, torch.where(mask, at, P).flatten(), torch.ones_like(at).flatten())[:P]


def _copied(s, pairs):
    # a pair that says nothing copies the program's own page to itself
    pool, pairs = s["pool"].view(torch.int32), pairs.long().clamp(min=0)
    pool[pairs[:, 1]] = pool[pairs[:, 0]]
    return pool


def _run_pages(s):
    c = s["case"]
    B, W, T, P = c["B"], c["W"], c["T"], c["P"]
    table, lens, source = s["table"].long(), s["lens"].long(), s["source"].long()
    new = s["new"].long()
    j, b = torch.arange(W, device=DEV), torch.arange(B, device=DEV)
    outside = s["refs"].long() - _count(table, j < (-(-lens // T))[:, None], P)
    from_ = source.clamp(min=0)
    keep = torch.minimum(torch.where(source >= 0, torch.minimum(s["keep"].long(), lens[from_]), 0), new)
    full, part, want = keep // T, keep % T > 0, -(-new // T)
    taken = table[from_]
    whole = _count(taken, j < full[:, None], P)
    last = taken.gather(1, full.clamp(max=W - 1)[:, None])[:, 0]
    first = torch.full((P + 1,), B, device=DEV).scatter_reduce(0, torch.where(part, last, P), b, "amin")[:P]
    at = last.clamp(min=0)
    stays = part & (outside[at] <= 0) & (whole[at] == 0) & (first[at] == b)
    copy = part & ~stays
    free = (outside <= 0) & (whole == 0) & (first == B)
    have = full + stays.long()
    needs = want - have
    rank = (needs.cumsum(0) - needs)[:, None] + j - have[:, None]
    up_to = free.long().cumsum(0)
    got = torch.searchsorted(up_to, (rank + 1).clamp(min=1))  # the rank's free page, lowest first
    got = torch.where(got < P, got, -1)
    out = torch.where(j < have[:, None], taken, torch.where(j < want[:, None], got, -1))
    refs = outside.clamp(min=0) + _count(out, (j < want[:, None]) & (out >= 0), P)
    dst = out.gather(1, full.clamp(max=W - 1)[:, None])[:, 0]
    does = copy & (dst >= 0)
    copies = torch.where(does[:, None], torch.stack([last, dst], -1), -1)
    left = free.sum() - needs.sum()
    info = torch.stack([left.clamp(min=0), (-left).clamp(min=0)])
    return {"table": out.to(torch.int32), "refs": refs.to(torch.int32), "copies": copies.to(torch.int32),
            "info": info.to(torch.int32), "pool": _copied(s, copies)}


def _run_compact(s):
    c = s["case"]
    W, T, P = c["W"], c["T"], c["P"]
    used, p = s["refs"] > 0, torch.arange(P, device=DEV)
    total = used.sum()
    mover, hole = used & (p >= total), ~used & (p < total)
    moves = mover.sum()
    i = torch.arange(P // 2, device=DEV)
    src = torch.searchsorted(mover.long().cumsum(0), i + 1)
    dst = torch.searchsorted(hole.long().cumsum(0), i + 1)
    copies = torch.where((i < moves)[:, None], torch.stack([src, dst], -1), -1)
    goes = torch.cat([p, p[:1]]).scatter(0, torch.where(i < moves, src, P), dst)[:P]
    table = s["table"].long()
    out = torch.where(torch.arange(W, device=DEV) < (-(-s["lens"].long() // T))[:, None],
                      goes[table.clamp(min=0)], -1)
    refs = torch.zeros(P, dtype=torch.int64, device=DEV).scatter_add(0, goes, s["refs"].long().clamp(min=0))
    return {"table": out.to(torch.int32), "refs": refs.to(torch.int32), "copies": copies.to(torch.int32),
            "info": torch.stack([total, moves]).to(torch.int32), "pool": _copied(s, copies)}


_PLAIN = {"rope": _run_rope, "append": _run_append, "attend": _run_attend, "pages": _run_pages,
          "compact": _run_compact}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("pages", "compact"):
        B, W, P = c["B"], c["W"], c["P"]
        page = c["Hkv"] * c["T"] * (c["D"] + 8)
        meta = 4 * (2 * B * W + 2 * P + 5 * B)
        # pages that move: a tenth of the sequences is forked; about a fifth of
        # the pages in use lies behind the last place in use
        moved = 0.1 * B * c["forks"] if c["op"] == "pages" else 0.12 * B * W
        return {"bytes": meta + 2 * page * moved, "flops": B * W + P}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        n = c["M"] * (Hq + Hkv)
        return {"bytes": n * D * (SIZE[c["x"]] + SIZE[c["y"]]) + 4 * c["M"] * (c["rot"] + 1),
                "flops": 3 * n * c["rot"]}
    n, lens = _lens(c)
    M = sum(n)
    if c["op"] == "append":
        # the cache's rows are written, and read back for the outputs
        rows = M * (Hq + 2 * Hkv) * D
        return {"bytes": rows * (SIZE[c["x"]] + SIZE[c["y"]]) + 4 * M * Hkv * (D + 8) + 4 * M * c["rot"],
                "flops": 3 * M * (Hq + Hkv) * c["rot"] + 8 * M * Hkv * D}
    w = c["window"] or max(lens)
    sees = sum(sum(min(w, m - k + i + 1) for i in range(k)) for k, m in zip(n, lens))
    held = sum(min(m, w + k - 1) for k, m in zip(n, lens))
    return {"bytes": held * Hkv * (D + 8) + 2 * M * Hq * D * SIZE[c["types"]], "flops": 4 * sees * Hq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _turned(x, pos, rot, pairs):
    # every pair as a complex number times exp(i * angle)
    f = torch.exp(torch.arange(rot // 2, dtype=torch.float64, device=DEV) * (-2.0 / rot) * torch.log(
        torch.tensor(BASE, dtype=torch.float64, device=DEV)))
    turn = torch.polar(torch.ones((pos.numel(), 1, rot // 2), dtype=torch.float64, device=DEV),
                       pos.double()[:, None, None] * f)
    part = x[..., :rot].double()
    z = part.unflatten(-1, (2, -1)).transpose(-1, -2) if pairs == "halves" else part.unflatten(-1, (-1, 2))
    z = torch.view_as_real(torch.complex(z[..., 0].contiguous(), z[..., 1].contiguous()) * turn)
    z = z.transpose(-1, -2).flatten(-2) if pairs == "halves" else z.flatten(-2)
    return torch.cat([z, x[..., rot:].double()], -1)


def _stands_for(x):
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale, offset = ((hi - lo) / 15).half().double(), lo.half().double()
    return torch.round((x - offset) / scale).clamp(0, 15) * scale + offset


def exact(case, seed):
    c = case
    if c["op"] in ("pages", "compact"):
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "rope":
        q, k, _ = _split(s)
        return {"q": _turned(q, s["positions"], c["rot"], c["pairs"]),
                "k": _turned(k, s["positions"], c["rot"], c["pairs"])}
    n, lens = _lens(c)
    if c["op"] == "append":
        q, k, v = _split(s)
        pos = torch.cat([torch.arange(m - i, m) for i, m in zip(n, lens)]).to(DEV)
        return {"q": _turned(q, pos, c["rot"], c["pairs"]),
                "k": _stands_for(_turned(k, pos, c["rot"], c["pairs"])), "v": _stands_for(v.double())}
    Hq, Hkv, D, T = c["Hq"], c["Hkv"], c["D"], c["T"]
    out, row = [], 0
    for b, (new, ln) in enumerate(zip(n, lens)):
        tiles = s["pool"][s["pages"][b, :-(-ln // T)].long()].reshape(-1, Hkv, T // TILE, TILE * (D + 8))
        tiles = tiles.transpose(1, 2).reshape(-1, Hkv, TILE * (D + 8))
        kv = []
        for first in (0, 1):
            code = tiles[..., first * TILE * D // 2:(first + 1) * TILE * D // 2].reshape(-1, Hkv, TILE, D // 2)
            pair = tiles[..., TILE * (D + 4 * first):TILE * (D + 4 * first + 4)].contiguous().view(torch.float16)
            pair = pair.reshape(-1, Hkv, TILE, 2).double()
            x = torch.stack([code % 16, code // 16], -1).reshape(-1, Hkv, TILE, D).double()
            x = x * pair[..., :1] + pair[..., 1:]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :ln])
        q = s["q"][row:row + new].double()
        gap = (torch.arange(new, device=DEV) + ln - new)[:, None] - torch.arange(ln, device=DEV)
        hidden = (gap < 0) | (gap >= (c["window"] or ln + 1))
        heads = []
        for h in range(Hq):
            k, v = kv[0][h // (Hq // Hkv)], kv[1][h // (Hq // Hkv)]
            a = torch.softmax((q[:, h] @ k.T / D ** 0.5).masked_fill(hidden, float("-inf")), -1)
            heads.append(a @ v)
        out.append(torch.stack(heads, 1))
        row += new
    return {"out": torch.cat(out)}
