"""Rotary positions, a cache held in 4 bits and attention over it, and the
bookkeeping of its pages, in numpy from their definitions.  Slow and plain;
shares no code with the CUDA library.

What a definition fixes to the bit (turned values, codes, page numbers) is
computed in the same 32-bit or whole-number steps; the rest in float64, with
the sums of magnitudes that an error bound needs."""
import numpy as np

F32 = np.float32
TILE = 16


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
def frequencies(rot, base, kind="plain", factor=1.0, old_len=0.0, low=0.0, high=0.0):
    f = []
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    if kind == "ramp":
        def index(turns):
            return rot / 2 * np.log(old_len / (2 * np.pi * turns)) / np.log(base)
        i0, i1 = max(np.floor(index(high)), 0.0), min(np.ceil(index(low)), rot - 1.0)
        i1 = max(i1, i0 + 0.001)
    for i in range(rot // 2):
        x = base ** (-2 * i / rot)
        if kind == "linear":
            x = x / factor
        elif kind == "ramp":
            t = min(max((i - i0) / (i1 - i0), 0.0), 1.0)
            x = x * (1 - t) + x / factor * t
        elif kind == "bands":
            wave = 2 * np.pi / x
            if wave > old_len / low:
                x = x / factor
            elif wave >= old_len / high:
                t = (old_len / wave - low) / (high - low)
                x = (1 - t) * x / factor + t * x
        f.append(x)
    return np.array(f)


def table(first, count, f, magnitude=1.0):
    a = np.arange(first, first + count, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1) * magnitude


def turn(x, cs, rot, near, inverse=False):
    """x fp32 [M, H, D], cs fp32 [M, rot / 2, 2]; every step one fp32 operation."""
    x = np.asarray(x, F32)
    y = x.copy()
    a = slice(0, rot, 2) if near else slice(0, rot // 2)
    b = slice(1, rot, 2) if near else slice(rot // 2, rot)
    c, s = cs[:, None, :, 0].astype(F32), cs[:, None, :, 1].astype(F32)
    if inverse:
        s = -s
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# ---------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------
def quantise(x):
    """Rows of fp32 values -> codes, scales, offsets (fp16 values as fp32)."""
    x = np.asarray(x, F32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        s = np.minimum((hi - lo) * F32(1 / 15), F32(65504)).astype(np.float16).astype(F32)
        z = np.clip(lo, F32(-65504), F32(65504)).astype(np.float16).astype(F32)
        inv = np.where(s > 0, F32(1) / s, F32(0)).astype(F32)
        c = np.clip(np.rint((x - z) * inv), 0, 15)
    return c.astype(np.uint8), s, z


def dequantise(c, s, z):
    return c.astype(F32) * s + z


def read_tile(tile, D):
    """One tile's bytes -> codes [2, 16, D] and (scale, offset) [2, 16, 2]."""
    codes = tile[:TILE * D].reshape(2, TILE, D // 2)
    codes = np.stack([codes & 15, codes >> 4], -1).reshape(2, TILE, D)
    pairs = tile[TILE * D:].copy().view(np.float16).reshape(2, TILE, 2).astype(F32)
    return codes, pairs


def write_row(pool, page, head, t, T, D, value, c, s, z):
    """Puts one row into a pool uint8 [P, H, T (D + 8)]."""
    tile = pool[page, head, (t // TILE) * TILE * (D + 8):(t // TILE + 1) * TILE * (D + 8)]
    at = (value * TILE + t % TILE) * (D // 2)
    tile[at:at + D // 2] = c[0::2] | (c[1::2] << 4)
    at = TILE * D + (value * TILE + t % TILE) * 4
    tile[at:at + 4] = np.array([s, z], np.float16).view(np.uint8)


def read_rows(pool, pages, length, head, T, D):
    """Keys and values [length, D] of a sequence as the cache holds them, with
    their codes, scales and offsets."""
    codes, pairs = [], []
    for j in range(-(-length // T)):
        block = pool[pages[j], head].reshape(T // TILE, TILE * (D + 8))
        for tile in block:
            c, p = read_tile(tile, D)
            codes.append(c)
            pairs.append(p)
    if not codes:
        return np.zeros((2, 0, D), np.uint8), np.zeros((2, 0, 2), F32)
    return np.concatenate(codes, 1)[:, :length], np.concatenate(pairs, 1)[:, :length]


def attend(q, pool, pages, row_start, lens, T, scale, window=0):
    """q [M, Hq, D] -> (out float64 [M, Hq, D], error bound before the last
    rounding).  The bound: weights rounded to 11 bits (2^-11 of their share),
    scores off by fp32 sums of D products, exponentials by 2^-21, sums of
    tiles cut off at 24 bits.  Below fp16's normal numbers a weight is off by up
    to half a step of 2^-24 instead: weights stand for w s / ref 64 there, where ref <= the
    largest scale s and the largest w >= 1/2, codes are at most 8 off the middle, so
    that each key adds up to 2^-25 / 64 s 8 / (1/2) = s 2^-27."""
    q = np.asarray(q, np.float64)
    M, Hq, D = q.shape
    H = pool.shape[1]
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b, ln in enumerate(lens):
        r0, r1 = row_start[b], row_start[b + 1]
        n = r1 - r0
        if n == 0 or ln <= 0:
            continue
        for h in range(H):
            c, p = read_rows(pool, pages[b], ln, h, T, D)
            s, z = p[..., :1].astype(np.float64), p[..., 1:].astype(np.float64)
            k, v = c * s + z
            mid = np.abs(s[1] * (c[1] - 8.0))
            rest = np.abs(z[1] + 8 * s[1])
            for i in range(n):
                pos = ln - n + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < lo or pos < 0:
                    continue
                at = slice(lo, pos + 1)
                for g in range(Hq // H):
                    x = q[r0 + i, h * (Hq // H) + g]
                    y = k[at] @ x * scale
                    w = np.exp(y - y.max())
                    w /= w.sum()
                    o = w @ v[at]
                    out[r0 + i, h * (Hq // H) + g] = o
                    # scores: D + 8 roundings of sums of |q| |code| s and |z| |q|
                    off = (D + 8) * 2.0 ** -24 * abs(scale) * np.abs(x).sum() * (15 * s[0][at] + np.abs(z[0][at])).max()
                    off += 2.0 ** -21 * (1 + np.abs(y - y.max()).max() * 2.0 ** -2)
                    tiles = (pos + 1 - lo) / 16 + 16
                    tol[r0 + i, h * (Hq // H) + g] = (
                        w @ mid[at] * (2.0 ** -11 + tiles * 2.0 ** -23 + 2 * off) +
                        w @ rest[at] * (tiles * 2.0 ** -23 + 2 * off) + np.abs(o) * (2 * off + tiles * 2.0 ** -24)) + (
                        (pos + 1 - lo) * s[1][at].max() * 2.0 ** -27)
    return out, tol


# ---------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------
def pages_update(pages, lens, refs, source, keep, new_lens, T):
    B, W = pages.shape
    P = len(refs)

    def clip(n):
        return min(max(int(n), 0), W * T)

    def page(b, j):
        p = int(pages[b, j])
        return p if 0 <= p < P else -1
    outside = [int(r) for r in refs]
    for b in range(B):
        for j in range(-(-clip(lens[b]) // T)):
            if page(b, j) >= 0:
                outside[page(b, j)] -= 1
    whole, parts = [0] * P, {}
    out = np.full((B, W), -1, np.int32)
    kept = []
    for b in range(B):
        s = int(source[b])
        want = clip(new_lens[b])
        k = min(clip(keep[b]), clip(lens[s]), want) if 0 <= s < B else 0
        kept.append((s, k, want))
        for j in range(k // T):
            out[b, j] = page(s, j)
            if page(s, j) >= 0:
                whole[page(s, j)] += 1
        if k % T and page(s, k // T) >= 0:
            parts.setdefault(page(s, k // T), b)
    refs_out = [max(outside[p], 0) + whole[p] for p in range(P)]
    free = [p for p in range(P) if outside[p] <= 0 and whole[p] == 0 and p not in parts]
    copies = np.full((B, 2), -1, np.int32)
    wanted = taken = 0
    for b, (s, k, want) in enumerate(kept):
        j, old = k // T, -1
        if k % T:
            p = page(s, j)
            if p >= 0 and outside[p] <= 0 and whole[p] == 0 and parts[p] == b:
                out[b, j] = p
                refs_out[p] = 1
                j += 1
            else:
                old = p
        first = j
        for j in range(j, -(-want // T)):
            wanted += 1
            if taken < len(free):
                out[b, j] = free[taken]
                refs_out[free[taken]] = 1
                if j == first and old >= 0:
                    copies[b] = old, free[taken]
                taken += 1
    return out, np.array(refs_out, np.int32), copies, np.array([len(free) - taken, wanted - taken], np.int32)


def pages_compact(pages, lens, refs, T):
    B, W = pages.shape
    P = len(refs)
    used = [p for p in range(P) if refs[p] > 0]
    n = len(used)
    holes = [p for p in range(n) if refs[p] <= 0]
    goes = {p: p for p in used}
    copies = np.full((P // 2, 2), -1, np.int32)
    for i, (p, hole) in enumerate(zip([p for p in used if p >= n], holes)):
        goes[p] = hole
        copies[i] = p, hole
    refs_out = np.zeros(P, np.int32)
    for p, to in goes.items():
        refs_out[to] = refs[p]
    out = np.full((B, W), -1, np.int32)
    for b in range(B):
        for j in range(-(-min(max(int(lens[b]), 0), W * T) // T)):
            out[b, j] = goes.get(int(pages[b, j]), -1)
    return out, refs_out, copies, np.array([n, len(holes)], np.int32)
