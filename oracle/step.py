"""The steps around a projection in float64 numpy, from their definitions:
norms around a block, low-rank adapters, verification of drafted tokens.
Slow and plain; shares no code with the CUDA library.

Each function also returns what an error bound needs (sums of magnitudes), in
the manner of the matmul oracle."""
import numpy as np

U32 = 2.0 ** -24                                   # unit roundoffs
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}   # half the smallest step


def rms(v, eps):
    return v / np.sqrt((v * v).sum(axis=-1, keepdims=True) / v.shape[-1] + eps)


def activation(gate, act):
    g = np.asarray(gate, dtype=np.float64)
    if act is None:
        return g
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return g * s if act == "silu" else s


def rmsnorm(r, w, eps):
    x = rms(np.asarray(r, dtype=np.float64), eps)
    return x if w is None else x * np.asarray(w, dtype=np.float64)


def norm_residual(y, r, w_post, gate, act, w_next, eps, alpha, post):
    """-> (r', x', |alpha act(gate) n|)."""
    n = np.asarray(y, dtype=np.float64)
    if post:
        n = rmsnorm(n, w_post, eps)
    elif w_post is not None:
        n = n * np.asarray(w_post, dtype=np.float64)
    add = alpha * n
    if gate is not None:
        add = add * activation(gate, act)
    r2 = np.asarray(r, dtype=np.float64) + add
    return r2, rmsnorm(r2, w_next, eps), np.abs(add)


def lora(x, A, B, ids, ranks, scales, y):
    """-> (y', tolerance terms (bound_v, bound_split, bound_sum)): for each
    output scale * sum_r |B| sum_k |x A|, scale * max_r |v| sum_r |B| and
    scale * sum_r |v B|."""
    x, A, B, y = (np.asarray(t, dtype=np.float64) for t in (x, A, B, y))
    out = y.copy()
    bv, bs, bm = np.zeros_like(y), np.zeros_like(y), np.zeros_like(y)
    for m, l in enumerate(ids):
        if l < 0 or l >= A.shape[0]:
            continue
        rank = A.shape[1] if ranks is None else int(ranks[l])
        s = 1.0 if scales is None else float(scales[l])
        a, b = A[l, :rank], B[l, :, :rank]
        v = a @ x[m]
        out[m] += s * (b @ v)
        bv[m] = abs(s) * (np.abs(b) @ (np.abs(a) @ np.abs(x[m])))
        bs[m] = abs(s) * np.abs(b).sum(axis=1) * (np.abs(v).max() if rank else 0.0)
        bm[m] = abs(s) * (np.abs(b) @ np.abs(v))
    return out, (bv, bs, bm)


def verify(logits, row_start, drafts, q, u, e, temperature):
    """-> (accepted [B], tokens [rows], margin): margin is the smallest
    relative distance of any decision (a draft's test, the drawn token against
    the runner-up) from a tie."""
    logits = np.asarray(logits, dtype=np.float64)
    rows, V = logits.shape
    nb = len(row_start) - 1
    accepted = np.zeros(nb, dtype=np.int32)
    tokens = np.full(rows, -1, dtype=np.int32)
    margin = np.inf

    def draw(w, b):
        nonlocal margin
        score = np.where(w > 0, w / np.asarray(e[b], dtype=np.float64), 0.0)
        if not (score > 0).any():
            return -1
        top = np.sort(score)[-2:]
        margin = min(margin, (top[-1] - top[0]) / top[-1] if V > 1 else np.inf)
        return int(score.argmax())

    for b in range(nb):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        for row in range(r0, r1):
            l, t, d = logits[row], float(temperature[b]), int(drafts[row])
            last = row == r1 - 1 or not 0 <= d < V
            top = l.max()
            allowed = top > -np.inf
            if not t > 0:
                best = int(l.argmax()) if allowed else -1
                if not last and d == best:
                    tokens[row] = d
                    accepted[b] += 1
                    continue
                tokens[row] = best
                break
            p = np.exp((l - top) / t) if allowed else np.zeros(V)
            p = p / p.sum() if allowed else p
            if last:
                tokens[row] = draw(p, b)
                break
            qd = 1.0 if q is None else float(q[row, d])
            lhs = float(u[row]) * qd
            if lhs > 0 or p[d] > 0:
                margin = min(margin, abs(lhs - p[d]) / max(lhs, p[d]))
            if lhs < p[d]:
                tokens[row] = d
                accepted[b] += 1
                continue
            if q is None:
                w = p.copy()
                w[d] = 0.0
            else:
                w = np.maximum(p - np.asarray(q[row], dtype=np.float64), 0.0)
            tokens[row] = draw(w if (w > 0).any() else p, b)
            break
    return accepted, tokens, margin
