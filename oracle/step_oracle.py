"""Plain fp64 CPU statements of what surrounds a drafted block: verification, the paged cache's
table calls, and shared-prefix attention.  Test infrastructure: shares no code with the CUDA path."""
import numpy as np


def softmax(z, heat=1.0):
    """Probabilities of one row of logits at a temperature; NaN reads as -inf, +inf as the largest
    finite value; all zeros when nothing is above -inf."""
    z = np.asarray(z, np.float64)
    z = np.where(np.isnan(z), -np.inf, np.minimum(z, np.finfo(np.float32).max))
    top = z.max()
    if top == -np.inf:
        return np.zeros_like(z)
    e = np.where(z > -np.inf, np.exp(np.maximum(z - top, -1e39) / heat), 0)
    return e / e.sum()


def verify(target, draft, blk, n_draft, temperature, u, noise):
    """(tokens, counts, prob, margin): margin[n] is how close (relatively) block n came to another
    result: the smallest of |u q - p| / p over its tests and 1 - second / first of its race,
    scaled by how much of p the residual cancels."""
    N, B, V = target.shape
    tokens = np.full((N, B), -1, np.int64)
    counts = np.zeros(N, np.int32)
    prob = np.zeros((N, B - 1))
    margin = np.full(N, np.inf)
    for n in range(N):
        heat = 1.0 if temperature is None else float(temperature[n])
        heat = heat if heat >= np.finfo(np.float32).tiny else 0.0
        D = B - 1 if n_draft is None else int(np.clip(n_draft[n], 0, B - 1))

        def p_of(b):
            row = np.asarray(target[n, b], np.float64)
            if heat:
                return softmax(row, heat)
            row = np.where(np.isnan(row), -np.inf, row)
            return (np.arange(V) == np.argmax(row)) * float(row.max() > -np.inf)

        def q_of(b):
            if draft is None or not heat:
                return (np.arange(V) == blk[n, 1 + b]).astype(np.float64)
            return softmax(draft[n * (B - 1) + b], heat)

        a = D
        for b in range(D):
            x, p, q = int(blk[n, 1 + b]), p_of(b), q_of(b)
            px, qx = (p[x], q[x]) if 0 <= x < V else (0.0, 1.0)
            prob[n, b] = 0.0 if px == 0 else 1.0 if qx == 0 else min(1.0, px / qx)
            if heat and px > 0:
                margin[n] = min(margin[n], abs(float(u[n, b]) * qx - px) / px)
            if not float(u[n, b]) * qx < px:
                a = b
                break
        p = p_of(a)
        tokens[n, :a] = blk[n, 1:1 + a]
        if not p.any():
            counts[n] = a
            continue
        if heat:
            w = np.maximum(p - q_of(a), 0) if a < D else p
            w = w if w.any() else p
            race = np.where(w > 0, w / np.asarray(noise[n, :V], np.float64), 0)
            order = np.argsort(-race, kind="stable")[:2]
            last = int(order[0])
            for i in order:   # cancellation in p - q widens a rounding of p
                if race[i] > 0 and len(order) > 1:
                    gap = 1 - race[order[1]] / race[order[0]]
                    margin[n] = min(margin[n], gap * min(1.0, w[i] / p[i]))
        else:
            last = int(np.argmax(p))
        tokens[n, a] = last
        counts[n] = a + 1
    return tokens, counts, prob, margin


def resize(table, lens, new_lens, refs, ps):
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    before = refs.copy()
    N, width = table.shape
    pages = lambda n: -(-n // ps)                                       # noqa: E731
    want = np.clip(new_lens, 0, width * ps)
    for n in range(N):
        low = min(lens[n], want[n])
        if want[n] != lens[n] and low % ps and before[table[n, low // ps]] > 1:
            want[n] = lens[n]
    for n in range(N):
        for j in range(pages(want[n]), pages(lens[n])):
            refs[table[n, j]] -= 1
            table[n, j] = -1
        table[n, max(pages(want[n]), pages(lens[n])):] = -1
    free = list(np.nonzero(refs == 0)[0])
    for n in range(N):
        for j in range(pages(lens[n]), pages(want[n])):
            if free:
                table[n, j] = free.pop(0)
                refs[table[n, j]] = 1
            else:
                table[n, j] = -1
                want[n] = min(want[n], j * ps)
    return table, want.astype(np.int32), refs


def fork(table, lens, parent, cut, refs, ps):
    """(child table, child lengths, refs, moves): moves = (source page, target page, tokens)."""
    refs = refs.copy()
    M, width = len(parent), table.shape[1]
    child = np.full((M, width), -1, np.int32)
    out = np.zeros(M, np.int32)
    for i, p in enumerate(parent):
        if 0 <= p < len(lens):
            out[i] = lens[p] if cut is None else min(lens[p], max(0, cut[i]))
            full = out[i] // ps
            child[i, :full] = table[p, :full]
            np.add.at(refs, child[i, :full], 1)
    free, moves = list(np.nonzero(refs == 0)[0]), []
    for i, p in enumerate(parent):
        full, part = out[i] // ps, out[i] % ps
        if part and free:
            child[i, full] = free.pop(0)
            refs[child[i, full]] = 1
            moves.append((int(table[p, full]), int(child[i, full]), int(part)))
        elif part:
            out[i] -= part
    return child, out, refs, moves


def compact(table, lens, refs, ps):
    """(table, refs, map, live, moves)."""
    live = int((refs > 0).sum())
    ids = np.arange(len(refs))
    src, dst = ids[(refs > 0) & (ids >= live)], ids[(refs <= 0) & (ids < live)]
    new = np.where(refs > 0, ids, -1)
    new[src] = dst
    out_refs = np.zeros_like(refs)
    out_refs[new[refs > 0]] = refs[refs > 0]
    out = np.full_like(table, -1)
    for n, length in enumerate(lens):
        held = -(-length // ps)
        out[n, :held] = new[table[n, :held]]
    return out, out_refs, new.astype(np.int32), live, list(zip(src.tolist(), dst.tolist()))


def attention(q, kp, vp, tails, scale):
    """q [N, T, heads, dim]; kp, vp [P, kv_heads, dim]; tails: per sequence (k, v) of its tokens.
    Returns out, lse, and for error bounds: spread = sqrt(sum_j p_j^2 v_j^2) and the largest
    sum_i |q_i k_i| * scale of each row."""
    q, kp, vp = (np.asarray(x, np.float64) for x in (q, kp, vp))
    N, T, heads, dim = q.shape
    group = heads // kp.shape[1]
    out, spread = np.zeros((N, T, heads, dim)), np.zeros((N, T, heads, dim))
    lse, size = np.full((N, T, heads), -np.inf), np.zeros((N, T, heads))
    for n in range(N):
        k = np.concatenate([kp, np.asarray(tails[n][0], np.float64)])
        v = np.concatenate([vp, np.asarray(tails[n][1], np.float64)])
        for t in range(T):
            sees = len(kp) + max(0, len(tails[n][0]) - T + t + 1)
            if sees == 0:
                continue
            for h in range(heads):
                kk, vv = k[:sees, h // group], v[:sees, h // group]
                s = kk @ q[n, t, h] * scale
                top = s.max()
                p = np.exp(s - top)
                lse[n, t, h] = top + np.log(p.sum())
                p /= p.sum()
                out[n, t, h] = p @ vv
                spread[n, t, h] = np.sqrt((p * p) @ (vv * vv))
                size[n, t, h] = (np.abs(kk) @ np.abs(q[n, t, h])).max() * abs(scale)
    return out, lse, spread, size
