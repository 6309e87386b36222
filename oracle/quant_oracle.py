"""The quantised cache and the log probabilities in 64 bits, one element or row at a time as they are
defined (test infrastructure: nothing in the package imports it)."""
import numpy as np


def scale_values():
    """The 256 scales: a byte's 16-bit float is the one whose bits are the byte << 7 (the last 8 are not used)."""
    with np.errstate(invalid="ignore"):
        return (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def most_of(bits):
    return 2 ** (bits - 1) - 1


def top_byte(bits):
    """The greatest scale: 512 of 8 bits, 7680 of 4."""
    return int(np.nonzero(scale_values()[:0xF8] == (512 if bits == 8 else 7680))[0][0])


def quantise(x, bits):
    """Rows [..., dim] -> (codes int [..., dim], scale bytes [..., dim/16], whether anything did not fit)."""
    x = np.asarray(x, np.float64)
    bad = bool(np.isnan(x).any())
    x = np.where(np.isnan(x), 0.0, x)
    groups = x.reshape(x.shape[:-1] + (-1, 16))
    most, s = most_of(bits), scale_values()[:top_byte(bits) + 1]
    top = np.abs(groups).max(-1)
    byte = np.searchsorted(s * most, top)          # the least scale that reaches the largest
    bad |= bool((byte == len(s)).any())
    byte = np.minimum(byte, len(s) - 1)
    step = s[byte][..., None]
    code = np.clip(np.rint(np.divide(groups, step, out=np.zeros_like(groups), where=step > 0)), -most, most)
    return code.reshape(x.shape).astype(np.int64), byte, bad


def values(codes, byte):
    return codes * np.repeat(scale_values()[byte], 16, -1)


def sizes(page_size, dim, bits):
    """(bytes of a token's codes, of its scales, of a head of a page)"""
    code, scale = dim * bits // 8, -(-(dim // 16) // 4) * 4
    return code, scale, -(-page_size * (code + scale) // 16) * 16


def put(head, t, codes, byte, page_size, bits):
    """Write a token's codes and scales into the bytes of one head of a page."""
    dim = len(codes)
    code, scale, _ = sizes(page_size, dim, bits)
    if bits == 8:
        head[t * code:(t + 1) * code] = codes + 128
    else:
        for w in range(dim // 8):
            word = 0
            for j in range(4):
                for e in range(2):
                    word |= int(codes[8 * w + 2 * j + e] + 8) << 4 * (j + 4 * e)
            head[t * code + 4 * w:t * code + 4 * w + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
    at = page_size * code + t * scale
    head[at:at + scale] = 0
    head[at:at + dim // 16] = byte


def get(head, t, page_size, dim, bits):
    """The values [dim] that a token of one head of a page stands for."""
    code, scale, _ = sizes(page_size, dim, bits)
    raw = head[t * code:(t + 1) * code]
    if bits == 8:
        codes = raw.astype(np.int64) - 128
    else:
        words = raw.copy().view(np.uint32)
        codes = np.array([int(words[d // 8]) >> 4 * (d % 8 // 2 + d % 2 * 4) & 15 for d in range(dim)]) - 8
    at = page_size * code + t * scale
    return values(codes, head[at:at + dim // 16])


def attention(q, k, v, sees, scale):
    """Queries [T, heads, dim] over keys and values [L, kv_heads, dim], query t those before sees[t].
    Returns out, lse and what bounds an implementation's error: the weighted mean of |v| [T, heads, dim] and
    the largest scale * sum |q||k| of a row [T, heads]."""
    T, heads, dim = q.shape
    group = heads // k.shape[1]
    out, lse = np.zeros((T, heads, dim)), np.full((T, heads), -np.inf)
    mean, size = np.zeros((T, heads, dim)), np.zeros((T, heads))
    for t in range(T):
        n = max(0, int(sees[t]))
        if n == 0:
            continue
        kk, vv = (np.repeat(x[:n], group, 1) for x in (k, v))
        z = np.einsum("hd,jhd->hj", q[t], kk) * scale
        size[t] = (np.einsum("hd,jhd->hj", np.abs(q[t]), np.abs(kk)) * scale).max(1)
        m = z.max(1, keepdims=True)
        p = np.exp(z - np.where(np.isfinite(m), m, 0.0))
        total = p.sum(1)
        with np.errstate(divide="ignore"):
            lse[t] = np.where(total > 0, m[:, 0] + np.log(total), -np.inf)
        w = p / np.where(total > 0, total, 1.0)[:, None]
        out[t], mean[t] = np.einsum("hj,jhd->hd", w, vv), np.einsum("hj,jhd->hd", w, np.abs(vv))
    return out, lse, mean, size


def logprobs(logits, token, temperature, top):
    """(logprob, entropy, rank, top ids, top logprobs) of one row."""
    l = np.asarray(logits, np.float64)
    if token == -1:
        return 0.0, 0.0, 0, [-1] * top, [0.0] * top
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    order = sorted(range(len(l)), key=lambda v: (-l[v], v))
    rank = order.index(token) + 1
    ids = [v for v in order[:top] if l[v] > -np.inf]
    rest = top - len(ids)
    if l.max() == -np.inf:
        return -np.inf, 0.0, rank, [-1] * top, [-np.inf] * top
    if temperature < np.finfo(np.float32).tiny:
        p = [0.0 if v == order[0] else -np.inf for v in ids]
        return (0.0 if rank == 1 else -np.inf), 0.0, rank, ids + [-1] * rest, p + [-np.inf] * rest
    z = (l - l.max()) / temperature
    log_p = z - np.log(np.exp(z).sum())
    seen = log_p[np.exp(log_p) > 0]
    entropy = -(np.exp(seen) * seen).sum()
    return (log_p[token], entropy, rank, ids + [-1] * rest, [log_p[v] for v in ids] + [-np.inf] * rest)
