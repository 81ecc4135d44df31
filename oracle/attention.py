"""Rotary positions and attention over pages of a cache, written from their definitions in 64 bits (angles in more)."""
import numpy as np

TWO_PI = np.longdouble("6.283185307179586476925286766559005768")


def positions(lens, lengths=None, seqs=None):
    """Position of every new token: from 0 in each sequence, or at the end of `lengths`."""
    start = [0] * len(lens) if lengths is None else [int(lengths[s]) - n for n, s in zip(lens, seqs)]
    return np.array([p + j for n, p in zip(lens, start) for j in range(n)], dtype=np.int64)


def rotary(x, pos, frequencies, interleaved=False, magnitude=1.0, inverse=False):
    """x [T, heads, D]; returns the turned x and, for bounds, |a| + |b| of each channel's pair (0 where a channel passes)."""
    x = np.asarray(x, dtype=np.float64)
    half = len(frequencies)
    angle = np.asarray(pos).astype(np.longdouble)[:, None] * np.asarray(frequencies, dtype=np.longdouble)
    angle = np.fmod(angle, TWO_PI)
    c, s = (np.asarray(f(angle), dtype=np.float64)[:, None] * magnitude for f in (np.cos, np.sin))
    if inverse:
        s = -s
    y, size = x.copy(), np.zeros_like(x)
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = (np.abs(a) + np.abs(b)) * abs(magnitude)
    return y, size


def attend(q, k_cache, v_cache, table, lengths, seqs, lens, scale, causal=True, window=0):
    """q [T, heads, D], caches [pages, page_tokens, kv_heads, D].  Returns the output, the logarithms of the sums, and for bounds:
    the weighted mean of |v|, the largest sum of |scale q k| products of a row, and the number of its keys.  Pages outside the
    cache are left out."""
    T, H, D = q.shape
    P, pt, Hk, _ = k_cache.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    size, products, count = np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H))
    t = 0
    for n, s in zip(lens, seqs):
        held = 0 <= s < len(lengths)
        length = max(int(lengths[s]), 0) if held else 0
        keys = np.arange(min(length, table.shape[1] * pt))
        page = table[s][keys // pt] if held else np.zeros(0, dtype=np.int64)
        keys, page = keys[(page >= 0) & (page < P)], page[(page >= 0) & (page < P)]
        for j in range(n):
            p = length - n + j
            seen = np.ones(len(keys), dtype=bool)
            if causal:
                seen &= keys <= p
            if window:
                seen &= keys > p - window
            if seen.any():
                k, v = (c[page[seen], keys[seen] % pt].transpose(1, 0, 2) for c in (k_cache, v_cache))  # [kv_heads, keys, D]
                x = scale * np.matmul(q[t].reshape(Hk, H // Hk, D), k.transpose(0, 2, 1))
                top = x.max(-1, keepdims=True)
                w = np.exp(x - top)
                total = w.sum(-1, keepdims=True)
                out[t] = (np.matmul(w, v) / total).reshape(H, D)
                size[t] = (np.matmul(w, np.abs(v)) / total).reshape(H, D)
                lse[t] = (top + np.log(total)).reshape(H)
                products[t] = (abs(scale) * np.matmul(np.abs(q[t]).reshape(Hk, H // Hk, D), np.abs(k).transpose(0, 2, 1))).max(-1).reshape(H)
                count[t] = x.shape[-1]
            t += 1
    return out, lse, size, products, count
