"""Plain numpy forms of the paged cache, rotary positions and attention, in f64
(tests only): what include/qmm.h defines, one token at a time."""
import numpy as np

F16, Q8_0 = 1, 8
INTERLEAVED, HALF = 0, 1


def record(dtype, page, dim):
    return 2 * page * dim if dtype == F16 else page * dim + page * dim // 16


def fields(pool, dtype, page, heads, dim, values):
    """(codes or f16 values, scales or None): views of a pool's bytes, [pages][heads] in front."""
    shape = (dim, page) if values else (page, dim)
    r = pool.reshape(-1, heads, record(dtype, page, dim))
    if dtype == F16:
        return r.view(np.float16).reshape(-1, heads, *shape), None
    n = page * dim
    return (r[..., :n].view(np.int8).reshape(-1, heads, *shape),
            np.ascontiguousarray(r[..., n:]).view(np.float16).reshape(-1, heads, dim // 32, page))


def decoded(pool, dtype, page, heads, dim, values):
    """f64 [pages][heads][page][dim]."""
    a, sc = fields(pool, dtype, page, heads, dim, values)
    x = a.astype(np.float64)
    if values:
        x = x.transpose(0, 1, 3, 2)
    if sc is not None:
        with np.errstate(invalid="ignore"):
            x = x * np.repeat(sc.astype(np.float64).transpose(0, 1, 3, 2), 32, axis=3)
    return x


def rotate(x, pos, freqs, rot, layout, mscale=1.0):
    """x f64 [..., D], one position for all."""
    a = float(pos) * freqs.astype(np.float64)
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    y = x.copy()
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == HALF else (slice(0, rot, 2), slice(1, rot, 2))
    u, w = x[..., i], x[..., j]
    y[..., i], y[..., j] = u * c - w * s, u * s + w * c
    return y


def unit(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def places(table, lens, starts, new, page, pages, rows, max_pages):
    """Per row: (sequence, index, page id or -1); None for padding."""
    out = [None] * rows
    for s in range(len(lens)):
        first = starts[s] if starts is not None else s * new
        n = starts[s + 1] - starts[s] if starts is not None else new
        for t in range(min(n, new)):
            i = lens[s] - n + t
            p = -1
            if 0 <= i < max_pages * page:
                p = int(table[s][i // page])
                p = p if 0 <= p < pages else -1
            if 0 <= first + t < rows:
                out[first + t] = (s, i, p)
    return out


def visible(s, i, table, lens, page, pages, max_pages, causal, window):
    """Indices of the tokens that index i of sequence s sees."""
    j = np.arange(max(0, min(int(lens[s]), max_pages * page)))
    if causal:
        j = j[j <= i]
        if window:
            j = j[j > i - window]
    pg = np.asarray(table[s])[j // page]
    return j[(pg >= 0) & (pg < pages)]


def attend(q, keys, vals, scale, softcap=0.0):
    """q [D], keys and vals [n][D], all f64: (output, probabilities, scores)."""
    if len(keys) == 0:
        return np.zeros(vals.shape[1]), np.zeros(0), np.zeros(0)
    x = (keys @ q) * scale
    if softcap:
        x = softcap * np.tanh(x / softcap)
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ vals, p, x
