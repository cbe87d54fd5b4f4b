"""fp64 oracle of the ragged serving step: block tables and slots from lengths, rotary
positions with several axes, and attention with a sliding window and sinks, for decode
and for chunks of several requests. Slow and direct; pools as in tq4_oracle."""
from __future__ import annotations

import numpy as np

from oracle import tq4_oracle as O


# ---------------------------------------------------------------- plan
def plan_step(past, new, free, tables, num_pages, max_tok):
    """One request after the other. Returns (tables, cu, seq_lens, pos, slot, taken, codes):
    codes is the set of problems met ("seq", "pages", "page_range")."""
    tables = np.array(tables, np.int64)
    n, max_pages = len(past), tables.shape[1]
    cu, lens = np.zeros(n + 1, np.int64), np.zeros(n, np.int64)
    pos, slot = np.zeros(max_tok, np.int64), np.full(max_tok, -1, np.int64)
    asked = taken = 0
    codes = set()
    for r in range(n):
        p, m = int(past[r]), int(new[r])
        bad = p < 0 or m < 0 or p + m > max_pages * O.PAGE
        rows = max(m, 0)
        has, need = -(-p // O.PAGE), -(-(p + m) // O.PAGE)
        fresh = 0 if bad else need - has
        bad = bad or cu[r] + rows > max_tok
        fits = not bad and (fresh == 0 or asked + fresh <= len(free))
        if bad:
            codes.add("seq")
        elif not fits:
            codes.add("pages")
        if fits:
            tables[r, has:need] = free[asked:asked + fresh]
            lens[r] = p + m
            taken = max(taken, asked + fresh) if fresh else taken
        asked += fresh
        a = int(cu[r])
        cu[r + 1] = min(a + rows, max_tok)
        known = not (p < 0 or m < 0 or p + m > max_pages * O.PAGE)
        for i in range(int(cu[r + 1]) - a):
            at = (p if known else 0) + i
            pos[a + i] = at
            if fits:
                page = int(tables[r, at // O.PAGE])
                if 0 <= page < num_pages:
                    slot[a + i] = page * O.PAGE + at % O.PAGE
                else:
                    codes.add("page_range")
    return tables, cu, lens, pos, slot, taken, codes


# ---------------------------------------------------------------- rotary positions
def rope_axes(half, sections, interleaved):
    """The axis of each of `half` frequencies."""
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    k = len(sections)
    return np.array([i % k if i < k * sections[i % k] else 0 for i in range(half)])


def rope_turn(x, cos, sin, adjacent):
    """x [n, heads, 256] with pair i of its first 2 * cos.shape[1] dims turned by (cos, sin)[n, i]."""
    x = np.asarray(x, np.float64)
    half = cos.shape[1]
    a = slice(0, 2 * half, 2) if adjacent else slice(0, half)
    b = slice(1, 2 * half, 2) if adjacent else slice(half, 2 * half)
    z = (x[..., a] + 1j * x[..., b]) * (cos + 1j * sin)[:, None, :]   # a rotation is a complex product
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def half_of(x):
    """fp64 to the nearest fp16, ties to even, in one rounding."""
    return np.asarray(x, np.float64).astype(np.float16)


def store(pool, slots, k, v, signs, centroids):
    """Encode k, v [n, 4, 256] into their slots (negative: skipped). Returns the rotated coordinates (yk, yv)."""
    slots = np.asarray(slots)
    live = slots >= 0
    page, off = slots[live] // O.PAGE, slots[live] % O.PAGE
    kw, vw, kn, vn = O._regions(pool)
    ys = []
    for x, words, norms in ((k, kw, kn), (v, vw, vn)):
        w, n, y = O.encode_vectors(np.asarray(x)[live], signs, centroids)
        for h in range(O.H_KV):
            words[page, h, off] = w[:, h]
            norms[page, h, off] = n[:, h]
        ys.append(y)
    return ys


# ---------------------------------------------------------------- windowed attention
def visible(positions, at, window, sinks):
    """Which of `positions` a query at position `at` sees."""
    positions = np.asarray(positions)
    return (positions <= at) & ((positions > at - window) | (positions < sinks))


def _rows(pool, table, pos, signs, centroids):
    """K and V [len(pos), 4, 256] stored at these positions of one request."""
    kw, vw, kn, vn = O._regions(pool)
    page, off = O._locate(table, pos)
    out = []
    for words, norms in ((kw, kn), (vw, vn)):
        w = np.stack([words[page, h, off] for h in range(O.H_KV)], 1)
        n = np.stack([norms[page, h, off] for h in range(O.H_KV)], 1)
        out.append(O.decode_vectors(w, n, signs, centroids))
    return out


def _attend(q, k, v, see, scale):
    """q [n, 24, 256], k, v [P, 4, 256], see [n, P]: softmax over the visible positions only."""
    out = np.zeros(q.shape, np.float64)
    for h in range(O.H_Q):
        s = np.where(see, scale * (q[:, h] @ k[:, h // O.GROUP].T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        out[:, h] = (p / p.sum(1, keepdims=True)) @ v[:, h // O.GROUP]
    return out


def request_attention(pool, table, T, q, window, sinks, scale, signs, centroids, k_new=None, v_new=None):
    """The last len(q) positions of a request of length T. k_new, v_new: those positions' own keys
    and values at full precision (a chunk); None: all from the pool. Only visible positions are read."""
    q = np.asarray(q, np.float64)
    n = q.shape[0]
    at = np.arange(T - n, T)
    some = visible(np.arange(T)[None], at[:, None], window, sinks).any(0)
    pos = np.flatnonzero(some)
    if k_new is None:
        k, v = _rows(pool, table, pos, signs, centroids)
    else:
        old = pos[pos < T - n]
        k, v = _rows(pool, table, old, signs, centroids) if old.size else (np.zeros((0, O.H_KV, O.D)),) * 2
        mine = pos[pos >= T - n] - (T - n)
        k = np.concatenate([k, np.asarray(k_new, np.float64)[mine]])
        v = np.concatenate([v, np.asarray(v_new, np.float64)[mine]])
    return _attend(q, k, v, visible(pos[None], at[:, None], window, sinks), scale)


def decode_attention_window(pool, tables, seq_lens, q, window, sinks, scale, signs, centroids):
    """q [n_req, n_q, 24, 256]; requests of length 0 give zeros."""
    out = np.zeros(np.shape(q), np.float64)
    for r, T in enumerate(seq_lens):
        if T:
            out[r] = request_attention(pool, tables[r], int(T), q[r], window, sinks, scale, signs, centroids)
    return out


def prefill_attention_ragged(pool, tables, seq_lens, cu, q, k, v, window, sinks, scale, signs, centroids):
    """q [rows, 24, 256], k, v [rows, 4, 256]: request r's chunk is rows cu[r] .. cu[r + 1] - 1; the rest is 0."""
    out = np.zeros(np.shape(q), np.float64)
    for r, T in enumerate(seq_lens):
        a, b = int(cu[r]), int(cu[r + 1])
        if T and b > a:
            out[a:b] = request_attention(pool, tables[r], int(T), q[a:b], window, sinks, scale, signs, centroids,
                                         k[a:b], v[a:b])
    return out
