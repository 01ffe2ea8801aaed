"""A KV cache in pages, in float64: norms, rotation and append of new rows, attention from them, commit.

Pins: ``tests/test_oracle_paged.py`` (the rotation against complex multiplication and its invariance of
position differences, attention against the contiguous oracle, the commit against a cache that never held
the rows)."""

import numpy as np

from . import attention


def place(table_row, pos, page_size, n_pages):
    """(page, position in it) of a position, or None where it lies past the table or its page is not there."""
    j = pos // page_size
    if pos < 0 or j >= len(table_row) or not 0 <= int(table_row[j]) < n_pages:
        return None
    return int(table_row[j]), pos % page_size


def turned(x, pos, weight, eps, rot, interleaved, inv_freq, scale):
    """One head: its norm (weight None: none), then its first `rot` dims rotated for position pos."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(weight, dtype=np.float64)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = float(pos) * float(inv_freq[i])
        c, s = scale * np.cos(t), scale * np.sin(t)
        y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


def rows_of(cu, n_rows, rows, b):
    """First row, rows owned and rows run of request b, with what is out of range clamped."""
    start = min(max(int(cu[b]), 0), rows)
    owned = max(start, min(int(cu[b + 1]), rows)) - start
    return start, owned, owned if n_rows is None else min(max(int(n_rows[b]), 0), owned)


def append(q, k, v, k_pages, v_pages, table, kv_len, cu, n_rows, pos, q_norm, k_norm, eps, rot, interleaved,
           inv_freq, scale):
    """q [T, Hq, D], k and v [T, Hkv, D]; pages [n_pages, page_size, Hkv, D] float64, written in place. The
    queries (NaN where a row does not run) and each request's status (3: not all of it has a place)."""
    out = np.full(q.shape, np.nan)
    status = np.zeros(len(table), dtype=np.int64)
    for b in range(len(table)):
        start, _, n = rows_of(cu, n_rows, len(q), b)
        P = max(int(kv_len[b]), 0)
        for r in range(n):
            t, at = start + r, (P if pos is None else int(pos[b])) + r
            for h in range(q.shape[1]):
                out[t, h] = turned(q[t, h], at, q_norm, eps, rot, interleaved, inv_freq, scale)
            w = place(table[b], P + r, k_pages.shape[1], len(k_pages))
            if w is None:
                status[b] = 3
                continue
            for h in range(k.shape[1]):
                k_pages[w][h] = turned(k[t, h], at, k_norm, eps, rot, interleaved, inv_freq, scale)
            v_pages[w] = v[t]
    return out, status


def attend(q, k_pages, v_pages, table, kv_len, cu, n_rows, scale):
    """q [T, Hq, D]. Output and lse; NaN in rows that nobody owns, zero and -inf in owned ones that do
    not run."""
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    size, G = k_pages.shape[1], q.shape[1] // k_pages.shape[2]
    for b in range(len(table)):
        start, owned, n = rows_of(cu, n_rows, len(q), b)
        out[start:start + owned], lse[start:start + owned] = 0, -np.inf
        P = min(max(int(kv_len[b]), 0), len(table[b]) * size)
        at = [place(table[b], p, size, len(k_pages)) for p in range(P + n)]
        for r in range(n):
            seen = [w for w in at[:P + r + 1] if w is not None]
            pages, within = [w[0] for w in seen], [w[1] for w in seen]
            for h in range(q.shape[1]):
                out[start + r, h], lse[start + r, h] = attention.row(
                    q[start + r, h], k_pages[pages, within, h // G], v_pages[pages, within, h // G], scale)
    return out, lse


def commit(k_pages, v_pages, table, kv_len, kept, k):
    """Pages [layers, n_pages, page_size, ...], cleared in place; the new lengths. kept None: k rows each are
    kept."""
    size, out = k_pages.shape[2], []
    for b in range(len(table)):
        P = max(int(kv_len[b]), 0)
        m = int(k[b]) if kept is None else int(kept[b])
        out.append(P + m)
        for p in range(P + m, P + int(k[b]) + (kept is not None)):
            w = place(table[b], p, size, k_pages.shape[1])
            if w is not None:
                k_pages[(slice(None),) + w] = 0
                v_pages[(slice(None),) + w] = 0
    return out
