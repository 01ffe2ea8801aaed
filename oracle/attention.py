"""Attention of verify rows over a shared prefix and a request's own cache, in float64."""

import numpy as np


def row(q, keys, values, scale):
    """softmax(scale q.K) V of one query over the positions it sees; the output and log sum exp.
    Nothing to see: zeros and -inf."""
    q = np.asarray(q, dtype=np.float64)
    if len(keys) == 0:
        return np.zeros_like(q), -np.inf
    s = scale * (np.asarray(keys, dtype=np.float64) @ q)
    m = s.max()
    w = np.exp(s - m)
    return (w @ np.asarray(values, dtype=np.float64)) / w.sum(), m + np.log(w.sum())


def verify_rows(q, prefix_k, prefix_v, prefix_len, own_k, own_v, kv_len, n_rows, scale):
    """q [R, Hq, D]; prefix [P, Hkv, D] or None; own [cap, Hkv, D]; one request. Row r sees the
    first prefix_len prefix positions and own positions 0..kv_len + r (below cap)."""
    R, Hq, D = q.shape
    cap, Hkv = own_k.shape[:2]
    out = np.zeros((R, Hq, D))
    lse = np.full((R, Hq), -np.inf)
    for r in range(min(R, max(n_rows, 0))):
        end = min(max(kv_len, 0) + r + 1, cap)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            ks, vs = own_k[:end, kh], own_v[:end, kh]
            if prefix_k is not None:
                n = min(max(prefix_len, 0), len(prefix_k))
                ks = np.concatenate([prefix_k[:n, kh], ks])
                vs = np.concatenate([prefix_v[:n, kh], vs])
            out[r, h], lse[r, h] = row(q[r, h], ks, vs, scale)
    return out, lse
