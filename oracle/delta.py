"""The gated delta rule in float64, token by token, from its definition:

    S~ = exp(g) S,  u = beta (v - S~^T k),  S' = S~ + k u^T,  o = scale S'^T q

per value head (state [dk, dv]; value head h reads key head h // (heads // key_heads))."""

import numpy as np


def run(S0, q, k, v, g, beta, scale):
    """S0 [H, dk, dv]; q, k [n, Hk, dk]; v [n, H, dv]; g, beta [n, H]. Returns the outputs
    [n, H, dv], the state after every row [n, H, dk, dv] and the steps (a, k, u) of the rows."""
    S = np.array(S0, dtype=np.float64)
    H = S.shape[0]
    per = H // q.shape[1]
    outs, states, steps = [], [], []
    for t in range(q.shape[0]):
        kt = np.repeat(np.asarray(k[t], dtype=np.float64), per, axis=0)
        qt = np.repeat(np.asarray(q[t], dtype=np.float64), per, axis=0)
        a = np.exp(np.asarray(g[t], dtype=np.float64))
        S = a[:, None, None] * S
        u = np.asarray(beta[t], dtype=np.float64)[:, None] * (
            np.asarray(v[t], dtype=np.float64) - np.einsum("hi,hij->hj", kt, S))
        S = S + kt[:, :, None] * u[:, None, :]
        outs.append(scale * np.einsum("hi,hij->hj", qt, S))
        states.append(S)
        steps.append((a, kt, u))
    return outs, states, steps


def chunked(S0, q, k, v, g, beta, scale, chunk):
    """The same outputs and last state by chunks: (I + A) u = beta (v - exp(G) S^T k) with
    A[i, j] = beta_i exp(G_i - G_j) k_i.k_j for j < i (G: running sums of g in the chunk)."""
    S = np.array(S0, dtype=np.float64)
    H = S.shape[0]
    per = H // q.shape[1]
    n = q.shape[0]
    out = np.zeros((n, H, S.shape[2]))
    for lo in range(0, n, chunk):
        hi = min(n, lo + chunk)
        for h in range(H):
            K, Q = k[lo:hi, h // per].astype(np.float64), q[lo:hi, h // per].astype(np.float64)
            G = np.cumsum(g[lo:hi, h].astype(np.float64))
            bt = beta[lo:hi, h].astype(np.float64)
            D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0.0)))
            A = np.tril(bt[:, None] * D * (K @ K.T), -1)
            rhs = bt[:, None] * (v[lo:hi, h] - np.exp(G)[:, None] * (K @ S[h]))
            u = np.linalg.solve(np.eye(hi - lo) + A, rhs)
            out[lo:hi, h] = scale * (np.exp(G)[:, None] * (Q @ S[h]) + (D * (Q @ K.T)) @ u)
            S[h] = np.exp(G[-1]) * S[h] + (np.exp(G[-1] - G)[:, None] * K).T @ u
    return out, S
