"""Pins of the float64 oracles of the trunk's token mixers."""

import numpy as np
import pytest

from oracle import attention as o_at
from oracle import delta as o_de
from oracle import state as o_st


def _inputs(rng, n, H, Hk, dk, dv):
    k = rng.standard_normal((n, Hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return (rng.standard_normal((H, dk, dv)), rng.standard_normal((n, Hk, dk)), k,
            rng.standard_normal((n, H, dv)), -rng.random((n, H)) * 2, rng.random((n, H)))


@pytest.mark.parametrize("n,chunk", [(1, 4), (7, 4), (16, 4), (33, 8), (5, 64)])
def test_chunked_equals_the_recurrence(n, chunk):
    S0, q, k, v, g, beta = _inputs(np.random.default_rng(n), n, 4, 2, 6, 5)
    outs, states, _ = o_de.run(S0, q, k, v, g, beta, 0.3)
    out, S = o_de.chunked(S0, q, k, v, g, beta, 0.3, chunk)
    np.testing.assert_allclose(out, np.stack(outs), atol=1e-12)
    np.testing.assert_allclose(S, states[-1], atol=1e-12)


def test_delta_rule_stores_and_overwrites():
    """beta = 1, no decay, unit key: reading the key back gives the last value written."""
    rng = np.random.default_rng(0)
    S0, q, k, v, g, beta = _inputs(rng, 2, 1, 1, 8, 4)
    k[1] = k[0]
    _, states, _ = o_de.run(S0, q, k, v, g * 0, beta * 0 + 1, 1.0)
    np.testing.assert_allclose(states[1][0].T @ k[1, 0], v[1, 0], atol=1e-12)


def test_steps_are_the_commit_step():
    rng = np.random.default_rng(1)
    S0, q, k, v, g, beta = _inputs(rng, 3, 2, 2, 4, 4)
    _, states, steps = o_de.run(S0, q, k, v, g, beta, 1.0)
    S = S0
    for (a, kk, u), want in zip(steps, states):
        S = a[:, None, None] * S + kk[:, :, None] * u[:, None, :]
        np.testing.assert_allclose(S, want, atol=1e-13)
    assert hasattr(o_st, "commit_replay")


def test_attention_is_the_softmax_over_both_parts():
    rng = np.random.default_rng(2)
    q = rng.standard_normal((2, 4, 8))
    pk, pv = rng.standard_normal((2, 5, 2, 8))
    ok, ov = rng.standard_normal((2, 6, 2, 8))
    out, lse = o_at.verify_rows(q, pk, pv, 3, ok, ov, 2, 2, 0.5)
    ks, vs = np.concatenate([pk[:3, 1], ok[:4, 1]]), np.concatenate([pv[:3, 1], ov[:4, 1]])
    w = np.exp(0.5 * ks @ q[1, 3])
    np.testing.assert_allclose(out[1, 3], w @ vs / w.sum(), atol=1e-12)
    np.testing.assert_allclose(lse[1, 3], np.log(w.sum()), atol=1e-12)
    out, lse = o_at.verify_rows(q, pk, pv, 3, ok, ov, 2, 1, 0.5)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
