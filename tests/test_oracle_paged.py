"""Pins of the paged cache's float64 oracle."""

import numpy as np
import pytest

from oracle import attention, paged


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,D", [(0, 8), (8, 8), (6, 16), (64, 64)])
def test_rotation_is_a_complex_product(interleaved, rot, D):
    rng = np.random.default_rng(rot + D)
    x, f, pos = rng.normal(size=D), rng.uniform(1e-4, 1, rot // 2), 12345
    y = paged.turned(x, pos, None, 0, rot, interleaved, f, 1.5)
    z, w = (v[0:rot:2] + 1j * v[1:rot:2] if interleaved else v[:rot // 2] + 1j * v[rot // 2:rot]
            for v in (x, y))
    assert np.allclose(w, 1.5 * z * np.exp(1j * pos * f), atol=1e-10)
    assert np.array_equal(y[rot:], x[rot:])


def test_products_of_rotated_heads_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=32), rng.normal(size=32), 1e4 ** (-np.arange(8) / 8)

    def dot(i, j):
        return paged.turned(q, i, None, 0, 16, False, f, 1) @ paged.turned(k, j, None, 0, 16, False, f, 1)

    assert np.allclose([dot(7, 3), dot(1007, 1003)], dot(4, 0))


def test_norm():
    x, w = np.array([3.0, 4.0]), np.array([1.0, 2.0])
    assert np.allclose(paged.turned(x, 9, w, 0, 0, False, [], 1), x * w / np.sqrt(12.5))


def cache(rng, B, pages, size, H, D, n_pages):
    k, v = rng.normal(size=(n_pages, size, H, D)), rng.normal(size=(n_pages, size, H, D))
    return k, v, rng.permutation(n_pages)[:B * pages].reshape(B, pages)


def test_attention_is_that_over_the_gathered_cache():
    rng = np.random.default_rng(1)
    k, v, table = cache(rng, 2, 3, 5, 2, 4, 9)
    q = rng.normal(size=(7, 4, 4))
    out, lse = paged.attend(q, k, v, table, [4, 8], [0, 3, 6], [3, 2], 0.5)
    for b, (P, n) in enumerate([(4, 3), (8, 2)]):
        kk, vv = (x[table[b]].reshape(15, 2, 4) for x in (k, v))
        want, wl = attention.verify_rows(q[3 * b:3 * b + 3], None, None, 0, kk, vv, P, n, 0.5)
        assert np.allclose(out[3 * b:3 * b + 3], want)
        assert np.array_equal(np.isneginf(wl), np.isneginf(lse[3 * b:3 * b + 3]))
        assert np.allclose(lse[3 * b:3 * b + n], wl[:n])
    assert np.isnan(out[6]).all() and np.isnan(lse[6]).all()


def test_a_page_that_is_not_there_is_as_if_its_positions_were_not():
    rng = np.random.default_rng(2)
    k, v, table = cache(rng, 1, 4, 2, 1, 4, 6)
    q = rng.normal(size=(1, 1, 4))
    table[0, 1] = -1
    out, _ = paged.attend(q, k, v, table, [6], [0, 1], None, 1.0)
    fewer, _ = paged.attend(q, k, v, table[:, [0, 2, 3]], [4], [0, 1], None, 1.0)
    assert np.allclose(out, fewer)
    out, lse = paged.attend(q, k, v, np.full((1, 4), 6), [6], [0, 1], None, 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_append_then_commit_leaves_only_the_kept_rows():
    rng = np.random.default_rng(3)
    k, v = np.zeros((6, 4, 2, 8)), np.zeros((6, 4, 2, 8))
    table = np.array([[5, 1, -1], [0, 2, 3]])
    x = rng.normal(size=(6, 4, 8))
    f = np.array([1.0, 0.1])
    args = (table, [6, 3], [0, 3, 6], [3, 2], None, None, None, 0, 4, True, f, 1.0)
    out, status = paged.append(x, x[:, :2], x[:, 2:], k, v, *args)
    assert status.tolist() == [3, 0]  # request 0's third row is past its two pages
    assert np.isnan(out[5]).all() and np.allclose(out[0, 0], paged.turned(x[0, 0], 6, None, 0, 4, True, f, 1))
    assert np.allclose(v[1, 2], x[0, 2:]) and np.allclose(v[1, 3], x[1, 2:]) and np.allclose(v[2, 0], x[4, 2:])
    kept, lens = [1, 1], [6, 3]
    new = paged.commit(k[None], v[None], table, lens, kept, [2, 1])
    assert new == [7, 4]
    k1, v1 = np.zeros_like(k), np.zeros_like(v)
    paged.append(x, x[:, :2], x[:, 2:], k1, v1, table, lens, [0, 3, 6], kept, *args[4:])
    assert np.array_equal(k, k1) and np.array_equal(v, v1)
    assert paged.commit(k[None], v[None], table, lens, None, [2, 0]) == [8, 3] and np.array_equal(k, k1)
