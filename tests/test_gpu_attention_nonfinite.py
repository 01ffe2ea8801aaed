"""Attention of the verify rows (spec_prefix_attention) with non-finite queries and keys: a row that
sees a score that is not a number shows it, in its outputs and its log sum exp, however the positions
are dealt to the SMs; every other row keeps its bytes. And scales of either sign."""

import pytest
import torch

from test_gpu_prefix_attention import Case

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
TYPES = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 72), ("f32", 64), ("f32", 256)]


@pytest.fixture(scope="module")
def spec():
    from gpu_util import ensure_built
    ensure_built()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def heads(c):
    return c.out[:, :c.Hq * c.D].float().view(c.B * c.R, c.Hq, c.D)


def check_rows(c, clean, clean_lse, bad):
    """bad [B*R, Hq]: rows that must be NaN; the others have the clean run's bytes."""
    bad = bad.cuda()
    assert torch.isnan(heads(c)[bad]).all() and torch.isnan(c.lse[bad]).all()
    assert torch.equal(heads(c)[~bad], clean[~bad]) and torch.equal(c.lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("B", [3, 24])  # the join's two forms: few output rows, many
@pytest.mark.parametrize("what", [NAN, INF])
def test_a_query_that_is_not_finite(spec, dtype, D, B, what):
    c = Case(B, 4, 8, 2, D, 300, 150, [(29 * b) % 140 for b in range(B)], dtype, seed=B)
    c.run(spec)
    clean, clean_lse = heads(c).clone(), c.lse.clone()
    bad = torch.zeros((B * 4, 8), dtype=torch.bool)
    for t, h in ((0, 3), (5, 0), (4 * B - 1, 7)):
        c.q[t, h * D + 5] = what  # an infinity times keys of either sign: both infinities are seen
        bad[t, h] = True
    c.run(spec)
    check_rows(c, clean, clean_lse, bad)


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("B", [2, 80])
def test_a_cache_of_one_position_whose_key_is_nan(spec, dtype, D, B):
    """The only position of its request's own cache: a piece of work that holds nothing else."""
    c = Case(B, 1, 8, 2, D, 200, 3, [0] * B, dtype, seed=1)
    c.run(spec)
    clean, clean_lse = heads(c).clone(), c.lse.clone()
    c.cache[1, 0, 0, 0, :D] = NAN  # request 1, KV head 0: its query heads 0..3
    c.run(spec)
    bad = torch.zeros((B, 8), dtype=torch.bool)
    bad[1, :4] = True
    check_rows(c, clean, clean_lse, bad)


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("B", [4, 40])
def test_runs_of_nan_keys(spec, dtype, D, B):
    """A whole prefix of them beside own caches without, then a run from a block's start over many
    SMs' shares, which half of the requests do not reach."""
    c = Case(B, 2, 8, 2, D, 6144, 40, [b % 38 for b in range(B)], dtype, seed=2,
             prefix_len=[6144 if b % 2 else 1024 for b in range(B)])
    c.run(spec)
    clean, clean_lse = heads(c).clone(), c.lse.clone()
    keys = c.prefix[0].clone()
    c.prefix[0] = NAN
    c.run(spec)
    check_rows(c, clean, clean_lse, torch.ones((2 * B, 8), dtype=torch.bool))
    c.prefix[0] = keys
    c.prefix[0, 1024:5120, D:2 * D] = NAN  # KV head 1: query heads 4..7
    c.run(spec)
    bad = torch.zeros((2 * B, 8), dtype=torch.bool)
    for b in range(1, B, 2):
        bad[2 * b:2 * b + 2, 4:] = True
    check_rows(c, clean, clean_lse, bad)


@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_beside_minus_infinity_alone(spec, dtype, D):
    """Scores of -Inf alone: nothing to see. One NaN among them: NaN."""
    c = Case(1, 1, 1, 1, D, 0, 300, [256], dtype, seed=3)
    c.q[0, 0] = 1.0
    c.cache[0, 0, 0, :, 0] = -INF
    c.run(spec)
    assert (heads(c) == 0).all() and torch.isneginf(c.lse).all()
    c.cache[0, 0, 0, 70, 1] = NAN
    c.run(spec)
    assert torch.isnan(heads(c)).all() and torch.isnan(c.lse).all()


@pytest.mark.parametrize("dtype,D", TYPES)
def test_negative_scale(spec, dtype, D):
    c = Case(3, 4, 8, 2, D, 333, 150, [100, 3, 62], dtype, prefix_len=[333, 0, 65], n_rows=[4, 2, 3],
             seed=4, scale=-(D ** -0.5))
    c.run(spec)
    c.check()


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("B", [2, 80])
@pytest.mark.parametrize("key", [-INF, -100.0])
def test_a_value_of_no_weight(spec, dtype, D, B, key):
    """A position that is seen with a weight of zero, from a score of -Inf or one too small for a
    float, and holds NaN or an infinity: 0 times that is NaN, in the dims where it lies and whether or
    not the position is a piece of work by itself."""
    c = Case(B, 1, 8, 2, D, 1, 300, [(53 * b) % 290 for b in range(B)], dtype, seed=5, scale=1.0)
    c.q[:] = 1.0
    c.prefix[0] = key  # the shared position; the own ones score about sqrt(D)
    c.run(spec)
    clean, lse = heads(c).clone(), c.lse.clone()
    assert torch.isfinite(clean).all()
    c.prefix[1, 0, 5], c.prefix[1, 0, D + 6] = NAN, INF
    c.run(spec)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[:, :4, 5] = bad[:, 4:, 6] = True
    assert torch.isnan(heads(c)[bad]).all()
    assert torch.equal(heads(c)[~bad], clean[~bad]) and torch.equal(c.lse, lse)
