"""The paged cache's calls with the token mixers, the LM head, the acceptance and the commit, as
examples/hybrid_trunk.py runs them: greedy decoding over pages, of which the requests share the prompt's,
gives the tokens of the contiguous caches, and drafts do not change them. fp32, so that no token hangs on
a bf16 rounding."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module")
def example():
    from gpu_util import ensure_built
    ensure_built()
    import hybrid_trunk
    return hybrid_trunk


SMALL = dict(dtype=torch.float32, d=128, vocab=1024, delta_layers=2, heads=4, key_heads=2, dk=32,
             dv=16, q_heads=4, kv_heads=2, head_dim=32)


def _prompt(n):
    return torch.randint(900, (n,), generator=torch.Generator().manual_seed(3)).tolist()


@pytest.mark.parametrize("page,prompt", [(16, 70), (16, 65), (1, 20), (24, 12), (64, 130)])
def test_pages_give_the_tokens_of_contiguous_caches(example, page, prompt):
    p = _prompt(prompt)
    plain, _ = example.decode(example.HybridTrunk(3, 1, 64, **SMALL), p, 24)
    got, _ = example.decode(example.HybridTrunk(3, 1, 64, paged=True, page=page, **SMALL), p, 24)
    assert got == plain


@pytest.mark.parametrize("mode", ["snapshot", "replay", "index"])
@pytest.mark.parametrize("requests,drafts,rot", [(1, 7, 0), (2, 3, 32), (4, 1, 16)])
def test_drafts_do_not_change_the_tokens(example, mode, requests, drafts, rot):
    p = _prompt(70)
    kw = dict(mode=mode, paged=True, rot=rot, **SMALL)
    plain, cycles = example.decode(example.HybridTrunk(requests, 1, 64, **kw), p, 24)
    assert cycles == 24
    trunk = example.HybridTrunk(requests, drafts + 1, 64, **kw)
    got, n = example.decode(trunk, p, 24, example.noisy_drafts(plain, 1024, 0.3), drafts)
    assert got == plain
    right, fewer = example.decode(trunk, p, 24, example.noisy_drafts(plain, 1024, 0.0), drafts)
    assert right == plain and fewer == -(-24 // (drafts + 1)) and fewer <= n <= 24


def test_bf16_decodes(example):
    trunk = example.HybridTrunk(2, 4, 64, paged=True, rot=64)
    tokens, n = example.decode(trunk, list(range(10, 300)), 12, lambda b, done, k: [1] * k, 3)
    assert all(len(t) == 12 for t in tokens) and n <= 12
