"""The token mixers, the LM head, the acceptance and the commit together, as examples/hybrid_trunk.py
runs them: greedy decoding with drafts, right and wrong ones, gives the tokens of decoding without,
whichever way the commit keeps the state. fp32, so that no token hangs on a bf16 rounding: two runs
differ by the order of a few fp32 sums, and the top two of the 1,024 logits lie much further apart."""

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


@pytest.mark.parametrize("mode", ["snapshot", "replay", "index"])
@pytest.mark.parametrize("requests,drafts", [(1, 7), (2, 3), (4, 1)])
def test_drafts_do_not_change_the_tokens(example, mode, requests, drafts):
    prompt = torch.randint(900, (70,), generator=torch.Generator().manual_seed(3)).tolist()
    plain, cycles = example.decode(example.HybridTrunk(requests, 1, 64, mode=mode, **SMALL),
                                   prompt, 24)
    assert cycles == 24
    trunk = example.HybridTrunk(requests, drafts + 1, 64, mode=mode, **SMALL)
    got, n = example.decode(trunk, prompt, 24, example.noisy_drafts(plain, 1024, 0.3), drafts)
    assert got == plain
    right, fewer = example.decode(trunk, prompt, 24, example.noisy_drafts(plain, 1024, 0.0), drafts)
    assert right == plain and fewer == -(-24 // (drafts + 1)) and fewer <= n <= 24


def test_bf16_decodes(example):
    trunk = example.HybridTrunk(2, 4, 64)
    prompt = list(range(10, 300))
    tokens, n = example.decode(trunk, prompt, 12, lambda b, done, k: [1] * k, 3)
    assert all(len(t) == 12 for t in tokens) and n <= 12
