"""The gated delta rule over prompts (spec_delta_prefill) with non-finite inputs: what a token holds
reaches that token and, through the state, the ones after it, in the columns and heads that the
formula takes it to, and nothing else. The float64 recurrence says which outputs and states are finite;
those have the bytes of the run without the value."""

import numpy as np
import pytest
import torch

from test_gpu_delta import Rows, State, npf

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
LENS = [150, 70, 131]


@pytest.fixture(scope="module")
def spec():
    from gpu_util import ensure_built
    ensure_built()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def prefill(spec, x, lens, S0):
    s = State(spec, len(lens), 1, x.H, x.dk, x.dv, 2)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    ws = torch.zeros(spec.spec_delta_prefill_workspace_bytes(sum(lens), len(lens), s.st),
                     dtype=torch.uint8).cuda()
    spec.spec_delta_prefill(len(lens), cu, sum(lens), s.st, 0, x.desc(spec), S0, ws)
    torch.cuda.synchronize()
    assert int(ws[4:8].cpu().numpy().view(np.uint32)[0]) == 0
    return npf(x.out[:, :x.H * x.dv]).reshape(-1, x.H, x.dv), npf(s.live[:, 0])


def compare(x, lens, S0, clean, got):
    lo = 0
    for b, n in enumerate(lens):
        with np.errstate(all="ignore"):
            outs, states, _ = x.oracle(npf(S0[b, 0]), lo, lo + n)
        for name, want, c, g in (("out", np.stack(outs), clean[0][lo:lo + n], got[0][lo:lo + n]),
                                 ("state", states[-1], clean[1][b], got[1][b])):
            fin = np.isfinite(want)
            assert np.array_equal(np.isfinite(g), fin), (b, name, np.argwhere(np.isfinite(g) != fin)[:5])
            assert np.array_equal(g[fin], c[fin]), (b, name)
        lo += n


# chunks, the row scan (other types and sizes)
SHAPES = [(4, 2, 128, 32, "bf16"), (4, 2, 128, 32, "f32"), (2, 1, 64, 32, "bf16")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("field,what", [(f, w) for f in ("q", "k", "v", "beta") for w in (NAN, INF)] +
                         [("g", NAN)])  # log decays are <= 0
def test_a_token_reaches_no_token_before_it(spec, shape, field, what):
    H, Hk, dk, dv, dtype = shape
    x = Rows(sum(LENS), H, Hk, dk, dv, dtype, seed=1)
    S0 = (torch.randn((3, 1, H, dk, dv), generator=torch.Generator().manual_seed(2)) * 0.5).cuda()
    clean = prefill(spec, x, LENS, S0)
    t = getattr(x, field)
    # of the first and the last request: places in a chunk, a step of 16 and a pair of tokens
    for j in (0, 5, 15, 16, 30, 37, 40, 63, 64, 100, 149):
        at, last = (j, 2 if field in "qk" else 1), 220 + min(j, 130)
        keep = t[[at[0], last]].clone()
        t[at] = what
        t[last, 0] = what
        got = prefill(spec, x, LENS, S0)
        compare(x, LENS, S0, clean, got)
        t[[at[0], last]] = keep


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_state_that_is_not_finite_stays_in_its_column(spec, shape):
    H, Hk, dk, dv, dtype = shape
    x = Rows(sum(LENS), H, Hk, dk, dv, dtype, seed=3)
    S0 = (torch.randn((3, 1, H, dk, dv), generator=torch.Generator().manual_seed(4)) * 0.5).cuda()
    clean = prefill(spec, x, LENS, S0)
    S0[1, 0, 1, 7, 18] = NAN
    compare(x, LENS, S0, clean, prefill(spec, x, LENS, S0))
