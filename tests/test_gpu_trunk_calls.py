"""What a call of the trunk's token mixers asks of its caller: workspaces no larger than it uses, no
pointers where there is nothing to read, and the stream that the caller has made current."""

import numpy as np
import pytest
import torch

from test_gpu_delta import Rows, State, npf, out_tol, rel, state_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spec():
    from gpu_util import ensure_built
    ensure_built()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def test_fp32_prompts_need_the_header_alone(spec):
    lens, H, d = [90, 0, 41], 2, 128
    x = Rows(sum(lens), H, H, d, d, "f32", seed=1)
    s = State(spec, len(lens), 1, H, d, d, 2)
    start = s.live.clone()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    assert spec.spec_delta_prefill_workspace_bytes(sum(lens), len(lens), s.st) > 256
    spec.spec_delta_prefill(len(lens), cu, sum(lens), s.st, 0, x.desc(spec), s.live,
                            torch.zeros(256, dtype=torch.uint8).cuda())
    outs, states, _ = x.oracle(npf(start[0, 0]), 0, 90)
    assert rel(x.result(0, 90), np.stack(outs)) <= out_tol(d, "f32")
    assert rel(npf(s.live[0, 0]), states[-1]) <= state_tol(d)
    # chunks are kept in the workspace: what the query says is needed, and refused without
    y = Rows(sum(lens), H, H, d, d, "bf16", seed=1)
    with pytest.raises(spec.SpecError, match="SPEC_ERR_INVALID"):
        spec.spec_delta_prefill(len(lens), cu, sum(lens), s.st, 0, y.desc(spec), s.live,
                                torch.zeros(256, dtype=torch.uint8).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("init", [False, True])
def test_no_rows_at_all_copies_the_states(spec, dtype, init):
    """Empty tensors have no address: of a call without rows only the states are touched."""
    B, H, d = 3, 2, 128
    x = Rows(0, H, H, d, d, dtype)
    s = State(spec, B, 2, H, d, d, 2)
    start, before = torch.randn_like(s.live), s.live.clone()
    desc = x.desc(spec)
    desc.q = desc.k = desc.v = desc.log_decay = desc.beta = desc.out = None
    cu = torch.zeros(B + 1, dtype=torch.int32).cuda()
    ws = torch.empty(spec.spec_delta_prefill_workspace_bytes(0, B, s.st), dtype=torch.uint8).cuda()
    spec.spec_delta_prefill(B, cu, 0, s.st, 1, desc, start if init else None, ws)
    want = start[:, 1] if init else torch.zeros_like(start[:, 1])
    assert torch.equal(s.live[:, 1], want) and torch.equal(s.live[:, 0], before[:, 0])
    with pytest.raises(spec.SpecError, match="SPEC_ERR_INVALID"):
        spec.spec_delta_prefill(B, cu, 1, s.st, 1, desc, None, ws)


@pytest.mark.parametrize("raw", [True, False], ids=["raw query", "stream object"])
def test_calls_run_on_the_current_stream(spec, raw, monkeypatch):
    """Whichever way torch is asked for it; a stream given is taken as it is."""
    monkeypatch.setattr(spec, "_raw_stream", None)
    if not raw:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    assert spec._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert spec._stream(None) == side.cuda_stream
        with torch.cuda.stream(other):
            assert spec._stream(None) == other.cuda_stream
        assert spec._stream(None) == side.cuda_stream
        assert spec._stream(other) == other.cuda_stream and spec._stream(7) == 7
    assert spec._stream(None) == torch.cuda.current_stream().cuda_stream
