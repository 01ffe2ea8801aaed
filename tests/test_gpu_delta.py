"""The gated delta rule (spec_delta_rows, spec_delta_prefill) against its float64 definition, and its
states against the commit that reads them.

Tolerances, as 2-norm of the error over 2-norm of the result. A row's dot products over dk terms
err by about sqrt(dk)/2 ulps of 2^-24, its other operations by a few; the map of a state error to
the next row has norm <= 1 (unit keys, 0 <= beta <= 1, decay <= 1), and errors and state are sums over
the same rows, so the ratio does not grow with them: 16 sqrt(dk) 2^-24 leaves a factor of about 16.
Outputs in bf16 are rounded once more, by at most 2^-9 of each value: 2^-8 with the rest.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import delta as o_de

pytestmark = pytest.mark.gpu

torch_dt = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def spec():
    from gpu_util import ensure_built
    ensure_built()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def state_tol(dk):
    return 16 * np.sqrt(dk) * 2.0 ** -24


def out_tol(dk, dtype):
    return 2.0 ** -8 if dtype == "bf16" else state_tol(dk)


def rel(x, y):
    x, y = np.asarray(x, dtype=np.float64), np.asarray(y, dtype=np.float64)
    assert x.shape == y.shape and np.isfinite(x).all()
    n = np.linalg.norm(y)
    return np.linalg.norm(x - y) / n if n else np.linalg.norm(x - y)


def npf(t):
    return t.detach().float().cpu().numpy()


class Rows:
    """Inputs as column ranges of one row per token (with `pad` unused columns on both sides)."""

    def __init__(self, rows, H, Hk, dk, dv, dtype, seed=0, pad=0, scale=0.25):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hk, self.dk, self.dv, self.dtype, self.scale = H, Hk, dk, dv, dtype, scale
        w = 2 * Hk * dk + H * dv
        n = max(rows, 1)
        x = torch.randn((n, w), generator=g)
        for at in (0, Hk * dk):
            y = x[:, at:at + Hk * dk].view(n, Hk, dk)
            y /= y.norm(dim=-1, keepdim=True)
        buf = torch.full((n, w + 2 * pad), float("nan")).to(torch_dt[dtype])
        buf[:, pad:pad + w] = x.to(torch_dt[dtype])
        self.buf = buf.cuda()
        m = self.buf[:rows, pad:pad + w]
        self.q, self.k, self.v = m[:, :Hk * dk], m[:, Hk * dk:2 * Hk * dk], m[:, 2 * Hk * dk:]
        self.g = (-3 * torch.rand((n, H), generator=g) ** 3)[:rows].contiguous().cuda()
        self.beta = torch.rand((n, H), generator=g)[:rows].contiguous().cuda()
        self.out = torch.full((n, H * dv + pad), float("nan"), dtype=torch_dt[dtype]).cuda()

    def desc(self, spec):
        d = spec.spec_delta_desc()
        d.dtype = spec.SPEC_BF16 if self.dtype == "bf16" else spec.SPEC_F32
        d.key_heads, d.scale = self.Hk, self.scale
        for f in "qkv":
            setattr(d, f, getattr(self, f).data_ptr())
            setattr(d, f + "_stride", self.buf.stride(0))
        d.log_decay, d.beta = self.g.data_ptr(), self.beta.data_ptr()
        d.out, d.out_stride = self.out.data_ptr(), self.out.stride(0)
        return d

    def oracle(self, S0, lo, hi):
        f = [npf(t[lo:hi]).reshape(hi - lo, *s) for t, s in
             ((self.q, (self.Hk, self.dk)), (self.k, (self.Hk, self.dk)), (self.v, (self.H, self.dv)))]
        return o_de.run(S0, *f, npf(self.g[lo:hi]), npf(self.beta[lo:hi]), self.scale)

    def result(self, lo, hi):
        return npf(self.out[lo:hi, :self.H * self.dv]).reshape(hi - lo, self.H, self.dv)


class State:
    def __init__(self, spec, B, layers, H, dk, dv, n_slots, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.live = (torch.randn((B, layers, H, dk, dv), generator=g) * 0.5).cuda()
        self.slots = torch.full((B, n_slots, layers, H, dk, dv), float("nan")).cuda()
        self.live_slot = torch.tensor([(2 * b + 1) % n_slots for b in range(B)],
                                      dtype=torch.int32).cuda()
        self.step_a = torch.full((B, n_slots - 1, layers, H), float("nan")).cuda()
        self.step_b = torch.full((B, n_slots - 1, layers, H, dk), float("nan")).cuda()
        self.step_c = torch.full((B, n_slots - 1, layers, H, dv), float("nan")).cuda()
        st = self.st = spec.spec_state_desc()
        st.rec_layers, st.rec_heads, st.rec_dk, st.rec_dv, st.n_slots = layers, H, dk, dv, n_slots
        st.rec_live, st.rec_slots = self.live.data_ptr(), self.slots.data_ptr()
        st.live_slot = self.live_slot.data_ptr()
        st.step_a, st.step_b, st.step_c = (t.data_ptr() for t in (self.step_a, self.step_b,
                                                                  self.step_c))

    def to_slots(self):
        for b, s in enumerate(self.live_slot.tolist()):
            self.slots[b, s] = self.live[b]


MODES = ["snapshot", "replay", "index"]


def mode_of(spec, name):
    return {"snapshot": spec.SPEC_COMMIT_SNAPSHOT, "replay": spec.SPEC_COMMIT_REPLAY,
            "index": spec.SPEC_COMMIT_INDEX}[name]


SHAPES = [  # B, R, layers, layer, H, Hk, dk, dv, dtype, pad
    (1, 1, 1, 0, 2, 2, 16, 16, "f32", 0),
    (1, 8, 3, 1, 16, 16, 128, 128, "bf16", 0),
    (3, 5, 2, 1, 8, 4, 128, 128, "bf16", 3),
    (2, 4, 1, 0, 6, 2, 20, 12, "f32", 1),
    (2, 3, 1, 0, 4, 1, 96, 64, "bf16", 8),
    (1, 2, 1, 0, 2, 1, 1, 4, "bf16", 0),
    (2, 2, 1, 0, 2, 1, 200, 36, "f32", 4),
    (33, 8, 1, 0, 4, 2, 64, 128, "bf16", 0),
    (1, 8, 1, 0, 1, 1, 256, 256, "bf16", 0),
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows(spec, shape, mode):
    B, R, layers, layer, H, Hk, dk, dv, dtype, pad = shape
    x = Rows(B * R, H, Hk, dk, dv, dtype, seed=B + R, pad=pad)
    n_slots = R + 2
    s = State(spec, B, layers, H, dk, dv, n_slots)
    if mode == "index":
        s.to_slots()
    n = [R if b % 3 == 0 else (b * 2) % (R + 1) for b in range(B)]
    before = s.slots.clone()
    spec.spec_delta_rows(B, R, s.st, layer, mode_of(spec, mode), x.desc(spec),
                         torch.tensor(n, dtype=torch.int32).cuda() if B > 1 else None)
    torch.cuda.synchronize()
    written = torch.zeros(s.slots.shape[:3], dtype=torch.bool)
    for b in range(B):
        outs, states, steps = x.oracle(npf(s.live[b, layer]), b * R, b * R + n[b])
        got = x.result(b * R, (b + 1) * R)
        if n[b]:
            assert rel(got[:n[b]], np.stack(outs)) <= out_tol(dk, dtype)
        assert (got[n[b]:] == 0).all()
        first = int(s.live_slot[b]) if mode == "index" else 0
        if mode != "index":
            assert torch.equal(s.slots[b, 0, layer], s.live[b, layer])
            written[b, 0, layer] = True
        for r in range(n[b]):
            if mode == "replay":
                a, k, u = steps[r]
                assert rel(npf(s.step_a[b, r, layer]), a) <= state_tol(1)
                assert np.array_equal(npf(s.step_b[b, r, layer]), k)
                assert rel(npf(s.step_c[b, r, layer]), u) <= state_tol(dk)
                continue
            at = (first + r + 1) % n_slots
            assert rel(npf(s.slots[b, at, layer]), states[r]) <= state_tol(dk)
            written[b, at, layer] = True
        if mode == "replay":
            for t in (s.step_a, s.step_b, s.step_c):  # steps of other rows and layers stay
                keep = torch.ones(t.shape[1:3], dtype=torch.bool)
                keep[:n[b], layer] = False
                assert torch.isnan(t[b][keep.cuda()]).all()
    same = (s.slots == before) | (torch.isnan(s.slots) & torch.isnan(before))
    assert same[~written.cuda()].all()


@pytest.mark.parametrize("shape", [(2, 8, 2, 16, 8, 128, 128, "bf16"), (3, 3, 1, 2, 2, 16, 16, "f32")])
def test_commit_of_every_mode_keeps_the_same_bytes(spec, shape):
    """For every accepted prefix: the state after snapshot commit, replay commit and index commit."""
    B, R, layers, H, Hk, dk, dv, dtype = shape
    for m in range(0, R + 1):
        kept = []
        for mode in MODES:
            s = State(spec, B, layers, H, dk, dv, R + 1)
            s.slots.zero_()
            if mode == "index":
                s.to_slots()
            for layer in range(layers):
                x = Rows(B * R, H, Hk, dk, dv, dtype, seed=layer)
                spec.spec_delta_rows(B, R, s.st, layer, mode_of(spec, mode), x.desc(spec))
            acc = np.zeros(B, dtype=spec.ACCEPT_OUT_DTYPE)
            acc["n_emit"] = m
            acc_d = torch.from_numpy(acc.view(np.uint8).copy()).cuda()
            k = torch.full((B,), R - 1, dtype=torch.int32).cuda()
            spec.spec_commit_rollback(B, s.st, acc_d, k, mode_of(spec, mode))
            if mode == "index":
                kept.append(torch.stack([s.slots[b, int(s.live_slot[b])] for b in range(B)]))
            else:
                kept.append(s.live.clone())
        assert torch.equal(kept[0].view(torch.int32), kept[1].view(torch.int32)), m
        assert torch.equal(kept[0].view(torch.int32), kept[2].view(torch.int32)), m


def test_rows_extremes(spec):
    """A decay of zero clears the state, beta 0 leaves it, and a live slot out of range runs nothing."""
    B, R, H, d = 3, 2, 2, 32
    x = Rows(B * R, H, H, d, d, "f32")
    x.g[0] = -float("inf")
    x.g[2:4] = 0
    x.beta[2:4] = 0
    s = State(spec, B, 1, H, d, d, R + 1)
    s.to_slots()
    s.live_slot[2] = R + 1
    spec.spec_delta_rows(B, R, s.st, 0, spec.SPEC_COMMIT_INDEX, x.desc(spec))
    _, states, _ = x.oracle(np.zeros((H, d, d)), 0, 2)
    assert rel(npf(s.slots[0, (1 + 2) % 3, 0]), states[1]) <= state_tol(d)
    assert torch.equal(s.slots[1, (0 + 2) % 3, 0], s.live[1, 0])
    assert (x.result(4, 6) == 0).all()


def run_prefill(spec, x, lens, layers, layer, init, stream=None, ws=None, gap=0):
    B, rows = len(lens), sum(lens) + gap
    s = State(spec, B, layers, x.H, x.dk, x.dv, 2, seed=5)
    start = s.live.clone()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    n = spec.spec_delta_prefill_workspace_bytes(rows, B, s.st)
    assert n > 0
    ws = torch.full((n,), 255, dtype=torch.uint8).cuda()  # no initial contents are needed
    spec.spec_delta_prefill(B, cu, rows, s.st, layer, x.desc(spec),
                            {"zero": None, "live": s.live, "other": start}[init], ws, stream)
    torch.cuda.synchronize()
    assert int(ws[4:8].cpu().numpy().view(np.uint32)[0]) == 0
    return s, start


LENS = [[1], [63], [64], [65], [128], [0, 1, 77, 0, 200], [5, 130, 64, 63, 1, 0], [515], [2, 2, 2],
        [1, 90, 4], [1, 90, 5]]  # either side of 32 rows a request on average


@pytest.mark.parametrize("init", ["zero", "live", "other"])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", [(4, 2, 128, 128, "bf16", 0), (3, 3, 128, 64, "bf16", 8),
                                   (2, 1, 128, 20, "bf16", 3), (2, 2, 64, 128, "bf16", 0),
                                   (2, 1, 40, 12, "f32", 1), (4, 2, 128, 128, "f32", 0)], ids=str)
def test_prefill(spec, shape, lens, init):
    H, Hk, dk, dv, dtype, pad = shape
    x = Rows(sum(lens), H, Hk, dk, dv, dtype, seed=sum(lens), pad=pad)
    layers, layer = (2, 1) if len(lens) > 1 else (1, 0)
    s, start = run_prefill(spec, x, lens, layers, layer, init)
    lo = 0
    for b, n in enumerate(lens):
        S0 = npf(start[b, layer]) if init != "zero" else np.zeros((H, dk, dv))
        outs, states, _ = x.oracle(S0, lo, lo + n)
        if n:
            assert rel(x.result(lo, lo + n), np.stack(outs)) <= out_tol(dk, dtype)
            assert rel(npf(s.live[b, layer]), states[-1]) <= state_tol(dk)
        else:
            assert np.array_equal(npf(s.live[b, layer]), S0.astype(np.float32))
        if layers > 1:
            assert torch.equal(s.live[b, 0], start[b, 0])
        lo += n


@pytest.mark.parametrize("kind", ["none", "clear", "strong", "repeat", "long"])
def test_prefill_hard_inputs(spec, kind):
    """No decay at all, decays of zero inside a chunk, decays whose products underflow, the same key
    again and again at beta 1 (the triangular system at its worst), and a long prompt."""
    n = 4097 if kind == "long" else 300
    x = Rows(n, 2, 1, 128, 128, "bf16", seed=9)
    if kind == "none":
        x.g.zero_()
    elif kind == "clear":
        x.g[[3, 64, 100, 101, 299]] = -float("inf")
    elif kind == "strong":
        x.g.fill_(-30.0)
        x.g[::3] = -0.01
    elif kind == "repeat":
        x.k[:] = x.k[0]
        x.beta.fill_(1.0)
        x.g.zero_()
    s, start = run_prefill(spec, x, [n], 1, 0, "live")
    outs, states, _ = x.oracle(npf(start[0, 0]), 0, n)
    assert rel(x.result(0, n), np.stack(outs)) <= out_tol(128, "bf16")
    assert rel(npf(s.live[0, 0]), states[-1]) <= state_tol(128)


def test_prefill_rows_past_the_prompts_are_left_alone(spec):
    x = Rows(100 + 28, 2, 1, 128, 128, "bf16")
    run_prefill(spec, x, [90, 10], 1, 0, "zero", gap=28)
    assert torch.isnan(x.out[100:]).all() and not torch.isnan(x.out[:100]).any()


def test_prefill_of_many_requests(spec):
    """More requests than are put in order of length."""
    lens = [(37 * i) % 90 for i in range(300)]
    x = Rows(sum(lens), 1, 1, 128, 16, "bf16", seed=4)
    s, start = run_prefill(spec, x, lens, 1, 0, "other")
    lo = np.concatenate([[0], np.cumsum(lens)])
    for b in (0, 1, 2, 90, 157, 255, 256, 299):
        S0 = npf(start[b, 0])
        outs, states, _ = x.oracle(S0, int(lo[b]), int(lo[b + 1]))
        want = states[-1] if lens[b] else S0
        assert rel(npf(s.live[b, 0]), want) <= state_tol(128), b
        if lens[b]:
            assert rel(x.result(int(lo[b]), int(lo[b + 1])), np.stack(outs)) <= out_tol(128, "bf16"), b


def test_prefill_twice_is_bitwise_the_same_and_on_another_stream(spec):
    lens = [200, 0, 333]
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side):
        x = Rows(sum(lens), 4, 2, 128, 128, "bf16", seed=3)
        torch.cuda.synchronize()
        s, _ = run_prefill(spec, x, lens, 1, 0, "zero", stream)
        got.append((x.out.clone(), s.live.clone()))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_descriptor_is_a_host_struct(spec):
    assert ctypes.sizeof(spec.spec_delta_desc) == 96
