"""Attention of the verify rows over a shared prefix and the requests' own caches
(spec_prefix_attention) against its float64 definition.

Tolerances, as 2-norm of the error over 2-norm of the result, per request. fp32: a score errs by
about sqrt(D)/2 ulps of |q||k| scale, and a weight by as much in relative terms, which for the
inputs here (|q||k| scale <= 32) is 16 sqrt(D) 2^-24; four times that is allowed. bf16: weights and
outputs are rounded to 2^-9 of their values each: 2^-8 in all. lse: the scores' absolute error,
64 sqrt(D) 2^-24, in fp32 arithmetic for both types.
"""

import numpy as np
import pytest
import torch

from oracle import attention as o_at

pytestmark = pytest.mark.gpu

torch_dt = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def spec():
    from gpu_util import ensure_built
    ensure_built()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def tol(D, dtype):
    return 2.0 ** -8 if dtype == "bf16" else 64 * np.sqrt(D) * 2.0 ** -24


def npf(t):
    return t.detach().float().cpu().numpy()


class Case:
    def __init__(self, B, R, Hq, Hkv, D, P, cap, kv_len, dtype, prefix_len=None, n_rows=None, layers=1,
                 layer=0, seed=0, q_pad=0, prefix_pad=0, scale=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = torch_dt[dtype]

        def rnd(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(dt)

        self.B, self.R, self.Hq, self.Hkv, self.D, self.P, self.cap = B, R, Hq, Hkv, D, P, cap
        self.dtype, self.layers, self.layer = dtype, layers, layer
        self.scale = D ** -0.5 if scale is None else scale
        self.q = rnd(B * R, Hq * D + q_pad)
        self.out = torch.full((B * R, Hq * D + q_pad), float("nan"), dtype=dt, device="cuda")
        self.prefix = rnd(2, P, Hkv * D + prefix_pad) if P else None
        self.cache = rnd(B, layers, 2, cap, Hkv * D)
        self.kv_len = torch.tensor(kv_len, dtype=torch.int64).cuda()
        self.prefix_len = None if prefix_len is None else torch.tensor(prefix_len,
                                                                       dtype=torch.int64).cuda()
        self.n_rows = None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32).cuda()
        self.lse = torch.full((B * R, Hq), float("nan"), device="cuda")

    def structs(self, spec):
        e = 2 if self.dtype == "bf16" else 4
        st = spec.spec_state_desc()
        st.kv, st.kv_layers, st.kv_capacity = self.cache.data_ptr(), self.layers, self.cap
        st.kv_row_bytes = self.Hkv * self.D * e
        st.kv_request_stride = self.cache.stride(0) * e
        st.kv_len = self.kv_len.data_ptr()
        d = spec.spec_attn_desc()
        d.dtype = spec.SPEC_BF16 if self.dtype == "bf16" else spec.SPEC_F32
        d.q_heads, d.kv_heads, d.head_dim, d.scale = self.Hq, self.Hkv, self.D, self.scale
        d.q, d.q_stride = self.q.data_ptr(), self.q.stride(0)
        d.out, d.out_stride = self.out.data_ptr(), self.out.stride(0)
        if self.P:
            d.prefix_k, d.prefix_v = self.prefix[0].data_ptr(), self.prefix[1].data_ptr()
            d.prefix_capacity, d.prefix_stride = self.P, self.prefix.stride(1)
            d.prefix_len = None if self.prefix_len is None else self.prefix_len.data_ptr()
        d.lse = self.lse.data_ptr()
        return st, d

    def run(self, spec, ws=None, stream=None):
        st, d = self.structs(spec)
        n = spec.spec_prefix_attention_workspace_bytes(self.B, self.R, st, d)
        assert n > 0
        if ws is None:
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
        spec.spec_prefix_attention(self.B, self.R, st, self.layer, d, self.n_rows, ws, stream)
        torch.cuda.synchronize()
        assert int(ws[4:8].cpu().numpy().view(np.uint32)[0]) == 0
        return ws

    def check(self):
        sh = (self.cap, self.Hkv, self.D)
        W = self.Hq * self.D
        for b in range(self.B):
            pre = (None, None) if not self.P else tuple(
                npf(self.prefix[i][:, :self.Hkv * self.D]).reshape(self.P, self.Hkv, self.D)
                for i in range(2))
            own = npf(self.cache[b, self.layer])
            rows = slice(b * self.R, (b + 1) * self.R)
            with np.errstate(invalid="ignore"):
                want, lse = o_at.verify_rows(
                    npf(self.q[rows, :W]).reshape(self.R, self.Hq, self.D), *pre,
                    self.P if self.prefix_len is None else int(self.prefix_len[b]),
                    own[0].reshape(sh), own[1].reshape(sh), int(self.kv_len[b]),
                    self.R if self.n_rows is None else int(self.n_rows[b]), self.scale)
            got = npf(self.out[rows, :W]).reshape(want.shape).astype(np.float64)
            assert np.isfinite(got).all(), b
            err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
            assert err <= tol(self.D, self.dtype) * norm, (b, err / max(norm, 1e-30))
            empty = np.isneginf(lse)
            assert (got[empty] == 0).all()
            gl = npf(self.lse[rows]).astype(np.float64)
            assert np.array_equal(np.isneginf(gl), empty)
            assert np.abs(gl[~empty] - lse[~empty]).max(initial=0) <= 64 * np.sqrt(self.D) * 2.0 ** -24


CASES = [
    dict(B=1, R=1, Hq=1, Hkv=1, D=64, P=0, cap=1, kv_len=[0], dtype="bf16"),
    dict(B=1, R=2, Hq=4, Hkv=2, D=64, P=0, cap=512, kv_len=[256], dtype="f32"),
    dict(B=1, R=2, Hq=16, Hkv=4, D=256, P=0, cap=2100, kv_len=[2049], dtype="bf16"),
    dict(B=1, R=8, Hq=16, Hkv=4, D=256, P=700, cap=70, kv_len=[61], dtype="bf16"),
    dict(B=5, R=3, Hq=6, Hkv=2, D=128, P=333, cap=130, kv_len=[0, 1, 63, 64, 127], dtype="bf16",
         prefix_len=[333, 0, 1, 64, 200], n_rows=[3, 2, 0, 1, 3]),
    dict(B=5, R=3, Hq=6, Hkv=2, D=128, P=333, cap=130, kv_len=[0, 1, 63, 64, 127], dtype="f32",
         prefix_len=[333, 0, 1, 64, 200], n_rows=[3, 2, 0, 1, 3]),
    dict(B=3, R=8, Hq=24, Hkv=1, D=256, P=129, cap=300, kv_len=[7, 200, 130], dtype="bf16"),
    dict(B=2, R=8, Hq=64, Hkv=1, D=64, P=65, cap=90, kv_len=[7, 60], dtype="bf16"),
    dict(B=4, R=2, Hq=4, Hkv=4, D=40, P=70, cap=90, kv_len=[7, 60, 0, 64], dtype="bf16"),
    dict(B=2, R=4, Hq=2, Hkv=2, D=8, P=70, cap=90, kv_len=[7, 60], dtype="f32"),
    dict(B=33, R=8, Hq=8, Hkv=2, D=64, P=190, cap=40, kv_len=list(range(33)), dtype="bf16"),
    # no row of any request; lengths outside their ranges; the cache full before the rows end
    dict(B=2, R=2, Hq=4, Hkv=2, D=64, P=70, cap=20, kv_len=[3, 4], dtype="bf16", n_rows=[0, 0]),
    dict(B=3, R=4, Hq=4, Hkv=2, D=64, P=70, cap=20, kv_len=[18, -5, 20], dtype="bf16",
         prefix_len=[500, -1, 70], n_rows=[9, -1, 4]),
    dict(B=3, R=4, Hq=4, Hkv=2, D=64, P=70, cap=20, kv_len=[18, -5, 20], dtype="f32",
         prefix_len=[500, -1, 70], n_rows=[9, 4, 4]),
    # strides wider than the rows, an inner layer
    dict(B=2, R=3, Hq=4, Hkv=2, D=128, P=100, cap=77, kv_len=[30, 70], dtype="bf16", layers=3,
         layer=1, q_pad=5, prefix_pad=24),
    dict(B=2, R=3, Hq=4, Hkv=2, D=256, P=100, cap=77, kv_len=[30, 70], dtype="bf16", layers=2,
         layer=1, q_pad=8, prefix_pad=8),
    dict(B=2, R=3, Hq=4, Hkv=2, D=64, P=100, cap=77, kv_len=[30, 70], dtype="f32", layers=2,
         layer=1, q_pad=3, prefix_pad=8),
    # weights on few positions
    dict(B=2, R=4, Hq=8, Hkv=2, D=128, P=500, cap=99, kv_len=[30, 70], dtype="bf16", scale=0.25),
    dict(B=1, R=8, Hq=16, Hkv=4, D=256, P=0, cap=9000, kv_len=[8900], dtype="bf16"),
    dict(B=9, R=8, Hq=16, Hkv=4, D=256, P=1500, cap=200, kv_len=[11 * i for i in range(9)],
         dtype="bf16", prefix_len=[1500 - 150 * i for i in range(9)]),
    dict(B=9, R=8, Hq=16, Hkv=4, D=128, P=1500, cap=200, kv_len=[11 * i for i in range(9)],
         dtype="bf16", prefix_len=[1500 - 150 * i for i in range(9)]),    # more tiles of rows than a group of CTAs takes, the last group not full
    dict(B=17, R=8, Hq=16, Hkv=1, D=64, P=500, cap=40, kv_len=[2 * i for i in range(17)], dtype="bf16"),
    dict(B=300, R=8, Hq=8, Hkv=2, D=128, P=333, cap=24, kv_len=[i % 17 for i in range(300)],
         dtype="bf16", prefix_len=[333 - 37 * (i % 10) for i in range(300)],
         n_rows=[i % 9 for i in range(300)]),
    dict(B=1024, R=1, Hq=1, Hkv=1, D=256, P=70, cap=9, kv_len=[i % 9 for i in range(1024)],
         dtype="bf16"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_float64(spec, i):
    c = Case(**CASES[i], seed=i)
    c.run(spec)
    c.check()


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("bf16", 128), ("bf16", 64), ("bf16", 72),
                                     ("f32", 64)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_masked_positions_reach_nothing(spec, dtype, D, what):
    """What lies past a row's positions: past the cache's valid length, in later rows of the same
    cycle, past a request's part of the prefix."""
    c = Case(4, 4, 8, 2, D, 200, 150, [100, 3, 62, 126], dtype, prefix_len=[200, 10, 0, 65],
             n_rows=[4, 2, 4, 3], seed=3)
    c.run(spec)
    clean, clean_lse = c.out.clone(), c.lse.clone()
    for b, (n, rows) in enumerate(zip([100, 3, 62, 126], [4, 2, 4, 3])):
        c.cache[b, :, :, n + rows:] = what
    c.run(spec)
    assert torch.equal(c.out, clean) and torch.equal(c.lse, clean_lse)
    c.check()
    # the last row's key and value: no earlier row sees them
    for b, (n, rows) in enumerate(zip([100, 3, 62, 126], [4, 2, 4, 3])):
        c.cache[b, :, :, n + rows - 1] = what
    # prefix positions that only request 0 sees
    c.prefix[:, 65:] = what
    c.run(spec)
    W = c.Hq * c.D
    for b, rows in enumerate([4, 2, 4, 3]):
        for r in range(c.R):
            t = b * c.R + r
            if r == rows - 1 or (b == 0 and r < rows):
                continue
            assert torch.equal(c.out[t, :W], clean[t, :W]), (b, r)
            assert torch.equal(c.lse[t], clean_lse[t])
    if what != what:  # what a row does see, it shows
        assert torch.isnan(c.out[0, :W].float()).all() and torch.isnan(c.lse[0]).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("f32", 64)])
def test_a_non_finite_value_it_sees_shows_in_its_dims_only(spec, dtype, D):
    c = Case(1, 3, 4, 2, D, 0, 150, [100], dtype, seed=4)
    c.run(spec)
    clean = c.out.clone()
    c.cache[0, 0, 1, 101, 5] = float("inf")  # position of row 1, KV head 0, dim 5
    c.run(spec)
    out = c.out.float().view(3, 4, D)
    assert torch.equal(c.out[0], clean[0])
    assert torch.isinf(out[1:, :2, 5]).all()
    out[1:, :2, 5] = 0
    assert torch.isfinite(out).all()


def test_twice_the_same_bytes_and_on_another_stream(spec):
    c = Case(6, 8, 16, 4, 256, 900, 300, [250, 3, 77, 128, 0, 64], "bf16", seed=5)
    ws = c.run(spec)
    first, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    for stream in (None, side):
        c.out.zero_()
        torch.cuda.synchronize()
        c.run(spec, ws, stream)
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


def test_workspace_serves_other_shapes_in_turn(spec):
    big = Case(6, 8, 16, 4, 256, 900, 300, [250, 3, 77, 128, 0, 64], "bf16", seed=5)
    small = Case(1, 1, 2, 2, 256, 0, 30, [20], "bf16", seed=6)
    ws = big.run(spec)
    small.run(spec, ws)
    small.check()
    big.out.zero_()
    big.run(spec, ws)
    big.check()


def test_offsets_past_32_bits(spec):
    """Requests whose caches lie more than 2^32 bytes apart, positions past 2^31 elements."""
    B, R, H, D, cap = 2, 2, 4, 256, 600000
    cache = torch.zeros((B, 1, 2, cap, H * D), dtype=torch.bfloat16, device="cuda")  # 4.9 GB
    tail = 4096
    c = Case(B, R, H, H, D, 0, tail + 4, [0, 0], "bf16", seed=7)
    cache[:, :, :, cap - tail - 4:] = c.cache
    # zero keys weigh exp(0) each and zero values add nothing: the rows see all of the cache
    c.cache, c.cap = cache, cap
    c.kv_len = torch.tensor([cap - 4, cap - 10], dtype=torch.int64).cuda()
    c.run(spec)
    c.check()
