"""The paged KV cache (spec_paged_append, spec_paged_attention, spec_paged_commit) against its float64
definition.

Tolerances. Attention, as 2-norm of the error over 2-norm of the result, per request: as for
spec_prefix_attention, whose arithmetic it is (fp32: a score errs by sqrt(D)/2 ulps of |q||k| scale <= 32
and a weight by as much in relative terms: 16 sqrt(D) 2^-24, four times that allowed; bf16: weights and
outputs rounded to 2^-9 each in the mean: 2^-8 in all; lse: the scores' absolute error, 64 sqrt(D) 2^-24).
Append, per element: half a step of the output type (eps / 2 of its value), and fp32's own errors, in units
of 2^-24 of the head's largest value: the sum of squares 13 (eight in a lane, five joins) halved by the
root, the root and the products 4, cos and sin 3 each (2 ulps and the angle's rounding to 2^-24 of half a
turn, pi ulps), the rotation's products and sum 3: 24 together, 32 allowed.
"""

import numpy as np
import pytest
import torch

from oracle import paged as o_pg

pytestmark = pytest.mark.gpu

torch_dt = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


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


class Cache:
    """Pages of `layers` layers, each request's in any order in the pool; layout "pools" ([layers][pages])
    or "pages" ([pages][layers], keys and values side by side). max_pages: entries of a table row, all of
    them pages of the request's own."""

    def __init__(self, B, max_pages, page, H, D, dtype, kv_len, layers=1, layout="pools", spare=3, table_pad=1,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.page, self.H, self.D, self.dtype, self.layers = B, page, H, D, dtype, layers
        n = self.n_pages = B * max_pages + spare
        dt = torch_dt[dtype]
        if layout == "pools":
            self.store = torch.randn((2, layers, n, page, H * D), generator=g, device="cuda").to(dt)
            self.k, self.v = self.store[0], self.store[1]
        else:
            self.store = torch.randn((n, layers, 2, page, H * D), generator=g, device="cuda").to(dt)
            self.k, self.v = (self.store[:, :, i].transpose(0, 1) for i in range(2))
        order = torch.randperm(n, generator=g, device="cuda")[:B * max_pages].to(torch.int32)
        self.wide = torch.full((B, max_pages + table_pad), -7, dtype=torch.int32, device="cuda")
        self.wide[:, :max_pages] = order.view(B, max_pages)
        self.table = self.wide[:, :max_pages]
        self.max_pages = max_pages
        self.kv_len = torch.tensor(kv_len, dtype=torch.int64).cuda()

    def desc(self, spec):
        c = spec.spec_paged_cache()
        c.dtype = spec.SPEC_BF16 if self.dtype == "bf16" else spec.SPEC_F32
        c.layers, c.kv_heads, c.head_dim = self.layers, self.H, self.D
        c.page_size, c.n_pages, c.max_pages = self.page, self.n_pages, self.max_pages
        c.k_pages, c.v_pages = self.k.data_ptr(), self.v.data_ptr()
        e = self.store.element_size()
        c.layer_stride, c.page_stride = self.k.stride(0) * e, self.k.stride(1) * e
        c.page_table, c.table_stride = self.wide.data_ptr(), self.wide.stride(0)
        c.kv_len = self.kv_len.data_ptr()
        return c

    def np(self, layer):
        return tuple(npf(x[layer]).astype(np.float64).reshape(self.n_pages, self.page, self.H, self.D)
                     for x in (self.k, self.v))


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


# --------------------------------------------------------------------------------- append
def run_append(spec, c, cu, rows, Hq, rot, pairs, norm, layer=0, n_rows=None, pos=None, scale=1.0, pad=0,
               in_place=False, base=1e4, seed=0, keys=True, kv_pos=None):
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    dt, H, D = torch_dt[c.dtype], c.H, c.D
    W = (Hq + 2 * H) * D + pad
    mixed = torch.randn((max(rows, 1), W), generator=g, device="cuda").to(dt)[:rows]
    q, k, v = mixed[:, :Hq * D], mixed[:, Hq * D:(Hq + H) * D], mixed[:, (Hq + H) * D:(Hq + 2 * H) * D]
    q0, k0, v0 = (npf(x).astype(np.float64).reshape(rows, x.shape[1] // D, D) for x in (q, k, v))
    q_out = q if in_place else torch.full((rows, Hq * D + pad), 7.0, dtype=dt, device="cuda")
    before = npf(q_out)[:, :Hq * D].reshape(rows, Hq, D)
    f = base ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) / max(rot // 2, 1))
    nq, nk = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")) if norm else None for _ in range(2))
    d = spec.spec_append_desc()
    d.q_heads, d.norm_eps, d.rot_dim, d.rot_interleaved, d.rot_scale = Hq, EPS, rot, pairs == "side", scale
    if Hq:
        d.q, d.q_stride, d.q_out, d.q_out_stride = q.data_ptr(), W, q_out.data_ptr(), q_out.stride(0)
    if keys:
        d.k, d.v, d.k_stride, d.v_stride = k.data_ptr(), v.data_ptr(), W, W
    if norm:
        d.q_norm, d.k_norm = nq.data_ptr(), nk.data_ptr()
    d.inv_freq = f.data_ptr()
    if pos is not None:
        p64 = torch.tensor(pos, dtype=torch.int64).cuda()
        d.pos = p64.data_ptr()
    kp, vp = c.np(layer)
    status = torch.full((c.B,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_append(c.B, i32(cu), rows, c.desc(spec), layer, d, i32(n_rows), status)
    torch.cuda.synchronize()
    table = c.table.cpu().numpy()
    args = (q0, k0, v0) if keys else (q0, k0[:, :0], v0[:, :0])
    want, st = o_pg.append(*args, kp if keys else kp[:, :, :0], vp if keys else vp[:, :, :0], table,
                           c.kv_len.tolist(), cu, n_rows, pos, nq if nq is None else npf(nq),
                           nk if nk is None else npf(nk), EPS, rot, pairs == "side", npf(f), scale)
    half = torch.finfo(dt).eps / 2

    def close(got, ref):
        top = np.abs(ref).max(axis=-1, keepdims=True, initial=0)
        assert (np.abs(got - ref) <= half * np.abs(ref) + 32 * 2.0 ** -24 * top).all(), np.abs(got - ref).max()

    got = npf(q_out)[:, :Hq * D].reshape(rows, Hq, D)
    ran = ~np.isnan(want[:, 0, 0]) if Hq else np.zeros(rows, dtype=bool)
    close(got[ran].astype(np.float64), want[ran])
    assert np.array_equal(got[~ran], before[~ran])
    if keys:
        assert status.tolist() == st.tolist()
        close(c.np(layer)[0], kp)
        assert np.array_equal(c.np(layer)[1], vp)
    else:
        assert status.tolist() == [0] * c.B


APPEND = [
    dict(lens=[1], B=1, D=64, H=1, Hq=1, dtype="bf16", rot=64, pairs="half", norm=True, kv_len=[0]),
    dict(lens=[2], B=1, D=64, H=2, Hq=4, dtype="f32", rot=64, pairs="half", norm=False, kv_len=[13]),
    dict(lens=[3, 0, 1, 40], B=4, D=128, H=2, Hq=6, dtype="bf16", rot=128, pairs="side", norm=True,
         kv_len=[5, 3, 0, 8]),
    dict(lens=[8] * 5, B=5, D=256, H=4, Hq=16, dtype="bf16", rot=64, pairs="half", norm=True,
         kv_len=[0, 1, 7, 8, 30], n_rows=[8, 0, 3, 1, 9], scale=1.2),
    dict(lens=[9, 5], B=2, D=256, H=2, Hq=2, dtype="f32", rot=256, pairs="half", norm=True, kv_len=[3, 40]),
    # rotations that end inside a lane's eight dims; heads that do not fill a warp's lanes
    dict(lens=[7, 6], B=2, D=40, H=3, Hq=3, dtype="bf16", rot=20, pairs="half", norm=True, kv_len=[3, 4]),
    dict(lens=[7, 6], B=2, D=96, H=1, Hq=5, dtype="f32", rot=54, pairs="half", norm=True, kv_len=[3, 4]),
    dict(lens=[7, 6], B=2, D=96, H=1, Hq=5, dtype="bf16", rot=54, pairs="side", norm=False, kv_len=[3, 4]),
    dict(lens=[4], B=1, D=8, H=2, Hq=4, dtype="bf16", rot=2, pairs="half", norm=True, kv_len=[2]),
    dict(lens=[4], B=1, D=8, H=1, Hq=1, dtype="f32", rot=8, pairs="side", norm=True, kv_len=[2]),
    dict(lens=[5], B=1, D=256, H=1, Hq=2, dtype="bf16", rot=250, pairs="half", norm=False, kv_len=[2]),
    dict(lens=[5], B=1, D=128, H=1, Hq=2, dtype="bf16", rot=0, pairs="half", norm=True, kv_len=[2]),
    dict(lens=[5], B=1, D=128, H=1, Hq=2, dtype="f32", rot=0, pairs="half", norm=False, kv_len=[2]),
    # strides that are no whole vectors, an inner layer, in place, a position of its own
    dict(lens=[5, 6], B=2, D=64, H=2, Hq=4, dtype="bf16", rot=32, pairs="half", norm=True, kv_len=[2, 9], pad=3,
         layers=3, layer=1),
    dict(lens=[5, 6], B=2, D=64, H=2, Hq=4, dtype="f32", rot=32, pairs="side", norm=True, kv_len=[2, 9], pad=1,
         layers=2, layer=1, layout="pages", in_place=True),
    dict(lens=[5, 6], B=2, D=128, H=2, Hq=4, dtype="bf16", rot=128, pairs="half", norm=True, kv_len=[2, 9],
         in_place=True, pos=[60000, 1]),
    # no queries; many requests
    dict(lens=[5, 6], B=2, D=128, H=2, Hq=0, dtype="bf16", rot=128, pairs="half", norm=True, kv_len=[2, 9]),
    dict(lens=[i % 5 for i in range(300)], B=300, D=64, H=1, Hq=2, dtype="bf16", rot=64, pairs="half", norm=True,
         kv_len=[i % 11 for i in range(300)]),
    # tables that end before the rows, lengths below zero
    dict(lens=[8, 8, 8], B=3, D=64, H=2, Hq=2, dtype="bf16", rot=64, pairs="half", norm=False,
         kv_len=[60, -4, 70]),
]


@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append(spec, i, page):
    a = dict(APPEND[i])
    lens, B, D, H, dtype = (a.pop(x) for x in ("lens", "B", "D", "H", "dtype"))
    c = Cache(B, 4 if page == 16 else 9, page, H, D, dtype, a.pop("kv_len"), layers=a.pop("layers", 1),
              layout=a.pop("layout", "pools"), seed=i)
    run_append(spec, c, cu_of(lens), sum(lens), seed=i, **a)


def test_append_rows_that_nobody_owns_and_pages_that_are_not_there(spec):
    c = Cache(3, 4, 8, 2, 64, "bf16", [4, 6, 0], seed=1)
    c.table[0, 1] = -1
    c.table[1, 1] = c.n_pages
    c.table[2, 3] = -2  # not needed
    run_append(spec, c, [2, 9, 14, 20], 25, 4, 64, "half", True)


def test_append_without_keys_writes_no_page(spec):
    c = Cache(2, 3, 8, 2, 64, "bf16", [4, 6], seed=2)
    before = c.store.clone()
    run_append(spec, c, [0, 3, 5], 5, 4, 64, "half", True, keys=False)
    assert torch.equal(c.store, before)


def test_append_no_rows(spec):
    c = Cache(2, 3, 8, 2, 64, "bf16", [4, 6], seed=2)
    before = c.store.clone()
    run_append(spec, c, [0, 0, 0], 0, 4, 64, "half", True)
    assert torch.equal(c.store, before)


@pytest.mark.parametrize("at", [0, 1, 65535, 10 ** 6 + 1, 2 ** 31 - 9, 2 ** 40 + 3])
def test_angles_of_far_positions(spec, at):
    """Exact products, for which 64-bit floats are too short past 2^29."""
    mpmath = pytest.importorskip("mpmath")
    D, half = 64, 32
    c = Cache(1, 1, 8, 1, D, "f32", [0])
    f = torch.tensor([10.0 ** (-4 * i / half) * (1 if i % 3 else -1) for i in range(half)]).cuda()
    f[1], f[2] = 6.5, 0.0
    x = torch.ones((1, D), device="cuda")
    out = torch.empty_like(x)
    d = spec.spec_append_desc()
    d.q_heads, d.rot_dim, d.rot_scale = 1, D, 1.0
    d.q, d.q_stride, d.q_out, d.q_out_stride, d.inv_freq = x.data_ptr(), D, out.data_ptr(), D, f.data_ptr()
    pos = torch.tensor([at], dtype=torch.int64).cuda()
    d.pos = pos.data_ptr()
    spec.spec_paged_append(1, i32([0, 1]), 1, c.desc(spec), 0, d)
    with mpmath.workdps(60):
        for i, v in enumerate(f.double().tolist()):
            t = mpmath.mpf(v) * at
            # the angle's rounding pi 2^-24, cos and sin 2 ulps each, their sum's rounding: 9 ulps of 1, times 2
            assert abs(float(out[0, i]) - float(mpmath.cos(t) - mpmath.sin(t))) <= 18 * 2.0 ** -24, (i, v)
            assert abs(float(out[0, half + i]) - float(mpmath.cos(t) + mpmath.sin(t))) <= 18 * 2.0 ** -24


# ------------------------------------------------------------------------------- attention
class Attn:
    def __init__(self, c, lens, Hq, n_rows=None, layer=0, pad=0, extra=0, scale=None, seed=0, first=0):
        g = torch.Generator(device="cuda").manual_seed(200 + seed)
        dt = torch_dt[c.dtype]
        self.c, self.Hq, self.layer, self.n_rows = c, Hq, layer, n_rows
        self.cu = [first + x for x in cu_of(lens)]
        self.rows = self.cu[-1] + extra
        self.scale = c.D ** -0.5 if scale is None else scale
        self.q = torch.randn((self.rows, Hq * c.D + pad), generator=g, device="cuda").to(dt)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((self.rows, Hq), 7.0, device="cuda")

    def desc(self, spec):
        d = spec.spec_paged_attn_desc()
        d.q_heads, d.scale = self.Hq, self.scale
        d.q, d.q_stride, d.out, d.out_stride = (self.q.data_ptr(), self.q.stride(0), self.out.data_ptr(),
                                                self.out.stride(0))
        d.lse = self.lse.data_ptr()
        return d

    def run(self, spec, ws=None, stream=None):
        c, d = self.c.desc(spec), self.desc(spec)
        n = spec.spec_paged_attention_workspace_bytes(self.c.B, self.rows, c, d)
        assert n > 0
        if ws is None:
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        cu, nr = i32(self.cu), i32(self.n_rows)
        torch.cuda.synchronize()
        spec.spec_paged_attention(self.c.B, cu, self.rows, c, self.layer, d, nr, ws, stream)
        torch.cuda.synchronize()
        assert int(ws[4:8].cpu().numpy().view(np.uint32)[0]) == 0
        return ws

    def check(self, finite=True):
        c, W = self.c, self.Hq * self.c.D
        k, v = c.np(self.layer)
        q = npf(self.q)[:, :W].reshape(self.rows, self.Hq, c.D)
        with np.errstate(invalid="ignore"):
            want, lse = o_pg.attend(q, k, v, c.table.cpu().numpy(), c.kv_len.tolist(), self.cu, self.n_rows,
                                    self.scale)
        got = npf(self.out)[:, :W].reshape(want.shape).astype(np.float64)
        gl = npf(self.lse).astype(np.float64)
        for b in range(c.B):
            s = slice(self.cu[b], self.cu[b + 1])
            assert np.isfinite(got[s]).all(), b
            err, norm = np.linalg.norm(got[s] - want[s]), np.linalg.norm(want[s])
            assert err <= tol(c.D, c.dtype) * norm, (b, err / max(norm, 1e-30))
            empty = np.isneginf(lse[s])
            assert (got[s][empty] == 0).all() and np.array_equal(np.isneginf(gl[s]), empty)
            assert np.abs(gl[s][~empty] - lse[s][~empty]).max(initial=0) <= 64 * np.sqrt(c.D) * 2.0 ** -24
        nobody = np.isnan(lse[:, 0])
        assert (got[nobody] == 7).all() and (gl[nobody] == 7).all()
        assert (npf(self.out)[:, W:] == 7).all()


ATTN = [
    dict(lens=[1], D=64, H=1, Hq=1, dtype="bf16", page=16, kv_len=[0]),
    dict(lens=[2], D=64, H=2, Hq=4, dtype="f32", page=16, kv_len=[256]),
    dict(lens=[2], D=256, H=4, Hq=16, dtype="bf16", page=64, kv_len=[2049]),
    dict(lens=[8] * 5, D=128, H=2, Hq=6, dtype="bf16", page=8, kv_len=[0, 1, 63, 64, 127],
         n_rows=[8, 2, 0, 1, 9]),
    dict(lens=[8] * 5, D=128, H=2, Hq=6, dtype="f32", page=8, kv_len=[0, 1, 63, 64, 127],
         n_rows=[8, 2, 0, 1, 9]),
    # prompts from their start, chunks, single tokens, none
    dict(lens=[0, 1, 77, 130, 300], D=128, H=2, Hq=4, dtype="bf16", page=16, kv_len=[5, 0, 0, 40, 0]),
    dict(lens=[0, 1, 77, 130, 300], D=256, H=2, Hq=8, dtype="bf16", page=32, kv_len=[5, 0, 0, 40, 0]),
    dict(lens=[0, 1, 77, 130, 300], D=64, H=2, Hq=4, dtype="bf16", page=64, kv_len=[5, 0, 0, 40, 0]),
    dict(lens=[0, 1, 77, 130], D=64, H=2, Hq=4, dtype="f32", page=16, kv_len=[5, 0, 0, 40]),
    dict(lens=[500, 3], D=64, H=1, Hq=8, dtype="bf16", page=128, kv_len=[200, 700]),
    dict(lens=[129], D=256, H=1, Hq=1, dtype="bf16", page=256, kv_len=[1000]),
    dict(lens=[40], D=128, H=1, Hq=64, dtype="bf16", page=32, kv_len=[64]),
    # head and page sizes of the CUDA cores
    dict(lens=[20, 3], D=72, H=2, Hq=6, dtype="bf16", page=16, kv_len=[30, 64]),
    dict(lens=[20, 3], D=8, H=2, Hq=2, dtype="f32", page=1, kv_len=[30, 64]),
    dict(lens=[20, 3], D=128, H=2, Hq=4, dtype="bf16", page=24, kv_len=[30, 64]),
    dict(lens=[20, 3], D=256, H=1, Hq=4, dtype="bf16", page=7, kv_len=[30, 64]),
    # rows nobody owns before and behind, strides, an inner layer, both layouts
    dict(lens=[5, 9], D=128, H=2, Hq=4, dtype="bf16", page=16, kv_len=[30, 70], layers=3, layer=1, pad=5,
         first=3, extra=4),
    dict(lens=[5, 9], D=256, H=2, Hq=4, dtype="bf16", page=64, kv_len=[30, 70], layers=2, layer=1, pad=8,
         layout="pages", extra=1),
    dict(lens=[5, 9], D=64, H=2, Hq=4, dtype="f32", page=16, kv_len=[30, 70], layers=2, layer=1, pad=3,
         layout="pages", first=1, extra=4),
    # tables that end before the rows, lengths out of range, no row at all
    dict(lens=[4, 4, 4], D=64, H=2, Hq=4, dtype="bf16", page=16, kv_len=[62, -5, 900], max_pages=4),
    dict(lens=[4, 4, 4], D=64, H=2, Hq=4, dtype="f32", page=16, kv_len=[62, -5, 900], max_pages=4),
    dict(lens=[4, 4], D=64, H=2, Hq=4, dtype="bf16", page=16, kv_len=[3, 4], n_rows=[0, -1]),
    # weights on few positions; a scale below zero
    dict(lens=[4, 30], D=128, H=2, Hq=8, dtype="bf16", page=32, kv_len=[300, 70], scale=0.25),
    dict(lens=[4, 30], D=64, H=2, Hq=8, dtype="bf16", page=32, kv_len=[300, 70], scale=-0.1),
    dict(lens=[i % 4 for i in range(300)], D=128, H=2, Hq=4, dtype="bf16", page=16,
         kv_len=[i % 37 for i in range(300)]),
    dict(lens=[1] * 512, D=256, H=1, Hq=1, dtype="bf16", page=64, kv_len=[i % 90 for i in range(512)]),
    dict(lens=[1, 2], D=256, H=4, Hq=16, dtype="bf16", page=64, kv_len=[9000, 5000]),
    # as many tiles over as many positions as have groups of CTAs walk them, some left over
    dict(lens=[300, 3, 0, 270], D=64, H=1, Hq=4, dtype="bf16", page=64, kv_len=[8100, 50, 9000, 9001]),
    dict(lens=[3, 620, 5], D=256, H=1, Hq=2, dtype="bf16", page=16, kv_len=[700, 7900, 9000]),
    dict(lens=[130], D=128, H=2, Hq=16, dtype="bf16", page=128, kv_len=[8192]),
]


def attn_case(i, **more):
    a = dict(ATTN[i], **more)
    lens, kv_len, page = a["lens"], a["kv_len"], a["page"]
    need = max(-(-(max(p, 0) + n) // page) for p, n in zip(kv_len, lens))
    c = Cache(len(lens), a.get("max_pages", max(need, 1)), page, a["H"], a["D"], a["dtype"], kv_len,
              layers=a.get("layers", 1), layout=a.get("layout", "pools"), seed=i)
    return Attn(c, lens, a["Hq"], seed=i,
                **{k: a[k] for k in ("n_rows", "layer", "pad", "extra", "scale", "first") if k in a})


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention_against_float64(spec, i):
    a = attn_case(i)
    a.run(spec)
    a.check()


KINDS = [("bf16", 256, 64), ("bf16", 256, 16), ("bf16", 128, 16), ("bf16", 128, 128), ("bf16", 64, 8),
         ("bf16", 72, 16), ("f32", 64, 16)]


@pytest.mark.parametrize("dtype,D,page", KINDS)
@pytest.mark.parametrize("entry", [-1, 1 << 30, -2 ** 31])
def test_pages_that_are_not_there(spec, dtype, D, page, entry):
    """First, inner and last pages, and all of a request's."""
    c = Cache(4, -(-150 // page), page, 2, D, dtype, [100, 3, 62, 126], seed=3)
    for b, j in ((0, 0), (0, 40 // page), (2, 64 // page)):
        c.table[b, j] = entry
    c.table[3, 126 // page] = entry  # of the new rows, whole or in part
    a = Attn(c, [5, 4, 3, 9], 6, seed=3)
    a.run(spec)
    a.check()
    c.table[1] = entry
    a.run(spec)
    a.check()
    assert (a.out[5:9] == 0).all() and torch.isneginf(a.lse[5:9]).all()


@pytest.mark.parametrize("dtype,D,page", KINDS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_masked_positions_reach_nothing(spec, dtype, D, page, what):
    """What lies past a row's positions: past the valid length, in later rows, on pages of others and of
    nobody; and what a row does see, it shows."""
    lens, kv_len, runs = [6, 4, 40, 3], [100, 3, 62, 126], [6, 2, 40, 3]
    c = Cache(4, -(-150 // page), page, 2, D, dtype, kv_len, seed=4)
    a = Attn(c, lens, 4, n_rows=runs, seed=4)
    a.run(spec)
    a.check()
    clean, clean_lse = a.out.clone(), a.lse.clone()
    used = torch.zeros((c.n_pages, page), dtype=torch.bool, device="cuda")
    for b, (P, n) in enumerate(zip(kv_len, runs)):
        for p in range(P + n):
            used[c.table[b, p // page].long(), p % page] = True
    for x in (c.k, c.v):
        x[0][~used] = what
    a.run(spec)
    assert torch.equal(a.out, clean) and torch.equal(a.lse, clean_lse)
    for b, (P, n) in enumerate(zip(kv_len, runs)):  # the last row's key and value: no earlier row sees them
        at = P + n - 1
        for x in (c.k, c.v):
            x[0, c.table[b, at // page].long(), at % page] = what
    a.run(spec)
    for b, n in enumerate(runs):
        for r in range(lens[b]):
            t = a.cu[b] + r
            if r != n - 1:
                assert torch.equal(a.out[t], clean[t]) and torch.equal(a.lse[t], clean_lse[t]), (b, r)
            elif what != what:
                assert torch.isnan(a.out[t].float()).all() and torch.isnan(a.lse[t]).all(), (b, r)


@pytest.mark.parametrize("dtype,D,page", KINDS)
def test_a_non_finite_value_shows_in_its_dims_only(spec, dtype, D, page):
    c = Cache(1, -(-300 // page), page, 2, D, dtype, [100], seed=5)
    a = Attn(c, [70], 4, seed=5)
    a.run(spec)
    clean = a.out.clone()
    at = 130
    c.v[0, c.table[0, at // page].long(), at % page, 5] = float("inf")  # position of row 30, KV head 0, dim 5
    a.run(spec)
    out = a.out.float().view(70, 4, D).clone()
    assert torch.equal(a.out[:30], clean[:30])
    assert torch.isinf(out[30:, :2, 5]).all()
    out[30:, :2, 5] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_twice_the_same_bytes_on_another_stream_and_in_a_graph(spec, dtype):
    c = Cache(6, 20, 16, 4, 128, dtype, [250, 3, 77, 128, 0, 64], seed=6)
    a = Attn(c, [8, 1, 50, 0, 300, 7] if dtype == "bf16" else [8, 1, 50, 0, 30, 7], 8, seed=6)
    ws = a.run(spec)
    a.check()
    first, lse = a.out.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    for stream in (None, side):
        a.out.zero_()
        a.run(spec, ws, stream)
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
    cu, cd, ad = i32(a.cu), c.desc(spec), a.desc(spec)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spec.spec_paged_attention(c.B, cu, a.rows, cd, 0, ad, None, ws)
    for _ in range(2):
        a.out.zero_()
        a.lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
    # the lengths are the device's: a replay sees them as they are then
    c.kv_len.sub_(c.kv_len.clamp(max=2))
    graph.replay()
    torch.cuda.synchronize()
    a.check()


def test_a_row_may_read_pages_of_another_request(spec):
    """A common prompt's pages stand in several tables."""
    c = Cache(3, 8, 16, 2, 128, "bf16", [100, 90, 80], seed=7)
    c.table[1, :5] = c.table[0, :5]
    c.table[2, :5] = c.table[0, :5]
    a = Attn(c, [3, 3, 3], 4, seed=7)
    a.run(spec)
    a.check()


def test_row_counts_that_are_not_as_documented_touch_nothing_else(spec):
    """Offsets out of range and out of order: the call ends, and rows outside all of them stay."""
    c = Cache(3, 8, 16, 2, 128, "bf16", [100, 90, 80], seed=8)
    a = Attn(c, [4, 4, 4], 4, extra=4, seed=8)
    for cu in ([0, 40, 2, 10 ** 9], [-5, 3, 3, -1], [0, 16, 0, 16]):
        a.cu = cu
        a.run(spec)
        assert torch.isfinite(a.out.float()).all()


def test_workspace_serves_other_shapes_in_turn(spec):
    big, small = attn_case(6), attn_case(0)
    ws = big.run(spec)
    small.run(spec, ws)
    small.check()
    big.out.fill_(7.0)
    big.run(spec, ws)
    big.check()


def test_no_rows(spec):
    c = Cache(2, 3, 16, 2, 64, "bf16", [4, 6])
    a = Attn(c, [0, 0], 4)
    a.run(spec)


def test_offsets_past_32_bits(spec):
    """Pages more than 2^32 bytes apart."""
    page, H, D = 64, 4, 256
    n = (5 << 30) // (page * H * D * 2)
    k = torch.zeros((1, n, page, H * D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Cache(2, 3, page, H, D, "bf16", [150, 101], seed=9)
    at = torch.tensor([[0, n - 1, n // 2], [n - 2, 1, n - 3]], dtype=torch.int32, device="cuda")
    for x, y in ((k, c.k), (v, c.v)):
        x[0, at.view(-1).long()] = y[0, c.table.reshape(-1).long()]
    want = Attn(c, [4, 40], 8, seed=9)
    want.run(spec)
    want.check()
    c.table.copy_(at)
    c.k, c.v, c.n_pages = k, v, n
    got = Attn(c, [4, 40], 8, seed=9)
    got.run(spec)
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


# ---------------------------------------------------------------------------------- commit
def acc_of(spec, kept, status=None):
    a = np.zeros(len(kept), dtype=spec.ACCEPT_OUT_DTYPE)
    a["n_emit"], a["status"] = kept, 0 if status is None else status
    return torch.from_numpy(a.view(np.uint8).copy()).cuda()


@pytest.mark.parametrize("layout", ["pools", "pages"])
@pytest.mark.parametrize("layers,H,D,page,dtype", [(1, 2, 64, 16, "f32"), (12, 4, 256, 64, "bf16"),
                                                   (3, 1, 8, 3, "bf16")])
def test_commit(spec, layout, layers, H, D, page, dtype):
    kv_len = [0, 5, 60, 63, 100, 30]
    kept, k, status = [1, 8, 1, 3, 2, 4], [0, 7, 7, 5, 3, 6], [0, 0, 0, 0, 0, 1]
    c = Cache(6, -(-112 // page), page, H, D, dtype, kv_len, layers=layers, layout=layout, seed=10)
    kp, vp = (npf(x).copy() for x in (c.k, c.v))
    st = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_commit(6, c.desc(spec), acc_of(spec, kept, status), i32(k), st)
    kept[5] = 0  # its acceptance failed
    lens = o_pg.commit(kp, vp, c.table.cpu().numpy(), kv_len, kept, k)
    assert c.kv_len.tolist() == lens and st.tolist() == [0] * 6
    assert np.array_equal(npf(c.k), kp) and np.array_equal(npf(c.v), vp)


def test_commit_of_what_is_out_of_range(spec):
    kv_len = [5, 5, 30, 40, -3, 5]
    c = Cache(6, 2, 16, 2, 64, "bf16", kv_len, seed=11)
    c.table[5, 0] = -1
    kp, vp = (npf(x).copy() for x in (c.k, c.v))
    st = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_commit(6, c.desc(spec), acc_of(spec, [1] * 6), i32([-1, 8, 3, 3, 2, 2]), st)
    assert st.tolist() == [spec.REQ_BAD_K, spec.REQ_BAD_K, spec.REQ_KV_OVERFLOW, spec.REQ_KV_OVERFLOW, 0, 0]
    table = c.table.cpu().numpy()
    lens = o_pg.commit(kp, vp, table[2:], kv_len[2:], [1] * 4, [3, 3, 2, 2])
    assert c.kv_len.tolist() == [5, 5] + lens
    assert np.array_equal(npf(c.k), kp) and np.array_equal(npf(c.v), vp)


def test_commit_of_a_chunk(spec):
    c = Cache(4, 4, 16, 2, 64, "bf16", [0, 50, 60, 3], seed=12)
    before = c.store.clone()
    st = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_commit(4, c.desc(spec), None, i32([40, 0, 9, -2]), st)
    assert c.kv_len.tolist() == [40, 50, 69, 3] and torch.equal(c.store, before)
    assert st.tolist() == [0, 0, spec.REQ_KV_OVERFLOW, spec.REQ_BAD_K]


# -------------------------------------------------------------------------------- together
def test_prompt_cycles_and_rollback_together(spec):
    """A prompt in chunks, then verify passes of which some rows are kept: attention's outputs, and the pages
    byte for byte, are those of a cache that saw the kept tokens alone, one call each."""
    B, H, Hq, D, page = 2, 2, 4, 64, 16
    total = 90
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randn((B, total, (Hq + 2 * H) * D), generator=g, device="cuda")
    wrong = torch.randn((B, total, (Hq + 2 * H) * D), generator=g, device="cuda")
    f = 1e4 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float32) / (D // 2))
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")

    def passes(c, rows, ws):
        """rows: per request a [n, ...] tensor. Append, attend; the outputs."""
        n = [x.shape[0] for x in rows]
        mixed, cu = torch.cat(rows), i32(cu_of(n))
        q = torch.empty((sum(n), Hq * D), device="cuda")
        out = torch.empty_like(q)
        a, d = spec.spec_append_desc(), spec.spec_paged_attn_desc()
        a.q_heads, a.norm_eps, a.rot_dim, a.rot_scale = Hq, EPS, D, 1.0
        a.q, a.k, a.v = (mixed.data_ptr() + 4 * x * D for x in (0, Hq, Hq + H))
        a.q_stride = a.k_stride = a.v_stride = mixed.stride(0)
        a.q_out, a.q_out_stride = q.data_ptr(), q.stride(0)
        a.q_norm = a.k_norm = w.data_ptr()
        a.inv_freq = f.data_ptr()
        d.q_heads, d.scale, d.q, d.q_stride = Hq, D ** -0.5, q.data_ptr(), q.stride(0)
        d.out, d.out_stride = out.data_ptr(), out.stride(0)
        spec.spec_paged_append(B, cu, sum(n), c.desc(spec), 0, a)
        spec.spec_paged_attention(B, cu, sum(n), c.desc(spec), 0, d, None, ws)
        torch.cuda.synchronize()
        return out.split(n)

    def fresh():
        c = Cache(B, -(-total // page), page, H, D, "f32", [0] * B, seed=13)
        c.store.zero_()
        return c

    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    c, outs, at = fresh(), [[] for _ in range(B)], [0, 0]
    for chunk in ([20, 7], [13, 0], [1, 30]):
        for b, o in enumerate(passes(c, [tokens[b, at[b]:at[b] + chunk[b]] for b in range(B)], ws)):
            outs[b].append(o)
            at[b] += chunk[b]
        spec.spec_paged_commit(B, c.desc(spec), None, i32(chunk))
    for kept in ([1, 4], [4, 2], [3, 3], [2, 1]):
        rows = [torch.cat([tokens[b, at[b]:at[b] + kept[b]], wrong[b, at[b]:at[b] + 4 - kept[b]]])
                for b in range(B)]
        for b, o in enumerate(passes(c, rows, ws)):
            outs[b].append(o[:kept[b]])
            at[b] += kept[b]
        spec.spec_paged_commit(B, c.desc(spec), acc_of(spec, kept), i32([3, 3]))
    assert c.kv_len.tolist() == at
    ref, plain = fresh(), [[] for _ in range(B)]
    for i in range(max(at)):
        n = [int(i < at[b]) for b in range(B)]
        for b, o in enumerate(passes(ref, [tokens[b, i:i + n[b]] for b in range(B)], ws)):
            plain[b].append(o)
        spec.spec_paged_commit(B, ref.desc(spec), None, i32(n))
    assert torch.equal(ref.store, c.store) and ref.kv_len.tolist() == at
    for b in range(B):
        x, y = torch.cat(outs[b]), torch.cat(plain[b])
        # both sides within the tolerance of the same sums
        assert (x - y).norm() <= 2 * tol(D, "f32") * y.norm()
