"""The paged KV cache's calls as a server makes them: many requests of like lengths (whose units are not
cut), captured cycles, two calls at once, the most rows there can be. Tolerances and helpers as in
test_gpu_paged."""

import numpy as np
import pytest
import torch

from oracle import paged as o_pg
from test_gpu_paged import (EPS, Attn, Cache, acc_of, cu_of, i32, npf, run_append, spec, tol,  # noqa: F401
                            torch_dt)

pytestmark = pytest.mark.gpu


def check_some(a, requests):
    """Of a call with many rows, these requests against float64."""
    c = a.c
    k, v = c.np(a.layer)
    table, lens = c.table.cpu().numpy(), c.kv_len.tolist()
    for b in requests:
        s = slice(a.cu[b], a.cu[b + 1])
        q = npf(a.q[s])[:, :a.Hq * c.D].reshape(-1, a.Hq, c.D)
        want, lse = o_pg.attend(q, k, v, table[b:b + 1], [lens[b]], [0, len(q)], None, a.scale)
        got = npf(a.out[s])[:, :a.Hq * c.D].reshape(want.shape).astype(np.float64)
        assert np.linalg.norm(got - want) <= tol(c.D, c.dtype) * np.linalg.norm(want), b
        assert np.abs(npf(a.lse[s]) - lse).max() <= 64 * np.sqrt(c.D) * 2.0 ** -24


@pytest.mark.parametrize("D,H,Hq,page", [(64, 4, 8, 16), (128, 4, 4, 64), (256, 4, 8, 32), (128, 1, 64, 8)])
@pytest.mark.parametrize("long", [0, 700])
def test_requests_of_like_lengths(spec, D, H, Hq, page, long):  # noqa: F811
    """As many units as the SMs or fewer, of like costs, so that each has a CTA to itself; and with one that is
    longer, so that they are cut."""
    B = 36
    lens = [300 + b % 20 for b in range(B)]
    lens[5] += long
    c = Cache(B, -(-(max(lens) + 3) // page), page, H, D, "bf16", lens, seed=21)
    c.table[7, 2] = -1
    c.table[8] = c.n_pages
    a = Attn(c, [3] * B, Hq, seed=21, n_rows=[b % 4 for b in range(B)])
    a.run(spec)
    a.check()


@pytest.mark.parametrize("D,H,Hq,page,lens,kv_len", [
    (128, 16, 32, 16, [0, 1, 77, 300, 600], [5, 90, 100, 40, 0]),
    (64, 8, 16, 64, [700, 3, 650], [0, 200, 100]),
    (256, 8, 8, 32, [3] * 30, [200 + 7 * b for b in range(30)]),
    (256, 2, 8, 8, [500, 0, 1, 1, 1, 300] * 3, [30 * b for b in range(18)]),
    # far more than an equal share, so that units are cut all the same
    (128, 4, 4, 128, [1] * 39 + [2], [20] * 39 + [4000]),
    (64, 1, 2, 16, [1] * 255 + [5], [b % 50 for b in range(256)]),
    (64, 1, 2, 16, [1] * 256 + [5], [b % 50 for b in range(257)]),
])
def test_several_units_of_a_cta(spec, D, H, Hq, page, lens, kv_len):  # noqa: F811
    """More units than SMs, dealt out whole by their costs, or cut; a page that is not there among them."""
    c = Cache(len(lens), -(-max(p + n for p, n in zip(kv_len, lens)) // page), page, H, D, "bf16", kv_len, seed=26)
    c.table[2, 0] = -1
    a = Attn(c, lens, Hq, seed=26)
    a.run(spec)
    a.check()


@pytest.mark.parametrize("dtype,D,rot,pairs,pad", [
    ("bf16", 64, 64, "half", 0), ("bf16", 64, 64, "side", 0), ("bf16", 64, 20, "half", 0), ("bf16", 64, 0, "half", 0),
    ("bf16", 40, 16, "half", 0), ("bf16", 64, 32, "half", 3), ("f32", 64, 48, "half", 0)])
def test_append_of_many_rows(spec, dtype, D, rot, pairs, pad):  # noqa: F811
    """As many rows as let a warp take several of a row's heads after one another."""
    c = Cache(3, 80, 16, 1, D, dtype, [3, 7, 40], seed=27)
    run_append(spec, c, cu_of([1200, 0, 800]), 2005, 32, rot, pairs, True, pad=pad, in_place=pad == 0, seed=27)


def test_a_page_twice_in_a_table(spec):  # noqa: F811
    c = Cache(2, 8, 16, 2, 128, "bf16", [100, 90], seed=22)
    c.table[0, 3] = c.table[0, 1]
    c.table[1, 0] = c.table[0, 1]
    a = Attn(c, [3, 20], 4, seed=22)
    a.run(spec)
    a.check()


@pytest.mark.parametrize("dtype,rows", [("bf16", [14] * 512), ("f32", [6] * 384 + [5] * 128)])
def test_the_most_tiles(spec, dtype, rows):  # noqa: F811
    """rows * 64 / tile + 512 requests = 4,096 tiles of 128 rows and 12,288 of 16, whose costs lie beside the
    largest heads' blocks in shared memory."""
    c = Cache(512, 5 if dtype == "bf16" else 6, 16, 1, 256, dtype, [b % 60 for b in range(512)], seed=23)
    a = Attn(c, rows, 64, seed=23)
    a.run(spec)
    assert torch.isfinite(a.out).all()
    check_some(a, [0, 1, 59, 383, 511])
    more = Attn(c, rows[:-1] + [rows[-1] + 2], 64, seed=23)
    assert spec.spec_paged_attention_workspace_bytes(512, more.rows, c.desc(spec), more.desc(spec)) == 0


class Cycle:
    """A verify cycle's three calls on one cache, with fixed inputs."""

    def __init__(self, spec, dtype, D, page, rows, kept, past, seed, ws):  # noqa: F811
        H, Hq = 2, 4
        B = len(past)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.c = Cache(B, -(-(max(past) + 40) // page), page, H, D, dtype, past, seed=seed)
        self.mixed = torch.randn((B * rows, (Hq + 2 * H) * D), generator=g, device="cuda").to(torch_dt[dtype])
        self.q = torch.empty((B * rows, Hq * D), dtype=torch_dt[dtype], device="cuda")
        self.out = torch.empty_like(self.q)
        self.f = 1e4 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float32) / (D // 2))
        self.w = torch.ones(D, device="cuda")
        self.cu, self.k, self.acc = i32(cu_of([rows] * B)), i32([rows - 1] * B), acc_of(spec, kept)
        self.status = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.B, self.rows, self.spec, self.ws = B, B * rows, spec, ws
        a, d, e = spec.spec_append_desc(), spec.spec_paged_attn_desc(), self.q.element_size()
        a.q_heads, a.norm_eps, a.rot_dim, a.rot_scale = Hq, EPS, D, 1.0
        a.q, a.k, a.v = (self.mixed.data_ptr() + e * x * D for x in (0, Hq, Hq + H))
        a.q_stride = a.k_stride = a.v_stride = self.mixed.stride(0)
        a.q_out, a.q_out_stride = self.q.data_ptr(), self.q.stride(0)
        a.q_norm = a.k_norm = self.w.data_ptr()
        a.inv_freq = self.f.data_ptr()
        d.q_heads, d.scale, d.q, d.q_stride = Hq, D ** -0.5, self.q.data_ptr(), self.q.stride(0)
        d.out, d.out_stride = self.out.data_ptr(), self.out.stride(0)
        self.a, self.d, self.desc = a, d, self.c.desc(spec)

    def enqueue(self, stream=None):
        s = self.spec
        s.spec_paged_append(self.B, self.cu, self.rows, self.desc, 0, self.a, None, self.status, stream)
        s.spec_paged_attention(self.B, self.cu, self.rows, self.desc, 0, self.d, None, self.ws, stream)
        s.spec_paged_commit(self.B, self.desc, self.acc, self.k, None, stream)

    def state(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.c.store, self.c.kv_len, self.q, self.out, self.status)]


KINDS = [("bf16", 128, 16, 4, [2, 1, 4], [100, 0, 61], 31), ("f32", 64, 7, 2, [1, 2, 1, 0], [10, 3, 0, 30], 32)]


def test_captured_cycles_and_graphs_that_share_a_workspace(spec):  # noqa: F811
    """Two caches' cycles, captured, share one workspace and are replayed in turn: each replay goes on from the
    lengths that the one before left, and the bytes are those of the same calls without graphs."""
    want = []
    for kind in KINDS:
        x = Cycle(spec, *kind, torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"))
        want.append([])
        for _ in range(4):
            x.enqueue()
            want[-1].append(x.state())
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    xs, graphs = [Cycle(spec, *kind, ws) for kind in KINDS], []
    for x in xs:
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.enqueue()
    for n in range(4):
        for g in graphs:
            g.replay()
        for x, w in zip(xs, want):
            assert all(torch.equal(p, q) for p, q in zip(x.state(), w[n]))


def test_two_at_once(spec):  # noqa: F811
    """On streams of their own, with workspaces of their own, over pages that both read."""
    c = Cache(4, 70, 64, 4, 128, "bf16", [4000, 3, 700, 2900], seed=24)
    a, b = Attn(c, [8, 100, 0, 7], 8, seed=24), Attn(c, [1, 0, 300, 2], 16, seed=25)
    wa, wb = a.run(spec), b.run(spec)
    a.check()
    b.check()
    alone = [x.clone() for x in (a.out, a.lse, b.out, b.lse)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    calls = [(x, i32(x.cu), c.desc(spec), x.desc(spec), w, s) for x, w, s in zip((a, b), (wa, wb), streams)]
    for x in (a, b):
        x.out.zero_()
        x.lse.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for x, cu, cd, ad, w, s in calls:
            spec.spec_paged_attention(c.B, cu, x.rows, cd, 0, ad, None, w, s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((a.out, a.lse, b.out, b.lse), alone))


def test_cycles_on_another_stream(spec):  # noqa: F811
    for kind in KINDS:
        x, y = (Cycle(spec, *kind, torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")) for _ in range(2))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            x.enqueue()
            y.enqueue(side)
        assert all(torch.equal(p, q) for p, q in zip(x.state(), y.state()))
