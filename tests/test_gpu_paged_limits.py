"""The paged cache's calls at the edges of what spec.h allows: weights that are not finite, most heads, lengths
past every position, pages of other sizes, many rows that do not run. Tolerances and helpers as in
test_gpu_paged."""

import numpy as np
import pytest
import torch

from oracle import paged as o_pg
from test_gpu_paged import EPS, Attn, Cache, acc_of, cu_of, i32, npf, run_append, spec, torch_dt  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,D,rot,pairs", [
    ("bf16", 128, 64, "half"), ("f32", 64, 32, "half"), ("bf16", 128, 64, "side"), ("f32", 64, 20, "side"),
    ("bf16", 96, 32, "half"), ("bf16", 64, 20, "half"), ("f32", 64, 0, "half")])
def test_a_weight_that_is_not_finite_shows_in_its_dim_and_its_pairs(spec, dtype, D, rot, pairs, what):  # noqa: F811
    """y = w x / rms of its own dim only, so a dim that is not turned shows its own weight alone."""
    H, Hq, n = 2, 3, 3
    dt = torch_dt[dtype]
    half = torch.finfo(dt).eps / 2
    g = torch.Generator(device="cuda").manual_seed(D + rot)
    x = torch.randn((n, (Hq + 2 * H) * D), generator=g, device="cuda").to(dt)
    f = 1e4 ** (-torch.arange(max(rot // 2, 1), device="cuda", dtype=torch.float32) / max(rot // 2, 1))
    x64 = npf(x).astype(np.float64).reshape(n, Hq + 2 * H, D)
    for at in sorted({0, 7, max(rot - 1, 0), rot % D, D - 1}):
        w = [1 + 0.3 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
        w[0][at] = w[1][at] = what
        c = Cache(1, 2, 8, H, D, dtype, [5])
        out = torch.zeros((n, Hq * D), dtype=dt, device="cuda")
        d, e = spec.spec_append_desc(), x.element_size()
        d.q_heads, d.norm_eps, d.rot_dim, d.rot_interleaved, d.rot_scale = Hq, EPS, rot, pairs == "side", 1.0
        d.q, d.k, d.v = (x.data_ptr() + e * i * D for i in (0, Hq, Hq + H))
        d.q_stride = d.k_stride = d.v_stride = x.stride(0)
        d.q_out, d.q_out_stride, d.inv_freq = out.data_ptr(), out.stride(0), f.data_ptr()
        d.q_norm, d.k_norm = (v.data_ptr() for v in w)
        spec.spec_paged_append(1, i32([0, n]), n, c.desc(spec), 0, d)
        got_q, (k, _) = npf(out).astype(np.float64).reshape(n, Hq, D), c.np(0)
        table = c.table.cpu().numpy()[0]
        for r in range(n):
            page, i = o_pg.place(table, 5 + r, 8, c.n_pages)
            for got, src, v in [(got_q[r], x64[r, :Hq], w[0]), (k[page, i], x64[r, Hq:Hq + H], w[1])]:
                for h in range(len(got)):
                    with np.errstate(invalid="ignore"):
                        want = o_pg.turned(src[h], 5 + r, npf(v), EPS, rot, pairs == "side", npf(f), 1.0)
                    fin = np.isfinite(want)
                    assert np.array_equal(got[h][~fin], want[~fin], equal_nan=True), (at, r, h)
                    top = np.abs(want[fin]).max()
                    assert (np.abs(got[h][fin] - want[fin]) <=
                            half * np.abs(want[fin]) + 32 * 2.0 ** -24 * top).all(), (at, r, h)


@pytest.mark.parametrize("Hq,H", [(1, 65535), (65535, 65536), (65536, 65536)])
@pytest.mark.parametrize("n", [0, 1, 2])
def test_append_of_the_most_heads(spec, Hq, H, n):  # noqa: F811
    """131,071 turns of a warp for a row, 196,607 and 196,608: no more parts of one than a grid has. Without rows
    too, where the call still says that every request is well."""
    D = 136
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((n, (Hq + 2 * H) * D), generator=g, device="cuda").to(torch.bfloat16)
    pages = torch.zeros((2, 3, 1, H * D), dtype=torch.bfloat16, device="cuda")
    table, kv_len = i32([[2, 0]]), torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.zeros((n, Hq * D), dtype=torch.bfloat16, device="cuda")
    c, d = spec.spec_paged_cache(), spec.spec_append_desc()
    c.dtype, c.layers, c.kv_heads, c.head_dim = spec.SPEC_BF16, 1, H, D
    c.page_size, c.n_pages, c.max_pages, c.table_stride = 1, 3, 2, 2
    c.k_pages, c.v_pages, c.page_stride = pages[0].data_ptr(), pages[1].data_ptr(), H * D * 2
    c.page_table, c.kv_len = table.data_ptr(), kv_len.data_ptr()
    d.q_heads, d.rot_dim, d.rot_scale = Hq, 0, 1.0
    d.q, d.k, d.v = (x.data_ptr() + 2 * i * D for i in (0, Hq, Hq + H))
    d.q_stride = d.k_stride = d.v_stride = x.stride(0)
    d.q_out, d.q_out_stride = out.data_ptr(), out.stride(0)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_append(1, i32([0, n]), n, c, 0, d, None, status)
    # without norms and rotation everything is copied
    assert status.tolist() == [0] and torch.equal(out, x[:, :Hq * D])
    at = [2, 0][:n]
    assert torch.equal(pages[0, at, 0], x[:, Hq * D:(Hq + H) * D])
    assert torch.equal(pages[1, at, 0], x[:, (Hq + H) * D:])
    assert not pages[:, [2, 0][n:] + [1]].any()


# ---------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,layout", [(192, "pools"), (320, "pages"), (4160, "pools"), (48, "pools")])
def test_pages_of_whole_blocks(spec, D, page, layout):  # noqa: F811
    """Pages of three and five blocks of positions, and a cache per request in one page; a page that is not there
    among several, lengths on either side of pages' ends, what masked positions hold."""
    lens, kv_len = [5, 130, 0, 3, 70], [page - 2, 0, 4, 2 * page, 300]
    pages = -(-max(n + P for n, P in zip(lens, kv_len)) // page)
    c = Cache(5, pages, page, 2, D, "bf16", kv_len, layers=2, layout=layout, seed=41)
    a = Attn(c, lens, 6, layer=1, seed=41)
    a.run(spec)
    a.check()
    clean = a.out.clone()
    for b, (n, P) in enumerate(zip(lens, kv_len)):  # behind the last row's position
        for x in (c.k, c.v):
            if (P + n) % page:
                x[1, c.table[b, (P + n) // page].long(), (P + n) % page:] = float("nan")
    a.run(spec)
    assert torch.equal(a.out, clean)
    c.table[3, 1] = -1
    c.table[4, 0] = c.n_pages
    for x in (c.k, c.v):
        x.nan_to_num_(nan=0.5)
    a.run(spec)
    a.check()


@pytest.mark.parametrize("dtype,D,Hq,pad", [("bf16", 64, 4, 0), ("bf16", 128, 6, 3), ("f32", 64, 4, 0), ("f32", 72, 2, 1)])
def test_many_rows_that_requests_own_and_do_not_run(spec, dtype, D, Hq, pad):  # noqa: F811
    """A padded batch: slots of thousands of rows of which a few run, all or none; rows behind and before them."""
    lens, runs = [6000, 5, 0, 3000, 40, 700], [3, 0, 0, 1, 40, 0]
    c = Cache(6, 20, 16, 2, D, dtype, [200, 7, 5, 0, 100, 30], seed=42)
    a = Attn(c, lens, Hq, n_rows=runs, pad=pad, first=9, extra=11, seed=42)
    a.run(spec)
    a.check()
    d, out = a.desc(spec), a.out.clone()  # without lse
    d.lse = None
    a.out.fill_(7.0)
    n = spec.spec_paged_attention_workspace_bytes(6, a.rows, c.desc(spec), d)
    spec.spec_paged_attention(6, i32(a.cu), a.rows, c.desc(spec), 0, d, i32(runs),
                              torch.zeros(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a.out, out)


# ------------------------------------------------------------------------- lengths past everything
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_near_the_end_of_their_type(spec, dtype):  # noqa: F811
    """As any length past the table: nothing is written or cleared and the status says so; rows attend to all that
    is there."""
    top = 2 ** 63 - 1
    lens = [top, top - 1, top - 3, 2 ** 62, 2 ** 31 - 3, 2 ** 32, -2 ** 63, 20]
    c = Cache(8, 3, 16, 2, 64, dtype, [0] * 8, seed=43)
    c.kv_len.copy_(torch.tensor(lens, dtype=torch.int64))
    before = c.store.clone()
    n = 4
    run_append(spec, c, cu_of([n] * 8), n * 8, 4, 0, "half", True, seed=43)  # its status too
    assert all(torch.equal(x[:, c.table[:6].reshape(-1).long()], y[:, c.table[:6].reshape(-1).long()])
               for x, y in zip(c.store, before))
    a = Attn(c, [n] * 8, 4, seed=43)
    a.run(spec)
    a.check()
    before = c.store.clone()
    st = torch.full((8,), 9, dtype=torch.int32, device="cuda")
    spec.spec_paged_commit(8, c.desc(spec), acc_of(spec, [1] * 8), i32([3] * 8), st)
    assert st.tolist() == [spec.REQ_KV_OVERFLOW] * 6 + [0, 0]
    assert (c.kv_len[:6] >= 2 ** 31 - 3).all() and c.kv_len.tolist()[3:] == [x + 1 for x in lens[3:6]] + [1, 21]
    keep = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    keep[c.table[6:].reshape(-1).long()] = False
    assert all(torch.equal(x[:, keep], y[:, keep]) for x, y in zip(c.store, before))
    spec.spec_paged_commit(8, c.desc(spec), None, i32([3] * 8), st)
    assert st.tolist() == [spec.REQ_KV_OVERFLOW] * 6 + [0, 0] and (c.kv_len[:6] > 0).all()


# --------------------------------------------------------------------- values of their descriptions
@pytest.mark.parametrize("pairs", ["half", "side"])
@pytest.mark.parametrize("dtype,pos", [("f32", [-7, -60000]), ("bf16", [-1, -(2 ** 20)])])
def test_positions_before_zero_turn_backwards(spec, pairs, dtype, pos):  # noqa: F811
    c = Cache(2, 3, 16, 2, 64, dtype, [5, 9], seed=44)
    run_append(spec, c, [0, 3, 7], 7, 4, 64, pairs, True, pos=pos, seed=44)


@pytest.mark.parametrize("dtype,D,page", [("bf16", 64, 16), ("bf16", 128, 64), ("bf16", 256, 32), ("f32", 64, 16)])
def test_a_scale_of_zero_gives_the_mean(spec, dtype, D, page):  # noqa: F811
    c = Cache(3, -(-200 // page), page, 2, D, dtype, [100, 3, 126], seed=45)
    c.table[0, 0] = -1
    a = Attn(c, [5, 1, 40], 4, scale=0.0, n_rows=[5, 1, 38], seed=45)
    a.run(spec)
    a.check()


@pytest.mark.parametrize("B,R,Hq,H,D,dtype", [
    (1, 8, 4, 2, 64, "bf16"), (5, 1, 1, 1, 64, "bf16"), (64, 8, 4, 2, 128, "bf16"), (65, 8, 4, 2, 128, "bf16"),
    (300, 3, 2, 1, 64, "bf16"), (512, 2, 1, 1, 64, "f32"), (64, 8, 2, 1, 64, "f32")])
def test_few_rows_of_many_requests_that_do_not_run(spec, B, R, Hq, H, D, dtype):  # noqa: F811
    """By the blocks of a request up to 64 of them and eight rows each, by a warp to a row above; one request that
    owns them all among others that own none."""
    c = Cache(B, 4, 16, H, D, dtype, [b % 37 for b in range(B)], seed=46)
    a = Attn(c, [R] * B, Hq, n_rows=[(3 * b) % (R + 1) for b in range(B)], first=2, extra=3, seed=46)
    a.run(spec)
    a.check()
    c = Cache(B, 40, 16, H, D, dtype, [b % 37 for b in range(B)], seed=47)
    a = Attn(c, [0] * (B - 1) + [R * B], Hq, n_rows=[0] * (B - 1) + [2], first=1, seed=47)
    a.run(spec)
    a.check()
