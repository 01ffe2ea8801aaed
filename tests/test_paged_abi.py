"""CPU checks of the paged cache's calls: struct layouts against the C compiler, refusals on the host before
anything touches the GPU, and the compiler's resource report."""

import ctypes
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2
P = 1 << 20


@pytest.fixture(scope="module")
def spec():
    from mtp_speculative_decoding_spec_gb300 import build
    build.build()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


@pytest.mark.parametrize("name", ["spec_paged_cache", "spec_append_desc", "spec_paged_attn_desc"])
def test_struct_layout_matches_the_c_compiler(spec, name, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    t = getattr(spec, name)
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec.h"', "int main(void){",
            f'printf("%zu\\n", sizeof({name}));']
    prog += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in t._fields_]
    (tmp_path / "l.c").write_text("\n".join(prog + ["return 0;}"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == \
        [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]


def args(spec):
    """Two layers of 10 pages of 16 positions, 2 heads of 128 bf16: a row is 512 bytes, a page 8,192."""
    c = spec.spec_paged_cache()
    c.dtype, c.layers, c.kv_heads, c.head_dim, c.page_size, c.n_pages = spec.SPEC_BF16, 2, 2, 128, 16, 10
    c.k_pages = c.v_pages = c.page_table = c.kv_len = P
    c.page_stride, c.layer_stride, c.table_stride, c.max_pages = 8192, 81920, 5, 4
    a = spec.spec_append_desc()
    a.q_heads, a.norm_eps, a.rot_dim, a.rot_scale = 8, 1e-6, 64, 1.0
    a.q = a.k = a.v = a.q_out = a.q_norm = a.k_norm = a.inv_freq = a.pos = P
    a.q_stride = a.q_out_stride = 1024
    a.k_stride = a.v_stride = 256
    d = spec.spec_paged_attn_desc()
    d.q_heads, d.scale = 8, 1.0
    d.q = d.out = d.lse = P
    d.q_stride = d.out_stride = 1024
    return c, a, d


def append(spec, c, a, B=2, cu=P, rows=8, layer=0, n_rows=None, status=None):
    return spec._abi.lib().spec_paged_append(B, cu, rows, c, layer, a, n_rows, status, None)


def attend(spec, c, d, B=2, cu=P, rows=8, layer=0, n_rows=None, ws=P, n=1 << 40):
    return spec._abi.lib().spec_paged_attention(B, cu, rows, c, layer, d, n_rows, ws, n, None)


def commit(spec, c, B=2, acc=P, k=P, status=None):
    return spec._abi.lib().spec_paged_commit(B, c, acc, k, status, None)


CACHE_BAD = [
    ("dtype", 2, INVALID), ("layers", 0, INVALID), ("kv_heads", 0, INVALID), ("head_dim", 0, INVALID),
    ("head_dim", 100, INVALID), ("head_dim", 264, UNSUPPORTED), ("page_size", 0, INVALID),
    ("n_pages", 0, INVALID), ("n_pages", 1 << 31, UNSUPPORTED), ("max_pages", 0, INVALID),
    ("max_pages", 6, INVALID), ("page_size", 1 << 30, UNSUPPORTED), ("k_pages", None, INVALID),
    ("v_pages", None, INVALID), ("k_pages", P + 8, INVALID), ("v_pages", P + 2, INVALID),
    ("page_table", None, INVALID), ("page_table", P + 2, INVALID), ("kv_len", None, INVALID),
    ("kv_len", P + 4, INVALID), ("page_stride", 8191, INVALID), ("page_stride", 8176, INVALID),
    ("page_stride", -8192, INVALID), ("layer_stride", -81920, INVALID), ("layer_stride", 81904, INVALID),
    ("layer_stride", 8192, INVALID), ("page_stride", 1 << 60, UNSUPPORTED),
]


@pytest.mark.parametrize("field,value,status", CACHE_BAD)
def test_cache_refusals(spec, field, value, status):
    c, a, d = args(spec)
    setattr(c, field, value)
    assert append(spec, c, a) == status
    assert attend(spec, c, d) == status
    assert commit(spec, c) == status


def test_layouts_of_layers(spec):
    """A page's layers together, and layers of whole pools, are caches; what overlaps is none. With no
    queries and no keys there is nothing to do, so that the call succeeds without a GPU."""
    c, a, _ = args(spec)
    a.q_heads, a.k, a.v = 0, None, None
    assert append(spec, c, a) == 0
    c.page_stride, c.layer_stride = 16384, 8192
    assert append(spec, c, a, layer=1) == 0
    c.page_stride = 16384 - 16
    assert append(spec, c, a) == INVALID
    c.n_pages, c.page_stride = 1, 0
    assert append(spec, c, a) == 0


APPEND_BAD = [
    ("q_heads", -1, INVALID), ("q_heads", 65537, UNSUPPORTED), ("q", None, INVALID), ("q_out", None, INVALID),
    ("k", None, INVALID), ("v", None, INVALID), ("q", P + 1, INVALID), ("q_out", P + 1, INVALID),
    ("k", P + 1, INVALID), ("v", P + 1, INVALID), ("q_stride", 1023, INVALID), ("q_out_stride", 1023, INVALID),
    ("k_stride", 255, INVALID), ("v_stride", 0, INVALID), ("rot_dim", 63, INVALID), ("rot_dim", -2, INVALID),
    ("rot_dim", 130, INVALID), ("inv_freq", None, INVALID), ("inv_freq", P + 2, INVALID),
    ("q_norm", P + 2, INVALID), ("k_norm", P + 1, INVALID), ("pos", P + 4, INVALID),
    ("norm_eps", -1.0, INVALID), ("norm_eps", float("nan"), INVALID),
]


@pytest.mark.parametrize("field,value,status", APPEND_BAD)
def test_append_refusals(spec, field, value, status):
    c, a, _ = args(spec)
    setattr(a, field, value)
    assert append(spec, c, a) == status


ATTN_BAD = [
    ("q_heads", 0, INVALID), ("q_heads", 7, INVALID), ("q_heads", 130, UNSUPPORTED), ("q", None, INVALID),
    ("out", None, INVALID), ("q", P + 1, INVALID), ("out", P + 1, INVALID), ("lse", P + 2, INVALID),
    ("q_stride", 1023, INVALID), ("out_stride", 1023, INVALID),
]


@pytest.mark.parametrize("field,value,status", ATTN_BAD)
def test_attention_refusals(spec, field, value, status):
    c, _, d = args(spec)
    setattr(d, field, value)
    if field == "q_heads" and value > 8:
        d.q_stride = d.out_stride = 1 << 16
    assert attend(spec, c, d) == status


def test_call_refusals(spec):
    c, a, d = args(spec)
    for kw, status in ((dict(B=0), INVALID), (dict(B=513), UNSUPPORTED), (dict(cu=None), INVALID),
                       (dict(cu=P + 2), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID),
                       (dict(layer=-1), INVALID), (dict(layer=2), INVALID), (dict(n_rows=P + 1), INVALID)):
        assert append(spec, c, a, **kw) == status, kw
        assert attend(spec, c, d, **kw) == status, kw
    assert append(spec, c, a, status=P + 2) == INVALID
    for kw in (dict(ws=None), dict(ws=P + 128)):
        assert attend(spec, c, d, **kw) == INVALID
    for kw, status in ((dict(B=0), INVALID), (dict(B=513), UNSUPPORTED), (dict(k=None), INVALID),
                       (dict(acc=P + 4), INVALID), (dict(status=P + 1), INVALID), (dict(k=P + 2), INVALID)):
        assert commit(spec, c, **kw) == status, kw
    lib = spec._abi.lib()
    assert lib.spec_paged_append(1, P, 1, None, 0, a, None, None, None) == INVALID
    assert lib.spec_paged_append(1, P, 1, c, 0, None, None, None, None) == INVALID
    assert lib.spec_paged_attention(1, P, 1, None, 0, d, None, P, 1 << 40, None) == INVALID
    assert lib.spec_paged_attention(1, P, 1, c, 0, None, None, P, 1 << 40, None) == INVALID
    assert lib.spec_paged_commit(1, None, P, P, None, None) == INVALID
    assert spec.spec_paged_attention_workspace_bytes(0, 8, c, d) == 0
    assert spec.spec_paged_attention_workspace_bytes(2, -1, c, d) == 0


@pytest.mark.parametrize("dtype,D,rows,over", [
    # 8 query heads on 2: G = 4; tiles of 128 rows and of 16, two requests
    ("bf16", 128, (4096 - 2) * 32, False), ("bf16", 128, (4096 - 1) * 32, True),
    ("bf16", 72, (12288 - 2) * 4, False), ("bf16", 72, (12288 - 1) * 4, True),
    ("f32", 64, (12288 - 2) * 4, False), ("f32", 64, (12288 - 1) * 4, True),
])
def test_most_rows(spec, dtype, D, rows, over):
    c, _, d = args(spec)
    c.dtype, c.head_dim = (spec.SPEC_BF16 if dtype == "bf16" else spec.SPEC_F32), D
    c.page_stride, c.layer_stride = 1 << 14, 10 << 14
    got = attend(spec, c, d, rows=rows, n=0)
    assert (got == UNSUPPORTED) if over else got not in (0, UNSUPPORTED)


def test_register_budget_and_no_spills(spec):
    """As for the other kernels: a block's warps go round-robin over four sub-partitions of 16K registers
    each, and no kernel spills."""
    logs = glob.glob(os.path.join(ROOT, "mtp_speculative_decoding_spec_gb300", "_build", "paged", "*.ptxas.log"))
    threads = {"append_kernel": 128, "paged_commit_kernel": 256, "attn_simt_kernel": 256,
               "attn_tc_kernel": 384, "paged_join_kernel": 256}
    seen = set()
    for path in logs:
        name = None
        for line in open(path):
            m = re.search(r"Compiling entry function '(\w+)'", line)
            if m:
                name = m.group(1)
            m = re.search(r"(\d+) bytes spill stores", line)
            if m and name:
                assert int(m.group(1)) == 0, f"{name} spills"
            m = re.search(r"Used (\d+) registers", line)
            if m and name:
                kernel = next(k for k in threads if k in name)
                warps = threads[kernel] // 32
                assert -(-int(m.group(1)) // 8) * 8 * 32 * -(-warps // 4) <= 16384, name
                seen.add(kernel)
    assert seen == set(threads)
