"""CPU checks of the trunk's token mixers: struct layouts against the C compiler, refusals on the host
before anything touches the GPU, and the compiler's resource report."""

import ctypes
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def spec():
    from mtp_speculative_decoding_spec_gb300 import build
    build.build()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


@pytest.mark.parametrize("name", ["spec_delta_desc", "spec_attn_desc"])
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


def delta_args(spec):
    st = spec.spec_state_desc()
    st.rec_layers, st.rec_heads, st.rec_dk, st.rec_dv, st.n_slots = 2, 4, 128, 128, 9
    st.rec_live = st.rec_slots = st.live_slot = 1 << 20
    st.step_a = st.step_b = st.step_c = 1 << 20
    d = spec.spec_delta_desc()
    d.dtype, d.key_heads, d.scale = spec.SPEC_BF16, 2, 1.0
    d.q = d.k = d.v = d.log_decay = d.beta = d.out = 1 << 20
    d.q_stride = d.k_stride = 256
    d.v_stride = d.out_stride = 512
    return st, d


def rows_call(spec, st, d, B=1, R=8, layer=0, mode=0):
    return spec._abi.lib().spec_delta_rows(B, R, st, layer, mode, d, None, None)


def prefill_call(spec, st, d, B=1, rows=64, layer=0, cu=1 << 20, init=None, ws=1 << 20, n=None):
    if n is None:
        n = spec.spec_delta_prefill_workspace_bytes(max(rows, 0), max(B, 1), st)
    return spec._abi.lib().spec_delta_prefill(B, cu, rows, st, layer, d, init, ws, n, None)


DELTA_BAD = [
    ("st", "rec_layers", 0, INVALID), ("st", "rec_heads", 0, INVALID), ("st", "rec_dk", 0, INVALID),
    ("st", "rec_dv", 6, INVALID), ("st", "rec_dv", 0, INVALID), ("st", "rec_dk", 257, UNSUPPORTED),
    ("st", "rec_live", None, INVALID), ("st", "rec_live", (1 << 20) + 4, INVALID),
    ("d", "dtype", 2, INVALID), ("d", "key_heads", 0, INVALID), ("d", "key_heads", 3, INVALID),
    ("d", "q", None, INVALID), ("d", "k", None, INVALID), ("d", "v", None, INVALID),
    ("d", "log_decay", None, INVALID), ("d", "beta", None, INVALID), ("d", "out", None, INVALID),
    ("d", "q_stride", 255, INVALID), ("d", "k_stride", 0, INVALID), ("d", "v_stride", 511, INVALID),
    ("d", "out_stride", 511, INVALID), ("d", "q", (1 << 20) + 1, INVALID),
    ("d", "beta", (1 << 20) + 2, INVALID),
]


@pytest.mark.parametrize("where,field,value,status", DELTA_BAD)
def test_delta_refusals(spec, where, field, value, status):
    for call in (rows_call, prefill_call):
        st, d = delta_args(spec)
        setattr({"st": st, "d": d}[where], field, value)
        if field == "rec_dk":
            d.q_stride = d.k_stride = 1024
        assert call(spec, st, d) == status, call


def test_delta_rows_refusals(spec):
    st, d = delta_args(spec)
    for kw in (dict(B=0), dict(R=0), dict(R=9), dict(layer=-1), dict(layer=2), dict(mode=3),
               dict(mode=-1)):
        assert rows_call(spec, st, d, **kw) == INVALID, kw
    for field, mode in (("rec_slots", 0), ("step_a", 1), ("step_b", 1), ("step_c", 1),
                        ("live_slot", 2)):
        st, d = delta_args(spec)
        setattr(st, field, None)
        assert rows_call(spec, st, d, mode=mode) == INVALID, field
    st, d = delta_args(spec)
    st.n_slots = 8
    assert rows_call(spec, st, d) == INVALID
    lib = spec._abi.lib()
    assert lib.spec_delta_rows(1, 1, None, 0, 0, d, None, None) == INVALID
    assert lib.spec_delta_rows(1, 1, st, 0, 0, None, None, None) == INVALID


def test_delta_prefill_refusals(spec):
    st, d = delta_args(spec)
    for kw in (dict(B=0), dict(rows=-1), dict(rows=1 << 31), dict(layer=2), dict(cu=None),
               dict(ws=None), dict(ws=(1 << 20) + 128), dict(n=0), dict(init=(1 << 20) + 8)):
        assert prefill_call(spec, st, d, **kw) == INVALID, kw
    assert spec.spec_delta_prefill_workspace_bytes(10, 0, st) == 0
    assert spec.spec_delta_prefill_workspace_bytes(-1, 1, st) == 0
    assert spec.spec_delta_prefill_workspace_bytes(0, 1, st) > 0
    with pytest.raises(spec.SpecError, match="SPEC_ERR_INVALID"):
        import torch
        spec.spec_delta_prefill(0, 1 << 20, 1, st, 0, d, None, torch.zeros(1), stream=0)


def attn_args(spec):
    st = spec.spec_state_desc()
    st.kv, st.kv_layers, st.kv_capacity, st.kv_row_bytes = 1 << 20, 2, 100, 2 * 128 * 2
    st.kv_request_stride, st.kv_len = 4 * 100 * 512, 1 << 20
    d = spec.spec_attn_desc()
    d.dtype, d.q_heads, d.kv_heads, d.head_dim, d.scale = spec.SPEC_BF16, 8, 2, 128, 1.0
    d.q = d.out = d.prefix_k = d.prefix_v = 1 << 20
    d.q_stride = d.out_stride = 1024
    d.prefix_capacity, d.prefix_stride = 50, 256
    return st, d


ATTN_BAD = [
    ("st", "kv", None, INVALID), ("st", "kv", (1 << 20) + 8, INVALID), ("st", "kv_len", None, INVALID),
    ("st", "kv_layers", 0, INVALID), ("st", "kv_capacity", 0, INVALID),
    ("st", "kv_row_bytes", 500, INVALID), ("st", "kv_request_stride", 8, INVALID),
    ("st", "kv_request_stride", 1024, INVALID), ("st", "kv_capacity", 1 << 31, UNSUPPORTED),
    ("d", "dtype", 2, INVALID), ("d", "kv_heads", 0, INVALID), ("d", "q_heads", 7, INVALID),
    ("d", "q_heads", 0, INVALID), ("d", "head_dim", 100, INVALID), ("d", "head_dim", 0, INVALID),
    ("d", "head_dim", 264, None), ("d", "q_heads", 130, UNSUPPORTED),
    ("d", "q", None, INVALID), ("d", "out", None, INVALID), ("d", "q", (1 << 20) + 1, INVALID),
    ("d", "q_stride", 1023, INVALID), ("d", "out_stride", 1023, INVALID),
    ("d", "prefix_k", None, INVALID), ("d", "prefix_v", (1 << 20) + 2, INVALID),
    ("d", "prefix_capacity", -1, INVALID), ("d", "prefix_capacity", 1 << 31, UNSUPPORTED),
    ("d", "prefix_stride", 255, INVALID), ("d", "prefix_stride", 257, INVALID),
]


@pytest.mark.parametrize("where,field,value,status", ATTN_BAD)
def test_attention_refusals(spec, where, field, value, status):
    st, d = attn_args(spec)
    setattr({"st": st, "d": d}[where], field, value)
    if field == "q_heads" and value > 8:
        d.q_stride = d.out_stride = 1 << 16
    if status is None:  # a head too long, its rows as wide as it says
        st.kv_row_bytes, status = 2 * value * 2, UNSUPPORTED
    got = spec._abi.lib().spec_prefix_attention(2, 4, st, 0, d, None, 1 << 20, 1 << 40, None)
    assert got == status


def test_attention_call_refusals(spec):
    lib = spec._abi.lib()
    st, d = attn_args(spec)
    for B, R, layer, status in ((0, 4, 0, INVALID), (2, 0, 0, INVALID), (2, 9, 0, INVALID),
                                (2, 4, 2, INVALID), (2, 4, -1, INVALID), (1025, 4, 0, UNSUPPORTED)):
        assert lib.spec_prefix_attention(B, R, st, layer, d, None, 1 << 20, 1 << 40, None) == status
    assert lib.spec_prefix_attention(2, 4, None, 0, d, None, 1 << 20, 1 << 40, None) == INVALID
    assert lib.spec_prefix_attention(2, 4, st, 0, None, None, 1 << 20, 1 << 40, None) == INVALID
    assert spec.spec_prefix_attention_workspace_bytes(0, 4, st, d) == 0


def test_register_budget_and_no_spills(spec):
    """As for the verify step's kernels: a block's warps go round-robin over four sub-partitions of
    16K registers each, and no kernel spills."""
    logs = glob.glob(os.path.join(ROOT, "mtp_speculative_decoding_spec_gb300", "_build", "trunk",
                                  "*.ptxas.log"))
    threads = {"delta_scan_kernel": 32, "delta_prep_kernel": 128, "delta_chain_kernel": 384, "attn_simt_kernel": 256, "attn_join_kernel": 256,
               "attn_tc_kernel": 384}
    seen = 0
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
                warps = next(n for k, n in threads.items() if k in name) // 32
                assert -(-int(m.group(1)) // 8) * 8 * 32 * -(-warps // 4) <= 16384, name
                seen += 1
    assert seen >= len(threads)
