"""Limits of spec_prefix_attention that are products of its sizes, on both sides. The calls here have no
workspace, so the ones within the limits are refused too, for that, before anything is launched."""

import pytest

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def spec():
    from mtp_speculative_decoding_spec_gb300 import build
    build.build()
    import mtp_speculative_decoding_spec_gb300 as spec
    return spec


def refusal(spec, B, R, group, dtype, prefix, cap=100, D=64):
    st, d = spec.spec_state_desc(), spec.spec_attn_desc()
    e = 4 if dtype == "f32" else 2
    st.kv, st.kv_layers, st.kv_capacity, st.kv_row_bytes = 1 << 20, 1, cap, D * e
    st.kv_request_stride, st.kv_len = 2 * cap * D * e, 1 << 20
    d.dtype = spec.SPEC_F32 if dtype == "f32" else spec.SPEC_BF16
    d.q_heads, d.kv_heads, d.head_dim, d.scale = group, 1, D, 1.0
    d.q = d.out = 1 << 20
    d.q_stride = d.out_stride = group * D
    if prefix:
        d.prefix_k = d.prefix_v = 1 << 20
        d.prefix_capacity, d.prefix_stride = prefix, D
    return spec._abi.lib().spec_prefix_attention(B, R, st, 0, d, None, None, 0, None)


@pytest.mark.parametrize("kw,over", [
    # 16-row tiles: 512 x 16 own ones, none of a prefix; one request more; a prefix, as many again
    (dict(B=512, R=8, group=32, dtype="f32", prefix=0), False),
    (dict(B=513, R=8, group=32, dtype="f32", prefix=0), True),
    (dict(B=512, R=8, group=32, dtype="f32", prefix=64), True),
    (dict(B=256, R=8, group=32, dtype="f32", prefix=64), False),
    (dict(B=257, R=8, group=32, dtype="f32", prefix=64), True),
    (dict(B=512, R=8, group=32, dtype="bf16", prefix=0, D=72), False),
    (dict(B=513, R=8, group=32, dtype="bf16", prefix=0, D=72), True),
    # the tensor cores' tiles of 128 rows: the largest call there is
    (dict(B=1024, R=8, group=64, dtype="bf16", prefix=64), False),
    # tiles by positions
    (dict(B=64, R=8, group=64, dtype="bf16", prefix=0, cap=1 << 30), True),
    (dict(B=64, R=8, group=64, dtype="bf16", prefix=0, cap=1 << 29), False),
])
def test_products_of_sizes(spec, kw, over):
    got = refusal(spec, **kw)
    assert (got == UNSUPPORTED) if over else got != UNSUPPORTED and got != 0
