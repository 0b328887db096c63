"""Decode attention's refusals of an output that its 8-byte stores cannot reach (no GPU)."""
import pytest

from test_prompt_abi import F, _pool


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


@pytest.mark.parametrize("out", [None, F + 2, F + 4, F + 6])
@pytest.mark.parametrize("dtype", ["KV_DTYPE_E4M3", "KV_DTYPE_BF16", "KV_DTYPE_E2M1"])
def test_output_alignment(kv, dtype, out):
    h = _pool(kv, dtype=getattr(kv, dtype))
    lib, big = kv._lib, 1 << 40
    calls = dict(
        attn=lib.paged_decode_attn(h, None, 2, 8, 1, F, F, 4, F, None, 0.1, out, F, big),
        checked=lib.paged_decode_attn_checked(h, None, 2, 8, 1, F, F, F, 4, F, 0.1, out, F, F, big),
        combine=lib.paged_decode_attn_combine(h, None, 2, 8, 1, None, out, F, big),
        step=lib.kv_decode_step(h, None, 2, 8, 1, None, F, F, F, 1, F, F, 4, F, F, 0.1, out, F, 0, F, big))
    assert calls == dict.fromkeys(calls, kv.KV_ERR_INVALID_ARG)
    assert kv.kv_last_launch_count(h) == 0
    kv.kv_pool_destroy(h)
