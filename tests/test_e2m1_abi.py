"""4-bit pools and normalised appends: what is refused before anything is enqueued (no GPU)."""
import math

import pytest

from test_prompt_abi import F, ROTARY, _pool


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


@pytest.mark.parametrize("over", [
    dict(layout=1, num_kv_heads=1, v_cache=None, v_scale=None), dict(page_size=32), dict(page_size=8),
    dict(head_dim_k=64), dict(head_dim_v=256), dict(scale_mode=1), dict(num_kv_heads=4097)])
def test_pool_shapes(kv, over):
    with pytest.raises(kv.KVError) as e:
        _pool(kv, dtype=kv.KV_DTYPE_E2M1, **over)
    assert e.value.status == kv.KV_ERR_UNSUPPORTED


@pytest.mark.parametrize("over", [dict(k_scale=None), dict(v_scale=None), dict(v_cache=None),
                                  dict(k_cache=F + 8), dict(dtype=3), dict(dtype=-1)])
def test_pool_refusals(kv, over):
    with pytest.raises(kv.KVError) as e:
        _pool(kv, **{"dtype": kv.KV_DTYPE_E2M1, **over})
    assert e.value.status == kv.KV_ERR_INVALID_ARG


def test_prompt_attention_needs_another_pool(kv):
    h = _pool(kv, dtype=kv.KV_DTYPE_E2M1)
    assert kv.paged_prefill_workspace_size(h, 2, 8, 10) == 0
    st = kv._lib.paged_prefill_attn(h, None, 2, 8, 10, F, F, F, 4, F, None, 0.1, F, F, 1 << 30)
    assert st == kv.KV_ERR_UNSUPPORTED
    kv.kv_pool_destroy(h)


def test_append_refusals(kv):
    h = _pool(kv, dtype=kv.KV_DTYPE_E2M1)
    ok = [h, None, 2, F, F, F, 5, F, F, 4, F]
    for i, bad in ((2, -1), (3, None), (3, F + 8), (4, None), (5, None), (6, -1), (7, None), (8, None),
                   (9, 0), (10, None)):
        a = list(ok)
        a[i] = bad
        assert kv._lib.kv_append_quantize(*a) == kv.KV_ERR_INVALID_ARG, i
    # a handoff comes from a bf16 pool of the same shape
    for over in (dict(dtype=kv.KV_DTYPE_E2M1), dict(dtype=kv.KV_DTYPE_E4M3),
                 dict(dtype=kv.KV_DTYPE_BF16, num_kv_heads=4),
                 dict(dtype=kv.KV_DTYPE_BF16, page_size=8)):
        src = _pool(kv, **over)
        assert kv._lib.kv_append_from_pool(h, None, 2, src, F, 4, F, F, F, 4, F) == kv.KV_ERR_INVALID_ARG
        kv.kv_pool_destroy(src)
    assert kv.kv_last_launch_count(h) == 0
    kv.kv_pool_destroy(h)


def _norm_args(over):
    a = {**ROTARY, **over}
    norm = {k: a.pop(k, d) for k, d in (("q_norm", F), ("k_norm", F), ("eps", 1e-6))}
    v = list(a.values())
    return [*v[:17], *norm.values(), *v[17:]]


@pytest.mark.parametrize("over", [
    dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(q_norm=F + 8), dict(k_norm=F + 2),
    dict(B=-1), dict(total=-1), dict(rot=24), dict(il=2), dict(k=None), dict(q=None), dict(pos=None),
    dict(ks=248), dict(q_out=F, q=F, qs=1032), dict(axes=0)])
def test_norm_refusals(kv, over):
    for dtype in (kv.KV_DTYPE_E4M3, kv.KV_DTYPE_BF16, kv.KV_DTYPE_E2M1):
        h = _pool(kv, dtype=dtype)
        assert kv._lib.kv_append_norm_rotary(h, None, *_norm_args(over)) == kv.KV_ERR_INVALID_ARG
        assert kv.kv_last_launch_count(h) == 0
        kv.kv_pool_destroy(h)


def test_norm_shapes(kv):
    assert kv._lib.kv_append_norm_rotary(None, None, *_norm_args({})) == kv.KV_ERR_INVALID_ARG
    for over in (dict(page_size=64), dict(page_size=16, head_dim_k=80), dict(page_size=2, head_dim_k=1024)):
        h = _pool(kv, **over)
        assert kv._lib.kv_append_norm_rotary(h, None, *_norm_args({})) == kv.KV_ERR_UNSUPPORTED
        kv.kv_pool_destroy(h)
    h = _pool(kv)
    none = dict(B=0, q=None, k=None, v=None, ind=None, table=None, tags=None, lens=None)
    assert kv._lib.kv_append_norm_rotary(h, None, *_norm_args(none)) == kv.KV_OK  # nothing to do
    kv.kv_pool_destroy(h)


def test_argument_order_of_the_binding(kv):
    names = list(ROTARY)
    assert names[:17] == ["B", "hq", "total", "q", "qs", "k", "ks", "v", "vs", "ind", "max_new", "pos",
                          "axes", "axis", "freq", "rot", "il"]
    plain, norm = kv._lib.kv_append_rotary.argtypes, kv._lib.kv_append_norm_rotary.argtypes
    assert list(norm) == [*plain[:19], *norm[19:22], *plain[19:]]


def test_layout_places_every_code_and_scale_once():
    from e2m1ref import PLACES

    for which in "kv":
        byte, high, scale = PLACES[which]
        nibbles = (2 * byte + high).ravel().tolist()
        assert sorted(nibbles) == list(range(2048))
        assert sorted(scale.ravel().tolist()) == list(range(1024, 1152))


def test_reference_against_hand_worked_rows():
    import numpy as np

    from e2m1ref import block_scale, quantise, values, write

    assert block_scale(6.0) == 2.0 ** -4 and block_scale(8.0) == 2.0 ** -3 and block_scale(0.0) == 1.0
    assert block_scale(1e-40) == 2.0 ** -100 and block_scale(3e38) == 2.0 ** 121
    # amax 6 over S = 1/16: s = 16, so a code of 1 is 1
    x = np.zeros((1, 128), np.float32)
    x[0, :16] = [6, -6, 5, 5.01, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -0.25, 0.5, 1, -1.5, 0]
    code, sc, _ = quantise(x, block_scale(6.0))
    assert sc[0].tolist() == [0x58] + [0] * 7
    assert code[0, :16].tolist() == [7, 15, 6, 7, 6, 4, 4, 2, 2, 0, 1, 8, 1, 2, 11, 0]
    for which in "kv":
        tile = np.zeros(1152, np.uint8)
        write(tile, which, 5, code[0], sc[0])
        got = values(tile, np.float32(2.0 ** -4), which)
        assert got[5, :16].tolist() == [6, -6, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, 0, 0.5, 1, -1.5, 0]
        assert not got[[s for s in range(16) if s != 5]].any()
