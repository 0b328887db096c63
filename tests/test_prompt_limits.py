"""Batches whose work items would not be counted in an int are refused before anything is
enqueued: the append's plan would pop pages for rows that no kernel could write."""
import pytest

from test_prompt_abi import PREFILL, READ, ROTARY, _pool, kv  # noqa: F401  (kv: the fixture)

SMALL = dict(page_size=1, head_dim_k=16, head_dim_v=16)


@pytest.mark.parametrize("B,total,page", [
    (1 << 30, 100, 16), (2, 2 ** 31 - 1, 1), ((1 << 30) - 4, 256, 16), (1 << 29, 1 << 30, 1)])
def test_items_of_rows(kv, B, total, page):  # noqa: F811
    h = _pool(kv, **(SMALL if page == 1 else {}))
    try:
        a = {**ROTARY, **dict(B=B, total=total, hq=0, q=None, q_out=None, rot=16)}
        assert kv._lib.kv_append_rotary(h, None, *a.values()) == kv.KV_ERR_UNSUPPORTED
        a = {**READ, **dict(B=B, total=total)}
        assert kv._lib.kv_read_rows(h, None, *a.values()) == kv.KV_ERR_UNSUPPORTED
        assert kv.kv_last_launch_count(h) == 0
    finally:
        kv.kv_pool_destroy(h)


def test_items_of_queries(kv):  # noqa: F811
    h = _pool(kv)
    try:
        B = 2 ** 31 - 1
        a = {**PREFILL, **dict(B=B, hq=64, total=(1 << 25) - 1)}
        assert kv._lib.paged_prefill_attn(h, None, *a.values()) == kv.KV_ERR_UNSUPPORTED
        assert kv._lib.paged_prefill_workspace_size(h, B, 64, (1 << 25) - 1) == 0
        assert kv.kv_last_launch_count(h) == 0
    finally:
        kv.kv_pool_destroy(h)
