"""kv_append_rotary, kv_read_rows and paged_prefill_attn refuse bad arguments
before enqueuing anything (no GPU needed), and so do their Python calls."""
import pytest
import torch


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


F = 0x10000  # an aligned address that nothing dereferences


def _pool(kv, **over):
    d = kv.kv_pool_desc()
    d.num_pages, d.page_size, d.num_kv_heads, d.head_dim_k, d.head_dim_v = 64, 16, 2, 128, 128
    d.dtype, d.layout = kv.KV_DTYPE_E4M3, kv.KV_LAYOUT_GQA
    d.k_cache = d.v_cache = d.k_scale = d.v_scale = d.tags = d.free_list = d.ctl = F
    for k, v in over.items():
        setattr(d, k, v)
    return kv.kv_pool_create(d)


LATENT = dict(layout=1, num_kv_heads=1, head_dim_k=576, head_dim_v=512, page_size=64,
              v_cache=None, v_scale=None)

ROTARY = dict(B=2, hq=8, total=10, q=F, qs=1024, k=F, ks=256, v=F, vs=256, ind=F, max_new=5, pos=F,
              axes=3, axis=F, freq=F, rot=128, il=0, q_out=F + 4096, table=F, tags=F, width=4, lens=F)


@pytest.mark.parametrize("over", [
    dict(B=-1), dict(hq=-1), dict(total=-1), dict(max_new=-1), dict(width=0), dict(axes=0),
    dict(axes=257), dict(rot=0), dict(rot=24), dict(rot=144), dict(il=2), dict(k=None),
    dict(v=None), dict(ind=None), dict(pos=None), dict(axis=None), dict(freq=None), dict(table=None),
    dict(tags=None), dict(lens=None), dict(q=None), dict(q_out=None), dict(q=F + 8),
    dict(k=F + 2), dict(v=F + 4), dict(q_out=F + 8), dict(qs=1016), dict(qs=1028), dict(ks=248),
    dict(vs=260), dict(q_out=F, q=F, qs=1032)])
def test_rotary_refusals(kv, over):
    h = _pool(kv)
    try:
        a = {**ROTARY, **over}
        assert kv._lib.kv_append_rotary(h, None, *a.values()) == kv.KV_ERR_INVALID_ARG
        assert kv.kv_last_launch_count(h) == 0
    finally:
        kv.kv_pool_destroy(h)


def test_rotary_shapes(kv):
    assert kv._lib.kv_append_rotary(None, None, *ROTARY.values()) == kv.KV_ERR_INVALID_ARG
    for over in (LATENT, dict(page_size=64)):  # rows of one tensor; a page of 64 x 128
        h = _pool(kv, **over)
        assert kv._lib.kv_append_rotary(h, None, *ROTARY.values()) == kv.KV_ERR_UNSUPPORTED
        kv.kv_pool_destroy(h)
    h = _pool(kv)
    none = {**ROTARY, **dict(B=0, q=None, k=None, v=None, ind=None, table=None, tags=None, lens=None)}
    assert kv._lib.kv_append_rotary(h, None, *none.values()) == kv.KV_OK  # nothing to do
    kv.kv_pool_destroy(h)


READ = dict(B=2, table=F, width=4, lens=F, start=None, ind=F, total=10, mask=None, k=F, v=F)


@pytest.mark.parametrize("over", [
    dict(B=-1), dict(total=-1), dict(width=0), dict(table=None), dict(lens=None), dict(ind=None),
    dict(k=None), dict(v=None), dict(k=F + 8), dict(v=F + 2)])
def test_read_refusals(kv, over):
    h = _pool(kv)
    try:
        a = {**READ, **over}
        assert kv._lib.kv_read_rows(h, None, *a.values()) == kv.KV_ERR_INVALID_ARG
        assert kv._lib.kv_read_rows(None, None, *READ.values()) == kv.KV_ERR_INVALID_ARG
        for nothing in (dict(B=0), dict(total=0)):
            a = {**READ, **dict(table=None, lens=None, ind=None, k=None, v=None), **nothing}
            assert kv._lib.kv_read_rows(h, None, *a.values()) == kv.KV_OK
        assert kv.kv_last_launch_count(h) == 0
    finally:
        kv.kv_pool_destroy(h)


PREFILL = dict(B=2, hq=8, total=10, q=F, ind=F, table=F, width=4, lens=F, mask=None, scale=0.1, out=F,
               ws=F, size=1 << 40)


@pytest.mark.parametrize("over", [
    dict(B=-1), dict(hq=0), dict(hq=7), dict(total=-1), dict(q=None), dict(ind=None),
    dict(table=None), dict(width=0), dict(lens=None), dict(out=None), dict(q=F + 8), dict(out=F + 2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(ws=None),
    dict(ws=F + 128)])
def test_prefill_refusals(kv, over):
    h = _pool(kv)
    try:
        a = {**PREFILL, **over}
        assert kv._lib.paged_prefill_attn(h, None, *a.values()) == kv.KV_ERR_INVALID_ARG
        for nothing in (dict(B=0), dict(total=0)):
            a = {**PREFILL, **dict(q=None, ind=None, out=None, ws=None, size=0), **nothing}
            assert kv._lib.paged_prefill_attn(h, None, *a.values()) == kv.KV_OK
        assert kv.kv_last_launch_count(h) == 0
    finally:
        kv.kv_pool_destroy(h)


@pytest.mark.parametrize("shape", [LATENT, dict(head_dim_k=64), dict(head_dim_v=256),
                                   dict(page_size=32), dict(num_kv_heads=4100)])
def test_prefill_shapes(kv, shape):
    h = _pool(kv, **shape)
    a = {**PREFILL, **dict(hq=4100)}
    assert kv._lib.paged_prefill_attn(h, None, *a.values()) == kv.KV_ERR_UNSUPPORTED
    assert kv._lib.paged_prefill_workspace_size(h, 2, 4100, 10) == 0
    kv.kv_pool_destroy(h)


def test_prefill_rows_are_counted_in_an_int(kv):
    h = _pool(kv)
    a = {**PREFILL, **dict(hq=64, total=1 << 25)}
    assert kv._lib.paged_prefill_attn(h, None, *a.values()) == kv.KV_ERR_UNSUPPORTED
    kv.kv_pool_destroy(h)


class Recorder:
    """Stands for the library: no call may come through a refusal."""

    def __getattr__(self, name):
        def called(*args):
            raise AssertionError(f"{name} called")

        return called


def test_python_calls_refuse_tensors(kv, monkeypatch):
    """Host tensors, other types and shapes are refused before the library is called.  With the
    current device's number set to that of host tensors (-1), the checks behind it are reached."""
    monkeypatch.setattr(kv, "_lib", Recorder())
    bf = torch.bfloat16
    q, k, v = torch.zeros(6, 8, 128, dtype=bf), torch.zeros(6, 2, 128, dtype=bf), torch.zeros(6, 2, 128, dtype=bf)
    ind, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    table, tags = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    pos, axis = torch.zeros(3, 6, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    freq, ws = torch.zeros(64, dtype=torch.float64), torch.zeros(256, dtype=torch.uint8)

    def rotary(**o):
        a = {**dict(B=2, hq=8, q=q, k=k, v=v, ind=ind, max_new=5, pos=pos, axis=axis, freq=freq, il=False,
                    q_out=q.clone(), table=table, tags=tags, lens=lens, stream=0), **o}
        kv.kv_append_rotary(0, *a.values())

    def read(**o):
        a = {**dict(B=2, table=table, lens=lens, start=None, ind=ind, mask=None, k=k, v=v, stream=0), **o}
        kv.kv_read_rows(0, *a.values())

    def prefill(**o):
        a = {**dict(B=2, hq=8, q=q, ind=ind, table=table, lens=lens, mask=None, scale=0.1, out=q.clone(),
                    ws=ws, stream=0), **o}
        kv.paged_prefill_attn(0, *a.values())

    monkeypatch.setattr(kv, "_device", lambda: 0)
    for call in (rotary, read, prefill):
        with pytest.raises(ValueError):
            call()
    monkeypatch.setattr(kv, "_device", lambda: -1)
    monkeypatch.setattr(kv, "_ptr", lambda t, dtype=None, name="": 0)
    for call in (rotary, read, prefill):
        with pytest.raises(AssertionError, match="called"):
            call()
    real = pytest.raises((ValueError, TypeError))
    bad = [(rotary, dict(q=q[:, :7])), (rotary, dict(q=q.transpose(0, 1))), (rotary, dict(k=k[:5])),
           (rotary, dict(k=k.float())), (rotary, dict(v=v[:, :, ::2])), (rotary, dict(ind=ind[:2])),
           (rotary, dict(pos=pos[:, :5])), (rotary, dict(axis=axis[:63])), (rotary, dict(table=table[:1])),
           (rotary, dict(tags=tags[:1])), (rotary, dict(lens=lens[:1])), (rotary, dict(q_out=q[:5].clone())),
           (rotary, dict(q=None)),
           (read, dict(ind=ind[:2])), (read, dict(lens=lens[:1])), (read, dict(table=table[:1])),
           (read, dict(v=v[:5])), (read, dict(start=lens[:1])), (read, dict(mask=axis[:1])),
           (prefill, dict(out=q[:5])), (prefill, dict(ind=ind[:2])), (prefill, dict(lens=lens[:1])),
           (prefill, dict(q=q[:, :4], out=q[:, :4])), (prefill, dict(mask=axis[:1]))]
    for call, o in bad:
        with real:
            call(**o)
    # queries turned in place must be contiguous
    wide = torch.zeros(6, 9, 128, dtype=bf)
    with pytest.raises(ValueError):
        rotary(q=wide[:, :8], q_out=wide[:, :8])
