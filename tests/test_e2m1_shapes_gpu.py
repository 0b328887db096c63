"""4-bit decode attention: three blocks of 16 query rows a kv head, and the fixed scratch's limit."""
import numpy as np
import pytest
import torch

from e2m1ref import Filled4
from test_e2m1_attn_gpu import _bounded, _queries, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


BLOCKS3 = [  # 33 to 48 query rows: query heads, kv heads, query tokens
    (33, 1, 1), (40, 1, 1), (48, 1, 1), (96, 2, 1), (105, 3, 1), (24, 2, 3), (160, 4, 1), (44, 4, 4), (384, 8, 1),
    (12, 1, 4), (240, 6, 1),
]


@pytest.mark.parametrize("hq,hkv,T", BLOCKS3)
@pytest.mark.parametrize("lens", [[0, 1, 2, 15, 16, 17], [31, 32, 33, 63, 64, 65], [700, 5, 0, 1033]])
def test_three_blocks_of_16_rows(kv, hq, hkv, T, lens):
    f = Filled4(kv, lens, hkv=hkv, seed=hq + T)
    q = _queries(len(lens), T, hq, 91, 0.5)
    got = _run(f, q, 0.09)
    assert f.pool.error() == 0
    for b, n in enumerate(lens):
        _bounded(f, b, got[b], q[b], 0.09)
        for i in range(min(T, max(0, T - n))):
            assert not got[b, i].any()


@pytest.mark.parametrize("hq,hkv", [(8, 1), (64, 1), (128, 4), (48, 1)])
def test_largest_batch_of_the_fixed_scratch(kv, hq, hkv):
    """The largest batch whose workspace is 32 MiB is served, the next is refused."""
    probe = Filled4(kv, [1], hkv=hkv)
    lo, hi = 1, 1 << 16  # workspaces grow with the batch
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if probe.pool.workspace_size(mid, hq, 1) <= 32 << 20 else (lo, mid)
    lens = np.random.default_rng(92).integers(1, 40, lo + 1).tolist()
    f = Filled4(kv, lens, hkv=hkv, seed=93)
    q = _queries(lo + 1, 1, hq, 94, 0.5)
    want, qd = _run(f, q, 0.09), q.cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kv.KVError) as e:
        kv.paged_decode_attn_noalloc(f.pool.handle, lo + 1, hq, 1, qd, f.table_d, f.lens_d, None, 0.09, out)
    assert e.value.status == kv.KV_ERR_UNSUPPORTED
    assert bool((out == 7.0).all())
    kv.paged_decode_attn_noalloc(f.pool.handle, lo, hq, 1, qd, f.table_d, f.lens_d, None, 0.09, out)
    got = out.cpu()
    assert f.pool.error() == 0 and bool((got[lo] == 7.0).all())
    for b in (0, 1, lo // 2, lo - 1):
        _bounded(f, b, got[b], q[b], 0.09)
        _bounded(f, b, want[b], q[b], 0.09)
