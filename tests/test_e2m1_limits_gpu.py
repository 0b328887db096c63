"""4-bit decode attention at the ends of its ranges: lengths next to 2^31."""
import numpy as np
import pytest
import torch

from e2m1ref import values
from test_e2m1_attn_gpu import _queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


@pytest.mark.parametrize("hq,n", [(8, 2 ** 31 - 1), (8, 2 ** 31 - 130), (16, 2 ** 31 - 1)])
def test_lengths_next_to_2_to_31(kv, hq, n):
    """A page table of 2^27 entries over 64 pages, each mapped many times.

    Bound: that of test_e2m1_attn_gpu, and the sums: a warp adds up to 2^16 pages one by one, in
    fp32 for the weights (2^-24 of the sum each) and in the matrix unit for the values (taken as
    2^-22 each): 2^-8 + 2^-6 of A beside its 2^-10."""
    P, pages, width = 16, 64, 2 ** 27
    rng = np.random.default_rng(81)
    tiles, scales = {}, {}
    for which in "kv":
        tiles[which] = rng.integers(0, 256, (pages, 1, 1152), dtype=np.uint8)
        tiles[which][..., 1024:] = rng.integers(0x20, 0x40, (pages, 1, 128))
        scales[which] = np.full((pages, 1), 0.25, np.float32)
    ids = torch.arange(width, dtype=torch.int32, device="cuda").remainder_(pages)
    pool = kv.KVPool(pages, P, 1, 128, 128, dtype=kv.KV_DTYPE_E2M1,
                     k_cache=torch.from_numpy(tiles["k"]).cuda(), v_cache=torch.from_numpy(tiles["v"]).cuda(),
                     k_scale=torch.from_numpy(scales["k"]).cuda(), v_scale=torch.from_numpy(scales["v"]).cuda())
    q = _queries(1, 1, hq, 82, 0.5)
    out = torch.full((1, 1, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pool.workspace_size(1, hq, 1), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    pool.attn(1, hq, 1, q.cuda(), ids.view(1, width), lens, None, 0.09, out, ws)
    assert pool.error() == 0
    # how often each (page, slot) is seen
    whole, rest = divmod(n, P)
    count = np.full((pages, P), whole // pages, np.float64)
    count[:whole % pages] += 1
    count[whole % pages, :rest] += 1
    k, v = (torch.from_numpy(values(tiles[w], scales[w], w)[:, 0].reshape(-1, 128)) for w in "kv")
    s = q[0, 0].double() @ k.t() * 0.09
    w = torch.exp(s - s.amax(-1, keepdim=True)) * torch.from_numpy(count.reshape(-1))
    w /= w.sum(-1, keepdim=True)
    ref, mag = w @ v, w @ v.abs()
    err = (out[0, 0].cpu().double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -8 + 2.0 ** -6) * mag).all())
