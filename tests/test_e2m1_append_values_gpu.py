"""A 4-bit page's block scale is of the groups whose 16 values are all finite: a group with a value
that is not leaves its finite values out too."""
import pytest
import torch

from e2m1ref import block_scale
from test_e2m1_append_gpu import Pair, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _bad_rows(n, hkv):
    """Rows whose largest finite value, 1000, lies in a group with a NaN or an infinity."""
    g = torch.Generator().manual_seed(n)
    x = _rows(g, n, hkv)
    x[n // 2, :, 80] = 1000.0
    x[n // 2, :, 95] = float("nan")
    x[0, -1, 80] = -1000.0
    x[0, -1, 81] = float("inf")
    return x


def _amax(x):
    """Of each head, over groups that are finite."""
    y = x.float().unflatten(-1, (8, 16))
    return torch.where(torch.isfinite(y).all(-1), y.abs().amax(-1), 0.0).amax((0, 2)).tolist()


@pytest.mark.parametrize("hkv", [1, 2])
@pytest.mark.parametrize("n", [1, 7, 16, 40])  # 40: the kernel of many rows
def test_append(kv, hkv, n):
    p = Pair(kv, 2, hkv, 16, 6, seed=n)
    k, v = _bad_rows(n, hkv), _bad_rows(n, hkv)
    p.append([n, 0], k, v)
    p.check()
    first = int(p.table[0, 0])
    want = [float(block_scale(a)) for a in _amax(k[:16])]
    assert p.pool.k_scale[first].tolist() == want
    assert max(want) < float(block_scale(1000.0))
    p.append([0, n], v, k)  # another page
    p.check()


@pytest.mark.parametrize("n", [7, 16, 40])
def test_handoff(kv, n):
    hkv, pages = 2, 8
    k, v = _bad_rows(n, hkv), _bad_rows(n, hkv)
    need = -(-n // 16)
    src = kv.KVPool(pages, 16, hkv, 128, 128, dtype=kv.KV_DTYPE_BF16)
    for j in range(need):
        m = min(16, n - 16 * j)
        src.k_cache[j, :, :m] = k[16 * j:16 * j + m].transpose(0, 1).cuda()
        src.v_cache[j, :, :, :m] = v[16 * j:16 * j + m].permute(1, 2, 0).cuda()
    p = Pair(kv, 1, hkv, pages, 4, seed=n)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    p.pool.append_from_pool(1, src, table, torch.tensor([n], dtype=torch.int32, device="cuda"), p.table, p.exp, p.lens)
    p.ref.append(k.float().numpy(), v.float().numpy(), [n])
    p.check()


@pytest.mark.parametrize("n", [1, 16, 20])
def test_rotary(kv, n):
    """The first 16 dims turn by nothing, the others pass through."""
    hkv = 2
    p = Pair(kv, 1, hkv, 8, 4, seed=n)
    k, v = _bad_rows(n, hkv), _bad_rows(n, hkv)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p.pool.append_rotary(1, 0, None, k.cuda(), v.cuda(), i32([0, n]), n, torch.zeros((1, n), dtype=torch.int32, device="cuda"),
                         torch.zeros(8, dtype=torch.uint8, device="cuda"),
                         torch.ones(8, dtype=torch.float64, device="cuda"), True, None, p.table, p.exp, p.lens)
    p.ref.append(k.float().numpy(), v.float().numpy(), [n])
    p.check()
