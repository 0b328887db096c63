"""Appends into 4-bit pools against the definition, bit for bit: codes, group and block
scales, page tables, tags and lengths, and every byte that no row owns."""
import numpy as np
import pytest
import torch

from e2m1ref import TILE, Model, block_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


class Pair:
    """A pool on the device and its host twin, from the same junk."""

    def __init__(self, kv, B, hkv, pages, width, seed=0):
        rng = np.random.default_rng(seed)
        free = rng.permutation(pages).astype(np.int32)
        tags = rng.integers(0, 2 ** 32, pages, dtype=np.uint32)
        ck, cv = (rng.integers(0, 256, (pages, hkv, TILE), dtype=np.uint8) for _ in range(2))
        ks, vs = (rng.random((pages, hkv), dtype=np.float32) for _ in range(2))
        self.kv, self.B, self.hkv = kv, B, hkv
        self.ref = Model(pages, hkv, free, tags, ck, cv, ks, vs, width, B)
        cu = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.pool = kv.KVPool(pages, 16, hkv, 128, 128, dtype=kv.KV_DTYPE_E2M1, tags=tags, free_list=free,
                              k_cache=cu(ck), v_cache=cu(cv), k_scale=cu(ks), v_scale=cu(vs))
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.exp = torch.zeros((B, width), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def append(self, counts, k, v, max_new=None, stream=None):
        """k, v: bf16 [rows][hkv][128] on the host."""
        ind = np.zeros(self.B + 1, np.int32)
        ind[1:] = np.cumsum(counts)
        pad = torch.zeros((max(0, 1 - k.shape[0]), self.hkv, 128), dtype=torch.bfloat16)
        self.pool.append(self.B, torch.cat([k, pad]).cuda(), torch.cat([v, pad]).cuda(),
                         torch.from_numpy(ind).cuda(), max(counts) if max_new is None else max_new,
                         self.table, self.exp, self.lens, stream)
        self.ref.append(k.float().numpy(), v.float().numpy(), counts)

    def check(self, error=0):
        r = self.ref
        assert self.pool.error() == error
        assert np.array_equal(self.lens.cpu().numpy(), r.lens)
        assert np.array_equal(self.table.cpu().numpy(), r.table)
        assert np.array_equal(self.exp.cpu().numpy().view(np.uint32), r.exp)
        assert np.array_equal(self.pool.tags.cpu().numpy().view(np.uint32), r.tags)
        assert int(self.pool.ctl[0]) == r.head
        for which in "kv":
            got = getattr(self.pool, which + "_scale").cpu().numpy()
            assert np.array_equal(got.view(np.uint32), r.scale[which].view(np.uint32)), which
            c = getattr(self.pool, which + "_cache").cpu().numpy()
            same = (c == r.cache[which]) | r.loose[which]
            assert same.all(), (which, np.argwhere(~same)[:5])


def _rows(g, n, hkv, mag=1.0):
    spread = torch.empty((1, hkv, 128)).uniform_(0.5, 4.0, generator=g) * mag
    return (torch.randn((n, hkv, 128), generator=g) * spread).to(torch.bfloat16)


@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("steps", [
    [[1, 1, 1, 1], [1, 1, 1, 1], [1, 0, 1, 1]],               # decode steps
    [[0, 1, 15, 16], [17, 16, 1, 16], [1, 15, 33, 0]],        # page borders, parts of pages
    [[40, 0, 100, 7], [3, 64, 0, 31], [90, 5, 48, 1]],        # the bulk kernel: whole and partly filled pages
    [[37, 37, 37, 37], [1, 2, 3, 4], [200, 0, 0, 0]],
])
def test_append_bit_for_bit(kv, hkv, steps):
    g = torch.Generator().manual_seed(hkv)
    p = Pair(kv, 4, hkv, 64, 24, seed=hkv)
    for counts in steps:
        n = sum(counts)
        p.append(counts, _rows(g, n, hkv), _rows(g, n, hkv))
        p.check()


@pytest.mark.parametrize("mag", [1e-4, 3e3, 1e30, 2.0 ** -90, 2.0 ** -120, 3e38])
def test_magnitudes(kv, mag):
    g = torch.Generator().manual_seed(1)
    p = Pair(kv, 2, 2, 16, 8)
    k, v = _rows(g, 41, 2, mag / 16), _rows(g, 41, 2, mag / 16)
    p.append([24, 17], k, v)
    p.check()
    p.append([9, 40], _rows(g, 49, 2, mag / 16), _rows(g, 49, 2, mag / 16))
    p.check()


def test_blocks_of_zeros_and_frozen_scales(kv):
    """A page of zeros takes a scale of 1; rows far above or below a page's first ones
    saturate or lose their group scale."""
    g = torch.Generator().manual_seed(2)
    p = Pair(kv, 3, 2, 16, 8)
    z = torch.zeros((15, 2, 128), dtype=torch.bfloat16)
    p.append([5, 5, 5], z, -z)
    p.check()
    assert float(p.pool.k_scale[int(p.table[0, 0]), 0]) == 1.0
    p.append([4, 4, 4], _rows(g, 12, 2, 1000.0), _rows(g, 12, 2, 1e-6))
    p.check()
    p.append([20, 20, 20], _rows(g, 60, 2), _rows(g, 60, 2))
    p.append([9, 9, 9], _rows(g, 27, 2, 1e6), _rows(g, 27, 2, 1e-6))
    p.check()


@pytest.mark.parametrize("bulk", [False, True])
def test_every_group_scale_and_tie(kv, bulk):
    """Rows whose groups take every e4m3 scale that a page can hold, with values on and
    beside every border between two codes."""
    import e2m1ref

    first = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    first[..., :16] = 6.0  # block scale 2^-4: a scale s stands for 6 s / 16
    scales = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    rows = []
    for s in scales.tolist():
        x = torch.zeros(128)
        top = 6.0 * s / 16
        borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s / 16
        x[0:16] = top
        b = borders.to(torch.bfloat16)
        up, down = ((b.view(torch.int16) + o).view(torch.bfloat16).float() for o in (1, -1))
        for i, part in enumerate((borders, up, down, -borders, -up, -down)):
            x[16 + 16 * i] = top
            x[17 + 16 * i:17 + 16 * i + 7] = part
        rows.append(x)
    k = torch.cat([first, torch.stack(rows)[:, None].to(torch.bfloat16)])
    p = Pair(kv, 1, 1, 16, 10)
    p.append([1], k[:1], k[:1])
    n = k.shape[0] - 1
    for lo in range(0, n, 15):  # every page begins with the row that sets its scale
        part = torch.cat([k[1 + lo:1 + min(n, lo + 15)], first])
        p.append([part.shape[0]], part, part, max_new=64 if bulk else part.shape[0])
    p.check()
    seen = {int(x) for x in p.ref.cache["k"][p.ref.table[0, :8]][:, 0][:, e2m1ref.PLACES["k"][2]].ravel()}
    assert len(seen) >= 100


@pytest.mark.parametrize("counts", [[3, 20], [40, 64]])
def test_values_that_are_not_finite(kv, counts):
    """A group with one gets a scale of NaN; the other groups and the page's scale are
    those of the finite ones."""
    g = torch.Generator().manual_seed(3)
    n = sum(counts)
    k, v = _rows(g, n, 2), _rows(g, n, 2)
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"))):
        k[i, 0, 16 * i + 5] = x
        v[n - 1 - i, 1, 16 * i + 2] = x
    k[2, 1] = float("nan")
    p = Pair(kv, 2, 2, 16, 8)
    p.append(counts, k, v)
    p.check()
    out = [torch.empty((n, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ind = torch.tensor([0, counts[0], n], dtype=torch.int32, device="cuda")
    p.pool.read_rows(2, p.table, p.lens, None, ind, None, *out)
    for got, x in zip(out, (k, v)):
        bad = ~torch.isfinite(x.view(n, 2, 8, 16)).all(-1)
        assert torch.equal(torch.isnan(got.cpu().view(n, 2, 8, 16)).all(-1), bad)
        assert bool(torch.isfinite(got.cpu().view(n, 2, 8, 16)[~bad]).all())


def _source(kv, lens, hkv, g):
    """A bf16 pool that holds rows of these lengths, its table, and the rows."""
    need = [-(-n // 16) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(need + [1]) + 2), -1, dtype=torch.int32)
    k = torch.full((pages, hkv, 16, 128), float("nan"), dtype=torch.bfloat16)
    v = torch.full((pages, hkv, 128, 16), float("nan"), dtype=torch.bfloat16)
    rk, rv = _rows(g, sum(lens), hkv), _rows(g, sum(lens), hkv)
    at = row = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = ids[at]
            m = min(16, n - 16 * j)
            k[ids[at], :, :m] = rk[row:row + m].transpose(0, 1)
            v[ids[at], :, :, :m] = rv[row:row + m].permute(1, 2, 0)
            at, row = at + 1, row + m
    src = kv.KVPool(pages, 16, hkv, 128, 128, dtype=kv.KV_DTYPE_BF16, k_cache=k.cuda(), v_cache=v.cuda())
    return src, table, rk, rv


@pytest.mark.parametrize("hkv", [1, 2, 5])
@pytest.mark.parametrize("lens", [[0, 1, 16, 17], [100, 0, 31, 333], [1]])
def test_handoff_is_the_append_of_its_rows(kv, hkv, lens):
    g = torch.Generator().manual_seed(hkv)
    src, table, rk, rv = _source(kv, lens, hkv, g)
    p = Pair(kv, len(lens), hkv, 48, 24, seed=5)
    p.pool.append_from_pool(len(lens), src, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            p.table, p.exp, p.lens)
    p.ref.append(rk.float().numpy(), rv.float().numpy(), lens)
    p.check()
    # the pool goes on as after any append
    n = [3] * len(lens)
    p.append(n, _rows(g, sum(n), hkv), _rows(g, sum(n), hkv))
    p.check()


def test_handoff_stops(kv):
    """Out of pages, a request that is not empty, and a source page out of range."""
    g = torch.Generator().manual_seed(0)
    lens = [20, 40, 30]
    src, table, rk, rv = _source(kv, lens, 2, g)
    l = torch.tensor(lens, dtype=torch.int32).cuda()
    p = Pair(kv, 3, 2, 4, 8)  # the second request does not fit
    p.pool.append_from_pool(3, src, table.cuda(), l, p.table, p.exp, p.lens)
    p.ref.append(rk[:20].float().numpy(), rv[:20].float().numpy(), [20, 0, 0])
    p.check(error=kv.KV_ERR_OUT_OF_PAGES)
    assert int(p.pool.ctl[2]) == 1
    p = Pair(kv, 3, 2, 16, 8)
    p.append([0, 5, 0], _rows(g, 5, 2), _rows(g, 5, 2))
    p.pool.append_from_pool(3, src, table.cuda(), l, p.table, p.exp, p.lens)
    p.ref.append(rk[:20].float().numpy(), rv[:20].float().numpy(), [20, 0, 0])
    p.check(error=kv.KV_ERR_INVALID_ARG)
    bad = table.clone()
    bad[1, 1] = 10 ** 6
    p = Pair(kv, 3, 2, 16, 8)
    p.pool.append_from_pool(3, src, bad.cuda(), l, p.table, p.exp, p.lens)
    before = {w: p.ref.cache[w].copy() for w in "kv"}, {w: p.ref.scale[w].copy() for w in "kv"}
    p.ref.append(rk.float().numpy(), rv.float().numpy(), lens)
    lost = p.ref.table[1, 1]  # mapped, but no row of it is written
    for w in "kv":
        p.ref.cache[w][lost], p.ref.scale[w][lost] = before[0][w][lost], before[1][w][lost]
    p.check(error=kv.KV_ERR_BAD_PAGE_ID)


def test_append_stops(kv):
    g = torch.Generator().manual_seed(0)
    for counts, width, pages, max_new, served, error in (
            ([20, 33, 1], 8, 4, 33, 1, kv.KV_ERR_OUT_OF_PAGES),
            ([20, 40, 1], 2, 16, 40, 1, kv.KV_ERR_INVALID_ARG),   # beyond the page table
            ([5, 9, 1], 8, 16, 8, 1, kv.KV_ERR_INVALID_ARG)):     # above max_new
        p = Pair(kv, 3, 2, pages, width)
        n = sum(counts)
        k, v = _rows(g, n, 2), _rows(g, n, 2)
        ind = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32).cuda()
        p.pool.append(3, k.cuda(), v.cuda(), ind, max_new, p.table, p.exp, p.lens)
        cut = sum(counts[:served])
        p.ref.append(k[:cut].float().numpy(), v[:cut].float().numpy(), counts[:served] + [0] * (3 - served))
        p.check(error=error)
        assert int(p.pool.ctl[2]) == served


def test_partly_filled_page_with_a_stale_tag(kv):
    g = torch.Generator().manual_seed(0)
    p = Pair(kv, 2, 2, 16, 8)
    p.append([5, 5], _rows(g, 10, 2), _rows(g, 10, 2))
    p.exp[1, 0] -= 1
    p.ref.exp[1, 0] -= np.uint32(1)
    k, v = _rows(g, 80, 2), _rows(g, 80, 2)
    ind = torch.tensor([0, 40, 80], dtype=torch.int32).cuda()
    p.pool.append(2, k.cuda(), v.cuda(), ind, 40, p.table, p.exp, p.lens)
    p.ref.append(k[:40].float().numpy(), v[:40].float().numpy(), [40, 0])
    p.check(error=kv.KV_ERR_TAG_MISMATCH)


def test_rows_and_bulk_kernels_agree_beyond_the_bulk_kernels_batch(kv):
    """More requests than the bulk kernel's table of items holds take the other one."""
    B = 16500
    g = torch.Generator().manual_seed(0)
    counts = [0] * B
    counts[0], counts[7], counts[B - 1] = 40, 33, 50
    k, v = _rows(g, 123, 1), _rows(g, 123, 1)
    p = Pair(kv, B, 1, 16, 4)
    p.append(counts, k, v)
    p.check()


def test_captured_and_replayed_on_another_stream(kv):
    g = torch.Generator().manual_seed(0)
    p = Pair(kv, 3, 2, 64, 16)
    k, v = _rows(g, 3 * 33, 2), _rows(g, 3 * 33, 2)
    kd, vd = k.cuda(), v.cuda()
    ind = torch.tensor([0, 33, 66, 99], dtype=torch.int32).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.pool.append(3, kd, vd, ind, 33, p.table, p.exp, p.lens, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.pool.append(3, kd, vd, ind, 33, p.table, p.exp, p.lens, stream=torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        p.ref.append(k.float().numpy(), v.float().numpy(), [33, 33, 33])
    p.check()


@pytest.mark.parametrize("hkv", [2, 7])
@pytest.mark.parametrize("lens", [[1, 15, 16, 17, 33, 100], [700]])
def test_rows_read_back_are_exact(kv, hkv, lens):
    """bf16(code * s * S): six significant bits, so the rows are the cache's values."""
    from e2m1ref import Filled4

    f = Filled4(kv, lens, hkv=hkv, seed=hkv)
    rng = np.random.default_rng(1)
    for windows in (False, True):
        start = [int(rng.integers(0, n)) if windows else 0 for n in lens]
        count = [int(rng.integers(1, n - s + 1)) if windows else n for n, s in zip(lens, start)]
        ind = torch.tensor([0, *np.cumsum(count)], dtype=torch.int32).cuda()
        out = [torch.full((sum(count) + 2, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        f.pool.read_rows(f.B, f.table_d, f.lens_d, torch.tensor(start, dtype=torch.int32).cuda() if windows
                         else None, ind, None, *out)
        assert f.pool.error() == 0
        for which, got in zip("kv", out):
            want = torch.cat([f.rows(b, which)[s:s + n] for b, (s, n) in enumerate(zip(start, count))])
            assert torch.equal(got[:-2].cpu().double(), want)
            assert bool((got[-2:] == 7.0).all())


def test_rows_read_back_refusals(kv):
    from e2m1ref import Filled4

    f = Filled4(kv, [40, 40, 40])
    f.table_d[1, 1] = 10 ** 6
    out = [torch.full((120, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ind = torch.tensor([0, 40, 80, 120], dtype=torch.int32).cuda()
    mask = torch.tensor([0, 0, 1], dtype=torch.uint8).cuda()
    f.pool.read_rows(3, f.table_d, f.lens_d, None, ind, mask, *out)
    assert f.pool.error() == kv.KV_ERR_BAD_PAGE_ID
    for which, got in zip("kv", out):
        got = got.cpu().double()
        assert torch.equal(got[:40], f.rows(0, which))
        assert torch.equal(got[40:56], f.rows(1, which)[:16]) and torch.equal(got[72:80], f.rows(1, which)[32:])
        assert bool((got[56:72] == 7.0).all()) and bool((got[80:] == 7.0).all())


def test_block_scale_keeps_codes_away_from_e4m3s_borders():
    """The largest group of a page's first rows has a scale in [10.6, 21.4)."""
    for amax in np.random.default_rng(0).uniform(1e-3, 1e3, 2000).astype(np.float32):
        assert 10.6 <= amax / (6 * block_scale(amax)) < 21.4
