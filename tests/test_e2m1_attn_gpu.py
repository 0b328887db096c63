"""Decode attention over 4-bit pools against the 64-bit form of the same cache.

Bound: an output is rounded to bf16 once (2^-8 of it).  With A the weighted mean of |v|:
weights are rounded to f16 (2^-11 of each; a weight below 2^-20 of its row's largest by
2^-31 of that, as many as 2^12 of them here), codes times group scales and the narrowed
queries are exact, and a score is a sum of fp32 products that is off by at most 2^-21 of
the sum of its terms' magnitudes, which these inputs keep below 2^9: 2^-12 of a weight.
2^-11 + 2^-12 + 2^-19 < 2^-10 of A."""
import numpy as np
import pytest
import torch

from e2m1ref import PLACES, Filled4
from promptref import attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _queries(B, T, hq, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, T, hq, 128), generator=g) * std).to(torch.bfloat16)


def _run(f, q, scale, mask=None, **kw):
    B, T, hq, _ = q.shape
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(f.pool.workspace_size(B, hq, T), dtype=torch.uint8, device="cuda")
    m = None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda")
    f.pool.attn(B, hq, T, q.cuda(), f.table_d, f.lens_d, m, scale, out, ws, **kw)
    return out.cpu()


def _bounded(f, b, got, q, scale, n=None):
    n = f.lens[b] if n is None else n
    k, v = f.rows(b, "k", n), f.rows(b, "v", n)
    T = q.shape[0]
    ref, mag = (attention(q.double(), k, x, scale, n - T) for x in (v, v.abs()))
    err, bound = (got.double() - ref).abs(), 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 1e-30
    assert bool((err <= bound).all()), (b, float((err / bound).max()))


SHAPES = [  # query heads, kv heads, query tokens
    (4, 4, 1), (8, 2, 1), (64, 8, 1), (5, 1, 1), (16, 16, 1), (42, 6, 1),  # up to 8 rows a kv head
    (4, 2, 4), (3, 1, 2), (8, 8, 8),                                        # of several tokens
    (9, 1, 1), (24, 2, 1), (96, 8, 1), (64, 2, 1), (64, 1, 1),              # 16-row warps
    (32, 4, 4), (16, 1, 4), (48, 3, 4), (6, 2, 3), (10, 1, 5), (64, 64, 64),
]


@pytest.mark.parametrize("hq,hkv,T", SHAPES)
@pytest.mark.parametrize("lens", [[0, 1, 2, 15, 16, 17], [31, 32, 33, 63, 64, 65], [700, 5, 0, 1033]])
def test_against_64_bits(kv, hq, hkv, T, lens):
    f = Filled4(kv, lens, hkv=hkv, seed=hq + T)
    q = _queries(len(lens), T, hq, 3, 0.5)
    got = _run(f, q, 0.09)
    assert f.pool.error() == 0
    for b, n in enumerate(lens):
        _bounded(f, b, got[b], q[b], 0.09)
        for i in range(min(T, max(0, T - n))):  # no visible position: zeros
            assert not got[b, i].any()


@pytest.mark.parametrize("hq,hkv", [(64, 8), (24, 2)])
def test_long_requests(kv, hq, hkv):
    lens = [20011, 9000]
    f = Filled4(kv, lens, hkv=hkv, seed=1, spread=1)
    q = _queries(2, 1, hq, 4, 0.5)
    got = _run(f, q, 0.09)
    for b in range(2):
        _bounded(f, b, got[b], q[b], 0.09)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1)])
@pytest.mark.parametrize("where", [0, 40, 399, 600, 950])
def test_one_key_far_above_the_rest(kv, hq, hkv, where):
    """Rows whose largest weight appears early, late or in the middle: the reference has to
    follow it, and the many small weights keep their bits."""
    f = Filled4(kv, [960], hkv=hkv, seed=2, spread=0)
    byte, high, scale = PLACES["k"]
    q = _queries(1, 1, hq, 5, 0.05)
    q[0, 0, :, :16] = 1.0
    p, slot = int(f.table[0, where // 16]), where % 16
    tile = f.cache["k"][p, 0]
    f.scale["k"][:] = 0.25
    for other in range(f.cache["k"].shape[0]):  # elsewhere those dims are small
        f.cache["k"][other, 0, scale[:, 0]] = np.where(f.cache["k"][other, 0, scale[:, 0]] == 0x7F, 0x7F, 0x10)
    tile[scale[slot, 0]] = 0x50  # 8
    for d in range(16):
        b = byte[slot, d]
        tile[b] = (tile[b] & 0x0F) | 0x70 if high[slot, d] else (tile[b] & 0xF0) | 0x07
    f.to_device()
    got = _run(f, q, 0.09)  # the key's score: 16 * 6 * 8 / 4 * 0.09 = 17
    _bounded(f, 0, got[0], q[0], 0.09)


def test_query_range(kv):
    """Any finite bf16 query: rows scaled by powers of two give the same bits."""
    f = Filled4(kv, [100, 37], hkv=2, seed=6)
    q = _queries(2, 1, 8, 7)
    base = _run(f, q, 0.09)
    for e in (-40, 40):
        assert torch.equal(_run(f, (q.float() * 2.0 ** e).to(torch.bfloat16), 0.09 * 2.0 ** -e), base)


def test_requests_that_get_nothing(kv):
    """Aborted, of a bad length, with a page out of range: their outputs stay, the others are right."""
    lens = [50, 50, 50, 50, 50]
    f = Filled4(kv, lens, hkv=2, seed=8)
    q = _queries(5, 1, 8, 9, 0.5)
    f.table_d[2, 3] = -1
    f.lens_d[3] = -4
    got = _run(f, q, 0.09, mask=[0, 1, 0, 0, 0])
    assert f.pool.error() in (kv.KV_ERR_BAD_PAGE_ID, kv.KV_ERR_INVALID_ARG)
    for b in (1, 2, 3):
        assert bool((got[b] == 7.0).all())
    for b in (0, 4):
        _bounded(f, b, got[b], q[b], 0.09)


@pytest.mark.parametrize("hq,T", [(8, 1), (32, 2)])
def test_checked(kv, hq, T):
    lens = [50, 33, 700, 16, 0]
    f = Filled4(kv, lens, hkv=2, seed=10)
    tags = torch.randint(0, 2 ** 31 - 1, (f.pool.num_pages,), dtype=torch.int32)
    f.pool.tags.copy_(tags)
    exp = tags[torch.from_numpy(f.table).long().clamp_min(0)].int()
    exp[1, 2] ^= 1    # the request's last page, one row of it
    exp[2, 20] ^= 1
    q = _queries(5, T, hq, 11, 0.5)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.full((5,), 9, dtype=torch.uint8, device="cuda")
    ws = torch.empty(f.pool.workspace_size(5, hq, T), dtype=torch.uint8, device="cuda")
    kv.paged_decode_attn_checked(f.pool.handle, 5, hq, T, q.cuda(), f.table_d, exp.cuda(), f.lens_d, 0.09,
                                 out, mask, ws)
    assert mask.tolist() == [0, 1, 1, 0, 0] and f.pool.error() == 0
    got = out.cpu()
    assert bool((got[1:3] == 7.0).all())
    for b in (0, 3, 4):
        _bounded(f, b, got[b], q[b], 0.09)


def test_phases_noalloc_and_two_calls_at_once(kv):
    f = Filled4(kv, [500, 77, 3], hkv=2, seed=12)
    q = _queries(3, 1, 16, 13, 0.5)
    want = _run(f, q, 0.09)
    qd, n = q.cuda(), f.pool.workspace_size(3, 16, 1)
    out, ws = torch.empty_like(qd), torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.paged_decode_attn_split(f.pool.handle, 3, 16, 1, qd, f.table_d, f.lens_d, None, 0.09, ws)
    kv.paged_decode_attn_combine(f.pool.handle, 3, 16, 1, None, out, ws)
    assert torch.equal(out.cpu(), want)
    kv.paged_decode_attn_noalloc(f.pool.handle, 3, 16, 1, qd, f.table_d, f.lens_d, None, 0.09, out)
    assert torch.equal(out.cpu(), want)
    # two streams, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(qd) for _ in range(2)]
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, o, w in zip(streams, outs, wss):
            f.pool.attn(3, 16, 1, qd, f.table_d, f.lens_d, None, 0.09, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)


def test_small_workspace_is_refused(kv):
    f = Filled4(kv, [50], hkv=2)
    n = f.pool.workspace_size(1, 8, 1)
    q = _queries(1, 1, 8, 1).cuda()
    with pytest.raises(kv.KVError):
        f.pool.attn(1, 8, 1, q, f.table_d, f.lens_d, None, 0.1, torch.empty_like(q),
                    torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    for hq, T in ((130, 1), (32, 5)):  # more than 64 rows a kv head
        with pytest.raises(kv.KVError) as e:
            f.pool.workspace_size(1, hq, T)
        assert e.value.status == kv.KV_ERR_UNSUPPORTED


def test_captured_with_lengths_that_change(kv):
    lens = [600, 40, 333]
    f = Filled4(kv, lens, hkv=2, seed=14)
    q = _queries(3, 1, 8, 15, 0.5)
    qd = q.cuda()
    out, ws = torch.empty_like(qd), torch.empty(f.pool.workspace_size(3, 8, 1), dtype=torch.uint8, device="cuda")
    f.pool.attn(3, 8, 1, qd, f.table_d, f.lens_d, None, 0.09, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.pool.attn(3, 8, 1, qd, f.table_d, f.lens_d, None, 0.09, out, ws)
    for now in ([600, 40, 333], [17, 0, 300], [1, 40, 32]):
        f.lens_d.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        got = out.cpu()
        for b, n in enumerate(now):
            _bounded(f, b, got[b], q[b], 0.09, n)


@pytest.mark.parametrize("hq", [8, 24])
def test_many_requests(kv, hq):
    """More than the split kernels' plan cache holds."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 70, 1400).tolist()
    f = Filled4(kv, lens, hkv=2, seed=16)
    q = _queries(1400, 1, hq, 17, 0.5)
    got = _run(f, q, 0.09)
    assert f.pool.error() == 0
    for b in list(range(0, 1400, 97)) + [1399]:
        _bounded(f, b, got[b], q[b], 0.09)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (20, 2)])
@pytest.mark.parametrize("n", [40, 64])
def test_values_that_are_not_finite(kv, hq, hkv, n):
    """A draft token's V that is no number reaches the tokens that see it, in its group's dims, and
    no other row; a key that is no number makes NaN of the rows that see it."""
    T = 4
    f = Filled4(kv, [n], hkv=hkv, seed=18)
    q = _queries(1, T, hq, 19, 0.5)
    clean = _run(f, q, 0.09)
    pos = n - 2  # the third of four tokens
    p, slot = int(f.table[0, pos // 16]), pos % 16
    f.cache["v"][p, 0, PLACES["v"][2][slot, 3]] = 0x7F
    f.to_device()
    got = _run(f, q, 0.09)
    G = hq // hkv
    nan = torch.isnan(got[0])
    assert bool(nan[2:, :G, 48:64].all())
    nan[2:, :G, 48:64] = False
    assert not nan.any()
    keep = torch.ones_like(nan)
    keep[2:, :G, 48:64] = False
    assert torch.equal(got[0][keep], clean[0][keep])
    f.cache["v"][p, 0, PLACES["v"][2][slot, 3]] = 0x38
    f.cache["k"][p, 0, PLACES["k"][2][slot, 5]] = 0x7F
    f.to_device()
    nan = torch.isnan(_run(f, q, 0.09)[0])
    assert bool(nan[2:, :G].all()) and not nan[:2].any() and not nan[:, G:].any()


@pytest.mark.parametrize("hq", [8, 24])
def test_one_call_step(kv, hq):
    """kv_decode_step: a request leaves and another joins its slot with a prompt, one is stale;
    the appended rows and the attention are those of the separate calls."""
    lens = [100, 33, 64, 7]
    f, h = (Filled4(kv, lens, hkv=2, seed=20, spare=16, extra_width=6) for _ in range(2))
    g = torch.Generator().manual_seed(21)
    new = [1, 1, 1, 40]
    k, v = (torch.randn((sum(new), 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ind = torch.tensor([0, 1, 2, 3, 43], dtype=torch.int32).cuda()
    q = _queries(4, 1, hq, 22, 0.5)
    leave = torch.tensor([0, 0, 0, 1], dtype=torch.uint8).cuda()
    for x in (f, h):
        x.tags_d[1, 0] += 1
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.empty(4, dtype=torch.uint8, device="cuda")
    ws = torch.empty(f.pool.step_workspace_size(4, hq, 1), dtype=torch.uint8, device="cuda")
    f.pool.step(4, hq, 1, leave, k, v, ind, 40, f.table_d, f.tags_d, f.lens_d, q.cuda(), 0.09, out, mask, 0, ws)
    assert mask.tolist() == [0, 1, 0, 0] and f.pool.error() == 0
    assert f.lens_d.tolist() == [101, 33, 65, 40]
    rel = torch.empty(kv.kv_release_workspace_size(4), dtype=torch.uint8, device="cuda")
    h.pool.release(4, h.table_d, h.tags_d, h.lens_d, leave, rel)
    counts = [1, 0, 1, 40]
    keep = torch.tensor([0, 2, *range(3, 43)]).cuda()
    ind2 = torch.tensor([0, 1, 1, 2, 42], dtype=torch.int32).cuda()
    h.pool.append(4, k[keep].contiguous(), v[keep].contiguous(), ind2, max(counts), h.table_d, h.tags_d, h.lens_d)
    for a, b in ((f.pool.k_cache, h.pool.k_cache), (f.pool.v_cache, h.pool.v_cache), (f.table_d, h.table_d)):
        assert torch.equal(a, b)
    want = _run(h, q, 0.09)
    got = out.cpu()
    assert bool((got[1] == 7.0).all())
    for b in (0, 2, 3):
        assert torch.equal(got[b], want[b])


PAIRS = [  # 17 to 32 and 49 to 64 query rows a kv head, of 4 or 8 kv heads
    (80, 4, 1), (128, 4, 1), (24, 4, 3), (192, 8, 1), (48, 4, 2), (64, 4, 4), (52, 4, 4), (98, 2, 1), (512, 8, 1),
]


@pytest.mark.parametrize("hq,hkv,T", PAIRS)
@pytest.mark.parametrize("lens", [[0, 1, 2, 15, 16, 17], [31, 32, 33, 63, 64, 65], [700, 5, 0, 1033]])
def test_warps_of_32_rows(kv, hq, hkv, T, lens):
    f = Filled4(kv, lens, hkv=hkv, seed=hq + T)
    q = _queries(len(lens), T, hq, 31, 0.5)
    got = _run(f, q, 0.09)
    assert f.pool.error() == 0
    for b in range(len(lens)):
        _bounded(f, b, got[b], q[b], 0.09)


@pytest.mark.parametrize("where", [0, 40, 600, 950])
@pytest.mark.parametrize("row", [3, 12, 17, 30])
def test_one_key_far_above_the_rest_for_one_row_of_32(kv, where, row):
    """One row's query lies along one key, which is several times longer than the others: its score
    is 40 and theirs below 20, so the row is that key's value; the block's other rows, and the other
    block's, keep their references.  (A row's terms sum to at most 40 / 0.09 < 2^9.)"""
    f = Filled4(kv, [1000], hkv=4, seed=33, spread=0)
    p, slot = int(f.table[0, where // 16]), where % 16
    f.cache["k"][p, 0, PLACES["k"][2][slot]] = 0x50  # 8: the others are below 2
    f.to_device()
    q = _queries(1, 1, 128, 34, 0.02)
    keys = f.rows(0, "k")[:, 0]
    k = keys[where]
    q[0, 0, row] = (k * (40.0 / float(k @ k) / 0.09)).to(torch.bfloat16)
    score = keys @ q[0, 0, row].double() * 0.09
    score[where] = -40.0
    assert float(score.max()) < 20
    got = _run(f, q, 0.09)[0]
    # The file's bound with its last part by itself: the other keys' weights, below 2^-20 of the
    # largest, are off by up to 2^-31 of it each, which is no part of A in a dim where that key's
    # value is 0: 999 * 2^-31 of the largest value for the row.
    v = f.rows(0, "v")
    ref, mag = (attention(q[0].double(), f.rows(0, "k"), x, 0.09, 999) for x in (v, v.abs()))
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag
    bound[0, row] += 999 * 2.0 ** -31 * v[:, 0].abs().max()
    assert bool(((got.double() - ref).abs() <= bound).all())
    assert float((got[0, row].double() - v[where, 0]).abs().max()) <= 2.0 ** -7 * float(v[where, 0].abs().max())


def test_values_that_are_not_finite_in_warps_of_32_rows(kv):
    T, n = 4, 40
    f = Filled4(kv, [n], hkv=4, seed=35)
    q = _queries(1, T, 32, 36, 0.5)
    clean = _run(f, q, 0.09)
    pos = n - 2
    p, slot = int(f.table[0, pos // 16]), pos % 16
    f.cache["v"][p, 0, PLACES["v"][2][slot, 3]] = 0x7F
    f.to_device()
    got = _run(f, q, 0.09)
    nan = torch.isnan(got[0])
    keep = torch.ones_like(nan)
    keep[2:, :8, 48:64] = False
    assert bool(nan[~keep].all()) and not nan[keep].any()
    assert torch.equal(got[0][keep], clean[0][keep])
    f.cache["v"][p, 0, PLACES["v"][2][slot, 3]] = 0x38
    f.cache["k"][p, 0, PLACES["k"][2][slot, 5]] = 0x7F
    f.to_device()
    nan = torch.isnan(_run(f, q, 0.09)[0])
    assert bool(nan[2:, :8].all()) and not nan[:2].any() and not nan[:, 8:].any()


@pytest.mark.parametrize("hq,B", [(128, 5), (256, 1200)])
def test_checked_and_captured_in_warps_of_32_rows(kv, hq, B):
    """32 and 64 rows: stale tags, and the same bits from a replayed graph and in the fixed scratch."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 60, B).tolist()
    lens[1], lens[3] = 50, 33
    f = Filled4(kv, lens, hkv=4, seed=37)
    tags = torch.zeros((B, f.table.shape[1]), dtype=torch.int32, device="cuda")
    tags[1, 2] = 5
    q = _queries(B, 1, hq, 38, 0.5)
    qd, out = q.cuda(), torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.full((B,), 9, dtype=torch.uint8, device="cuda")
    ws = torch.empty(f.pool.workspace_size(B, hq, 1), dtype=torch.uint8, device="cuda")

    def run():
        kv.paged_decode_attn_checked(f.pool.handle, B, hq, 1, qd, f.table_d, tags, f.lens_d, 0.09, out, mask, ws)

    run()
    first = out.cpu()
    assert mask.nonzero().flatten().tolist() == [1] and f.pool.error() == 0
    assert bool((first[1] == 7.0).all())
    for b in [0, 2, 3, 4, B - 1]:
        _bounded(f, b, first[b], q[b], 0.09)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    out.fill_(7.0)
    graph.replay()
    assert torch.equal(out.cpu(), first)
