"""paged_prefill_attn against the 64-bit form.

Bound of an output o = sum_j p_j v_j / sum_j p_j, with A = sum_j p_j |v_j| / sum_j p_j:
  bf16 output           2^-9 |o| (half a step is 2^-8 of the value at most)  -> 2^-8 |o|
  P rounded to f16      2^-11 of each weight (bf16 pools: P to bf16, 2^-8)   -> 2^-11 A | 2^-8 A
  scores                the dot product's fp32 sums: 128 terms, 2^-24 each of sum |q k|, which here
                        stays below 64 in log2 units after scaling (queries and keys are drawn
                        so): 128 * 64 * 2^-24 = 2^-11, times ln 2; the exponential 2^-22 of its
                        value and its argument's rounding, 64 * 2^-24; twice (o and the sum)
                                                                            -> 2^-10 A
  accumulation          blocks' sums of up to 2^13 terms in fp32, rescales  -> 2^-11 A
In all |err| <= 2^-8 |o| + c A, c = 2^-11 + 2^-10 + 2^-11 = 2^-9 (bf16 pools: 2^-8 + 2^-9 + 2^-10)."""
import math

import pytest
import torch

from promptref import Filled, attention, indptr

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _queries(f, new, hq, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((sum(new), hq, 128), generator=g) * scale).to(torch.bfloat16)


def _run(f, q, new, aborted=None, extra=0, sm_scale=SCALE, ws=None, out=None, stream=None):
    hq = q.shape[1]
    total = q.shape[0] + extra
    qd = torch.zeros((total, hq, 128), dtype=torch.bfloat16, device="cuda")
    qd[:q.shape[0]] = q.cuda()
    if out is None:
        out = torch.full((total, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ab = None if aborted is None else torch.tensor(aborted, dtype=torch.uint8, device="cuda")
    if ws is None:  # whatever the workspace held, NaN among it
        ws = torch.full((f.pool.prefill_workspace_size(f.B, hq, total),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    f.pool.prefill_attn(f.B, hq, qd, indptr(new).cuda(), f.table_d, f.lens_d, ab, sm_scale, out, ws,
                        stream)
    return out


def _check(f, q, new, out, skip=(), sm_scale=SCALE):
    got = out.cpu().double()
    ind = indptr(new)
    c = 2.0 ** -9 if f.fp8 else 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10
    for b in range(f.B):
        lo, hi = int(ind[b]), int(ind[b + 1])
        if lo == hi:
            continue
        if b in skip:
            assert bool((got[lo:hi] == 7.0).all()), b
            continue
        k, v = f.rows(b, "k"), f.rows(b, "v")
        old = f.lens[b] - new[b]
        ref = attention(q[lo:hi].double(), k, v, sm_scale, old)
        mag = attention(q[lo:hi].double(), k, v.abs(), sm_scale, old)
        err = (got[lo:hi] - ref).abs()
        bound = 2.0 ** -8 * ref.abs() + c * mag + 1e-30
        worst = float((err / bound).max())
        assert worst <= 1.0, (b, worst, float(err.max()))
    assert bool((got[int(ind[-1]):] == 7.0).all())


# (lengths with the new tokens, new tokens)
BATCHES = {
    "one token": ([1], [1]),
    "few": ([37, 64, 100, 255], [5, 17, 1, 33]),
    "whole prompts": ([300, 1, 129, 128, 127], [300, 1, 129, 128, 127]),
    "none for some": ([50, 0, 70, 16], [0, 0, 70, 3]),
    "more queries than rows": ([3, 0, 20], [10, 2, 20]),
    "single tokens": ([16, 17, 1000, 2049, 5], [1, 1, 1, 1, 1]),
    "mixed": ([700, 333, 1500, 40], [257, 1, 64, 40]),
}


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [(8, 2), (1, 1), (12, 1), (5, 1), (6, 3), (32, 2)])
@pytest.mark.parametrize("name", list(BATCHES))
def test_batches(kv, name, heads, fp8):
    lens, new = BATCHES[name]
    hq, hkv = heads
    f = Filled(kv, lens, hkv=hkv, fp8=fp8, seed=41)
    q = _queries(f, new, hq, 42)
    out = _run(f, q, new, extra=3)
    _check(f, q, new, out)
    assert f.pool.error() == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lens,new,heads", [
    ([9000], [1], (8, 1)),            # one row group, cut over many CTAs
    ([6000, 5000], [16, 15], (64, 8)),  # one tile and a bit less
    ([4500], [600], (16, 2)),         # items cut by ranges
    ([2100], [2100], (8, 2)),
    ([3001, 17, 900], [33, 17, 129], (136, 1)),  # groups larger than a tile
])
def test_longer(kv, lens, new, heads, fp8):
    f = Filled(kv, lens, hkv=heads[1], fp8=fp8, seed=43)
    q = _queries(f, new, heads[0], 44)
    _check(f, q, new, _run(f, q, new))
    assert f.pool.error() == 0


def test_many_requests(kv):
    lens = [1 + (37 * i) % 300 for i in range(700)]
    new = [min(n, (11 * i) % 9) for i, n in enumerate(lens)]
    f = Filled(kv, lens, hkv=1, seed=45)
    q = _queries(f, new, 4, 46)
    _check(f, q, new, _run(f, q, new))


@pytest.mark.parametrize("fp8", [True, False])
def test_growing_scores(kv, fp8):
    """Keys that grow along the sequence make the running maximum move in every block."""
    f = Filled(kv, [1500], hkv=1, fp8=fp8, seed=47)
    ramp = torch.linspace(0.1, 3.0, 94)
    for j in range(94):
        p = int(f.table[0, j])
        if fp8:
            f.ks[p] = 1e-3 * ramp[j]
        else:
            f.k[p] = (f.k[p].float() * ramp[j]).to(torch.bfloat16)
    if fp8:
        f.pool.k_scale.copy_(f.ks)
    else:
        f.pool.k_cache.copy_(f.k)
    q = _queries(f, [200], 8, 48, 3.0)
    _check(f, q, [200], _run(f, q, [200]))


@pytest.mark.parametrize("mag", [1e-30, 1e6])
def test_query_and_value_magnitudes(kv, mag):
    """Any finite query: large ones meet small keys, so that the scores stay as they are; V scales
    from 1e-30 to 1e6 in one row."""
    f = Filled(kv, [400], hkv=2, seed=49)
    f.ks /= mag
    f.vs[::3] *= 1e-28
    f.vs[1::3] *= 1e8
    f.pool.k_scale.copy_(f.ks)
    f.pool.v_scale.copy_(f.vs)
    q = _queries(f, [90], 8, 50, mag)
    _check(f, q, [90], _run(f, q, [90]))


@pytest.mark.parametrize("sm_scale", [-0.05, 0.0, 0.3])
@pytest.mark.parametrize("fp8", [True, False])
def test_scales_of_any_sign(kv, sm_scale, fp8):
    f = Filled(kv, [300], hkv=1, fp8=fp8, seed=51)
    f.ks = None if f.ks is None else f.ks * 0.3
    if fp8:
        f.pool.k_scale.copy_(f.ks)
    q = _queries(f, [140], 4, 52)
    _check(f, q, [140], _run(f, q, [140], sm_scale=sm_scale), sm_scale=sm_scale)


def test_aborted_and_refused_requests(kv):
    lens, new = [200, 300, 100, 50], [20, 300, 30, 10]
    f = Filled(kv, lens, hkv=2, seed=53)
    f.lens_d[2] = 10 ** 6  # beyond its page table
    q = _queries(f, new, 8, 54)
    out = _run(f, q, new, aborted=[0, 1, 0, 0])
    _check(f, q, new, out, skip=(1, 2))
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG


def test_bad_page_ids(kv):
    lens, new = [900, 600], [40, 30]
    for bad in (-5, 10 ** 7):
        f = Filled(kv, lens, hkv=1, seed=55)
        f.table_d[0, 20] = bad
        q = _queries(f, new, 8, 56)
        out = _run(f, q, new)
        _check(f, q, new, out, skip=(0,))
        assert f.pool.error() == kv.KV_ERR_BAD_PAGE_ID


def test_equals_decode_attention(kv):
    """A batch of four tokens a request is also paged_decode_attn's."""
    lens = [100, 77, 1030]
    for fp8 in (True, False):
        f = Filled(kv, lens, hkv=2, fp8=fp8, seed=57)
        q = _queries(f, [4] * 3, 16, 58)
        out = _run(f, q, [4] * 3)
        _check(f, q, [4] * 3, out)
        ws = torch.empty(f.pool.workspace_size(3, 16, 4), dtype=torch.uint8, device="cuda")
        dec = torch.zeros((3, 4, 16, 128), dtype=torch.bfloat16, device="cuda")
        f.pool.attn(3, 16, 4, q.cuda().view(3, 4, 16, 128), f.table_d, f.lens_d, None, SCALE, dec, ws)
        _check(f, q, [4] * 3, dec.view(12, 16, 128))


def test_repeatable(kv):
    f = Filled(kv, [1800, 700], hkv=2, seed=59)
    new = [300, 1]
    q = _queries(f, new, 16, 60)
    a = _run(f, q, new)
    for _ in range(3):
        assert torch.equal(a.view(torch.int16), _run(f, q, new).view(torch.int16))


def test_graph_with_moving_lengths(kv):
    """A captured call plans on the device: replays follow lengths and row counts."""
    f = Filled(kv, [500, 300], hkv=2, seed=61)
    g1 = torch.Generator().manual_seed(62)
    q = torch.randn((260, 8, 128), generator=g1).to(torch.bfloat16)
    qd, out = q.cuda(), torch.full((260, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ind = indptr([100, 160]).cuda()
    ws = torch.empty(f.pool.prefill_workspace_size(2, 8, 260), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.pool.prefill_attn(2, 8, qd, ind, f.table_d, f.lens_d, None, SCALE, out, ws)
    for lens, new in (([500, 300], [100, 160]), ([129, 300], [1, 7]), ([40, 299], [40, 0])):
        f.lens = lens
        f.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        ind.copy_(indptr(new))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        _check(f, q[:sum(new)], new, out)


def test_two_streams(kv):
    """Two calls at once, each with its own workspace."""
    f = Filled(kv, [2500, 1200], hkv=4, seed=63)
    new = [500, 40]
    q = _queries(f, new, 16, 64)
    ref = _run(f, q, new)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(ref, 7.0) for _ in ss]
    torch.cuda.synchronize()
    for s, o in zip(ss, outs):
        with torch.cuda.stream(s):
            _run(f, q, new, out=o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16))


def test_no_queries(kv):
    f = Filled(kv, [10], hkv=1, seed=65)
    out = _run(f, torch.zeros((0, 8, 128), dtype=torch.bfloat16), [0], extra=5)
    assert bool((out == 7.0).all()) and f.pool.error() == 0
    assert math.isfinite(SCALE)


@pytest.mark.parametrize("ind", [[0, 40, 81], [-5, 40, 60], [100000, 100040, 100060], [0, 40, 20]])
def test_rows_outside_the_queries(kv, ind):
    """Requests whose rows lie outside q are refused, wherever they begin."""
    f = Filled(kv, [60, 90], hkv=2, seed=67)
    q = _queries(f, [80], 8, 68)
    out = torch.full((80, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(f.pool.prefill_workspace_size(2, 8, 80), dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(2, 8, q.cuda(), torch.tensor(ind, dtype=torch.int32).cuda(), f.table_d, f.lens_d, None,
                        SCALE, out, ws)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    if ind[0] == 0:
        f.B = 1
        _check(f, q[:40], [40], out)
    else:
        assert bool((out[:40] == 7.0).all())
