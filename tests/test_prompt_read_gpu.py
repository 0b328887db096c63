"""kv_read_rows against the 64-bit form: the values are one fp32 product and
one bf16 rounding, so they equal the rounding of the exact product except
where the fp32 product falls on the other side of a bf16 border: at most one
bf16 half step (2^-8 relative) and fp32's 2^-24 apart."""
import pytest
import torch

from promptref import Filled, indptr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _read(f, first, counts, total=None, aborted=None, stream=None, null_start=False):
    ind = indptr(counts)
    rows = int(ind[-1]) if total is None else total
    shape_k = (rows, f.dk) if f.latent else (rows, f.hkv, f.dk)
    k = torch.full(shape_k, 7.0, dtype=torch.bfloat16, device="cuda")
    v = None if f.latent else torch.full((rows, f.hkv, f.dv), 7.0, dtype=torch.bfloat16,
                                         device="cuda")
    st = None if null_start else torch.tensor(first, dtype=torch.int32, device="cuda")
    ab = None if aborted is None else torch.tensor(aborted, dtype=torch.uint8, device="cuda")
    f.pool.read_rows(f.B, f.table_d, f.lens_d, st, ind.cuda(), ab, k, v, stream)
    return ind, k, v


def _check(f, first, ind, k, v, skip=()):
    for which, got in (("k", k), ("v", v)):
        if got is None:
            continue
        got = got.cpu()
        for b in range(f.B):
            lo, hi = int(ind[b]), int(ind[b + 1])
            if b in skip:
                assert bool((got[lo:hi] == 7.0).all())
                continue
            ref = f.rows(b, which)[first[b]:first[b] + hi - lo]
            x = got[lo:hi].double()
            assert bool(((x - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()), (which, b)
        assert bool((got[int(ind[-1]):] == 7.0).all())


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("shape", [
    dict(hkv=2), dict(hkv=8), dict(hkv=1, dk=64, dv=64), dict(hkv=3, dk=256, dv=80, page=32),
    dict(hkv=2, dk=128, dv=128, page=64), dict(hkv=2, dk=16, dv=16, page=5),
    dict(hkv=1, dk=576, dv=512, page=64, latent=True), dict(hkv=1, dk=48, dv=16, page=7, latent=True)])
def test_all_rows(kv, shape, fp8):
    f = Filled(kv, [1, 37, 64, 0, 255, 16, 17], fp8=fp8, seed=3, **shape)
    ind, k, v = _read(f, [0] * f.B, f.lens, null_start=True)
    _check(f, [0] * f.B, ind, k, v)
    assert f.pool.error() == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("latent", [True, False])
def test_windows(kv, fp8, latent):
    shape = dict(hkv=1, dk=576, dv=512, page=64, latent=True) if latent else dict(hkv=4)
    f = Filled(kv, [200, 33, 16, 129, 90], fp8=fp8, seed=4, **shape)
    first, counts = [15, 32, 0, 1, 90], [17, 1, 16, 127, 0]
    ind, k, v = _read(f, first, counts, total=sum(counts) + 5)
    _check(f, first, ind, k, v)
    assert f.pool.error() == 0


def test_many_requests(kv):
    lens = [1 + (7 * i) % 50 for i in range(1200)]
    f = Filled(kv, lens, hkv=1, seed=5)
    first = [n // 3 for n in lens]
    ind, k, v = _read(f, first, [n - a for n, a in zip(lens, first)])
    _check(f, first, ind, k, v)


def test_aborted_and_refused_requests(kv):
    f = Filled(kv, [40, 50, 60, 70], seed=6)
    # an aborted request, one that asks for more rows than it has, one with a negative start
    first = [0, 0, 1, -1]
    ind, k, v = _read(f, first, [40, 50, 60, 10], aborted=[0, 1, 0, 0])
    _check(f, first, ind, k, v, skip=(1, 2, 3))
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG


def test_bad_page(kv):
    f = Filled(kv, [40, 50], seed=7)
    f.table_d[1, 1] = 10 ** 6
    ind, k, v = _read(f, [0, 0], [40, 50])
    assert f.pool.error() == kv.KV_ERR_BAD_PAGE_ID
    assert bool((k[40 + 16:40 + 32] == 7.0).all())  # that page's rows alone
    f2 = Filled(kv, [40, 50], seed=7)
    _check(f2, [0, 0], indptr([40, 0]), k[:40], v[:40])
    assert bool(((k[72:90].cpu().double() - f2.rows(1, "k")[32:50]).abs()
                 <= 2.0 ** -7 * f2.rows(1, "k")[32:50].abs()).all())


def test_graph_and_other_stream(kv):
    f = Filled(kv, [100, 33], seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ind, k, v = _read(f, [0, 0], f.lens, stream=s)
    s.synchronize()
    _check(f, [0, 0], ind, k, v)
    ind_d, k2, v2 = ind.cuda(), torch.zeros_like(k), torch.zeros_like(v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.pool.read_rows(f.B, f.table_d, f.lens_d, None, ind_d, None, k2, v2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2)


@pytest.mark.parametrize("ind", [[0, 40, 81], [-5, 40, 60], [100000, 100040, 100060], [0, 40, 20]])
def test_rows_outside_the_outputs(kv, ind):
    """Requests whose rows do not fit the outputs are refused, wherever they begin."""
    f = Filled(kv, [60, 60], hkv=2, seed=91)
    k = torch.full((80, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    f.pool.read_rows(2, f.table_d, f.lens_d, None, torch.tensor(ind, dtype=torch.int32).cuda(), None, k, v)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    rows = f.rows(0, "k")[:40] if ind[0] == 0 else None
    assert bool((k[40 if ind[0] == 0 else 0:] == 7.0).all() if ind[0] >= 0 else (k[:40] == 7.0).all())
    if rows is not None:
        assert bool(((k[:40].cpu().double() - rows).abs() <= (2.0 ** -8 + 2.0 ** -23) * rows.abs()).all())
