"""kv_append_rotary against the 64-bit form.

Bounds.  The fraction of a turn is a 64-bit product, rounded to fp32 (2^-24 of
at most half a turn: 2 pi * 2^-25 < 2^-22 in the angle), sine and cosine add at
most 2 ulp (2^-22), so a rotated value is off by at most 2^-20 of its pair's
length beside the two products' and the sum's roundings (2^-22 of it): 2^-19 of
the pair's length in all.  A bf16 output adds half a step, 2^-8 of the value; an
e4m3 code adds half a step, 2^-4 of the value or half the smallest step, 2^-10
scales, and its scale is off by what the largest value is off."""
import math

import pytest
import torch

from promptref import Filled, e4m3_values, indptr, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _inputs(f, new, hq, rot, axes, seed, far=0, packed=False):
    g = torch.Generator().manual_seed(seed)
    t = sum(new)
    dims = hq * f.dk + f.hkv * (f.dk + f.dv)
    if packed:  # one projection's output
        x = torch.randn((t, dims + 24), generator=g).to(torch.bfloat16)
        q = x[:, :hq * f.dk].unflatten(1, (hq, f.dk)) if hq else None
        k = x[:, hq * f.dk:(hq + f.hkv) * f.dk].unflatten(1, (f.hkv, f.dk))
        v = x[:, (hq + f.hkv) * f.dk:dims].unflatten(1, (f.hkv, f.dv))
        xd = x.cuda()
        qd = xd[:, :hq * f.dk].unflatten(1, (hq, f.dk)) if hq else None
        kd = xd[:, hq * f.dk:(hq + f.hkv) * f.dk].unflatten(1, (f.hkv, f.dk))
        vd = xd[:, (hq + f.hkv) * f.dk:dims].unflatten(1, (f.hkv, f.dv))
    else:
        q = torch.randn((t, hq, f.dk), generator=g).to(torch.bfloat16) if hq else None
        k = torch.randn((t, f.hkv, f.dk), generator=g).to(torch.bfloat16)
        v = torch.randn((t, f.hkv, f.dv), generator=g).to(torch.bfloat16)
        qd, kd, vd = (None if z is None else z.cuda() for z in (q, k, v))
    pos = torch.randint(0, 4000, (axes, t), generator=g, dtype=torch.int32) + far
    axis = (torch.randint(0, axes, (rot // 2,), generator=g)).to(torch.uint8)
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return (q, k, v, pos, axis, freq), (qd, kd, vd, pos.cuda(), axis.cuda(), freq.cuda())


def _call(f, new, hq, dev, interleaved, max_new=None, ind=None, q_out=None, stream=None):
    qd, kd, vd, pos, axis, freq = dev
    if hq and q_out is None:
        q_out = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ind = indptr(new).cuda() if ind is None else ind
    f.pool.append_rotary(f.B, hq, qd, kd, vd, ind, max(new + [0]) if max_new is None else max_new,
                         pos, axis, freq, interleaved, q_out, f.table_d, f.tags_d, f.lens_d, stream)
    return q_out


def _pair_len(x, rot, interleaved):
    """Each value's pair length (its own magnitude behind rot)."""
    y = x.double().abs().clone()
    h = rot // 2
    i = torch.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    n = torch.sqrt(y[..., a] ** 2 + y[..., b] ** 2)
    y[..., a], y[..., b] = n, n
    return y


def _check(f, new, host, q_out, interleaved, served=None, old=None):
    q, k, v, pos, axis, freq = host
    rot = 2 * len(freq)
    served = f.B if served is None else served
    ind = indptr(new)
    cut = int(ind[served])
    old = f.lens if old is None else old
    if q is not None:
        got, ref = q_out.cpu().double(), rotate(q, pos, axis, freq, interleaved)
        bound = 2.0 ** -19 * _pair_len(q, rot, interleaved) + 2.0 ** -8 * ref.abs() + 1e-38
        assert bool(((got - ref).abs() <= bound)[:cut].all())
        assert bool((got[cut:] == 7.0).all())
    kr, klen = rotate(k, pos, axis, freq, interleaved), _pair_len(k, rot, interleaved)
    vr = v.double()
    table, P = f.table_d.cpu(), f.page
    kc, vc = f.pool.k_cache.cpu(), f.pool.v_cache.cpu()
    head = f.free_head
    for b in range(served):
        assert int(f.lens_d[b]) == old[b] + new[b]
        row = 0
        while row < new[b]:
            j, slot = divmod(old[b] + row, P)
            n = min(P - slot, new[b] - row)
            p = int(table[b, j])
            if slot == 0:  # popped in order
                assert p == int(f.free_list[head])
                head += 1
            rows = slice(int(ind[b]) + row, int(ind[b]) + row + n)
            for which, x, ln in (("k", kr[rows], klen[rows]), ("v", vr[rows], None)):
                x = x.transpose(0, 1)  # [heads][rows][dim]
                slack = 2.0 ** -19 * ln.transpose(0, 1) if ln is not None else torch.zeros(1)
                got = (kc[p, :, slot:slot + n] if which == "k"
                       else vc[p, :, :, slot:slot + n].transpose(1, 2))
                if not f.fp8:
                    assert bool(((got.double() - x).abs() <= slack + 2.0 ** -8 * x.abs()).all())
                    continue
                s = (f.pool.k_scale if which == "k" else f.pool.v_scale)[p].cpu().double()
                if slot == 0:
                    amax = x.abs().amax((1, 2))
                    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
                    off = 2.0 ** -19 * (ln.amax() if ln is not None else 0) / 448 + 2.0 ** -23 * want
                    assert bool(((s - want).abs() <= off).all())
                val = e4m3_values()[got.long()] * s[:, None, None]
                lim = 448 * s[:, None, None]
                xs = torch.minimum(torch.maximum(x, -lim), lim)
                # the quotient's rounding before the code's: 2^-23 of the value
                bound = slack + (2.0 ** -4 + 2.0 ** -20) * xs.abs() + 2.0 ** -10 * s[:, None, None]
                assert bool(((val - xs).abs() <= bound).all()), (b, j, which)
            row += n
    if served == f.B:
        assert f.pool.error() == 0


SHAPES = [dict(hkv=2), dict(hkv=8), dict(hkv=1, dk=64, dv=64), dict(hkv=3, dk=256, dv=128, page=8),
          dict(hkv=2, dk=80, dv=48, page=25), dict(hkv=1, dk=16, dv=16, page=1)]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_ragged(kv, shape, interleaved, fp8):
    s = SHAPES[shape]
    f = Filled(kv, [0, 5, 16, 31, 100, 7], fp8=fp8, seed=11, spare=400, extra_width=400, **s)
    new = [33, 1, 16, 0, 129, 40]
    rot = 16 * max(1, f.dk // 32)
    host, dev = _inputs(f, new, 3 * f.hkv, rot, 3, 12)
    out = _call(f, new, 3 * f.hkv, dev, interleaved)
    _check(f, new, host, out, interleaved)


@pytest.mark.parametrize("axes,rot", [(1, 128), (2, 64), (3, 128), (4, 16)])
def test_axes_and_partial_rotation(kv, axes, rot):
    f = Filled(kv, [20, 0, 3], hkv=4, seed=13, spare=40, extra_width=20)
    new = [50, 17, 1]
    host, dev = _inputs(f, new, 16, rot, axes, 14, packed=True)
    _check(f, new, host, _call(f, new, 16, dev, False), False)


def test_far_positions(kv):
    """Positions near 2^31 turn by exact fractions (the 64-bit product's own
    rounding, 2^-53 of 2^31 radians, is 2^-22)."""
    f = Filled(kv, [0, 9], seed=15, spare=20, extra_width=8)
    new = [20, 30]
    host, dev = _inputs(f, new, 4, 128, 2, 16, far=2 ** 31 - 5000)
    _check(f, new, host, _call(f, new, 4, dev, False), False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_positions_and_frequencies(kv, interleaved):
    """Turns of either sign and of more than a whole turn a position (4000 positions of 40 radians
    in 64 bits: the fraction of a turn is off by 2^-38)."""
    f = Filled(kv, [0, 9], hkv=2, seed=43, spare=20, extra_width=8)
    new = [20, 30]
    host, dev = _inputs(f, new, 6, 96, 2, 44)
    for i, t in ((3, "pos"), (5, "freq")):
        if t == "pos":
            host[i][:, ::2] *= -1
        else:
            host[i][::3] *= -40.0
        dev[i].copy_(host[i])
    _check(f, new, host, _call(f, new, 6, dev, interleaved), interleaved)


def test_frequency_that_is_not_finite(kv):
    """Its pairs become NaN, in queries and bf16 keys; every other dim is right."""
    f = Filled(kv, [0], hkv=1, fp8=False, seed=45, spare=4, extra_width=3)
    host, dev = _inputs(f, [18], 2, 128, 1, 46)
    dev[5][3], dev[5][60] = float("nan"), float("inf")
    out = _call(f, [18], 2, dev, False).cpu().double()
    bad = [3, 67, 60, 124]
    rest = [i for i in range(128) if i not in bad]
    ref = rotate(host[0], host[3], host[4], host[5], False)
    bound = 2.0 ** -19 * _pair_len(host[0], 128, False) + 2.0 ** -8 * ref.abs() + 1e-38
    assert bool(torch.isnan(out[..., bad]).all())
    assert bool(((out - ref).abs() <= bound)[..., rest].all())
    k = f.pool.k_cache.cpu()[f.table_d[0, 0].item(), 0].double()  # the first page's 16 rows
    kr, kl = rotate(host[1], host[3], host[4], host[5], False)[:16, 0], _pair_len(host[1], 128, False)[:16, 0]
    assert bool(torch.isnan(k[:, bad]).all())
    assert bool(((k - kr).abs() <= 2.0 ** -19 * kl + 2.0 ** -8 * kr.abs() + 1e-38)[:, rest].all())


def test_decode_rows_and_no_queries(kv):
    f = Filled(kv, list(range(30, 94)), hkv=2, seed=17, spare=70, extra_width=3)
    new = [1] * 64
    host, dev = _inputs(f, new, 0, 128, 3, 18)
    _check(f, new, host, _call(f, new, 0, dev, False), False)


def test_in_place_queries(kv):
    f = Filled(kv, [3, 40], seed=19, spare=20, extra_width=8)
    new = [20, 18]
    host, dev = _inputs(f, new, 8, 64, 1, 20)
    _check(f, new, host, _call(f, new, 8, dev, False, q_out=dev[0]), False)


def test_zero_rows_and_tiny_values(kv):
    f = Filled(kv, [0, 0], seed=21, spare=20, extra_width=8)
    new = [16, 20]
    host, dev = _inputs(f, new, 4, 128, 1, 22)
    for x in (host[1], dev[1], host[2], dev[2]):
        x[:16] = 0
        x[16:] *= 1e-30  # scales below 2^-90 take the IEEE divide
    _check(f, new, host, _call(f, new, 4, dev, False), False)
    p = int(f.table_d[0, 0])
    assert bool((f.pool.k_scale[p] == 1.0).all())


def test_equals_plain_append_without_turning(kv):
    """At position 0 nothing turns: the cache equals kv_append_quantize's, bit for bit."""
    for fp8 in (True, False):
        fs = [Filled(kv, [5, 0, 16], hkv=2, fp8=fp8, seed=23, spare=40, extra_width=10)
              for _ in range(2)]
        new = [30, 48, 1]
        host, dev = _inputs(fs[0], new, 4, 128, 1, 24)
        dev[3].zero_()
        _call(fs[0], new, 4, dev, False)
        fs[1].pool.append(3, dev[1], dev[2], indptr(new).cuda(), 48, fs[1].table_d, fs[1].tags_d,
                          fs[1].lens_d)
        a, b = fs[0].pool, fs[1].pool
        raw = lambda t: t.view(torch.uint8)  # noqa: E731
        assert torch.equal(raw(a.k_cache), raw(b.k_cache))
        assert torch.equal(raw(a.v_cache), raw(b.v_cache))
        assert torch.equal(a.tags, b.tags) and torch.equal(a.ctl, b.ctl)
        assert torch.equal(fs[0].table_d, fs[1].table_d)
        if fp8:
            assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


def test_growing_rows_requantise(kv):
    """KV_SCALE_REQUANTIZE: larger rows in a partly filled page raise its scale."""
    f = Filled(kv, [5], hkv=1, seed=25, spare=4, extra_width=2, scale_mode=kv.KV_SCALE_REQUANTIZE)
    before = f.rows(0, "k")
    host, dev = _inputs(f, [4], 2, 128, 1, 26)
    dev[1].mul_(1000)
    host[1].mul_(1000)
    p = int(f.table[0, 0])
    old = float(f.ks[p, 0])
    _call(f, [4], 2, dev, False)
    s = float(f.pool.k_scale[p, 0])
    ref = rotate(host[1], *host[3:], False)
    assert s > old and abs(s - float(ref.abs().max()) / 448) <= 2.0 ** -18 * s
    now = e4m3_values()[f.pool.k_cache[p, 0].cpu().long()] * s
    assert bool(((now[:5] - before[:, 0]).abs()
                 <= (2.0 ** -4 + 2.0 ** -20) * before[:, 0].abs() + 2.0 ** -10 * s).all())
    assert bool(((now[5:9] - ref[:, 0]).abs()
                 <= (2.0 ** -4 + 2.0 ** -18) * ref[:, 0].abs() + 2.0 ** -10 * s).all())


def test_stops_leave_the_rest(kv):
    """Out of pages at request 1: request 0 is served, the others keep everything."""
    f = Filled(kv, [3, 0, 20], seed=27, spare=2, extra_width=20)
    new = [20, 40, 5]
    host, dev = _inputs(f, new, 4, 128, 1, 28)
    out = _call(f, new, 4, dev, False)
    _check(f, new, host, out, False, served=1)
    assert f.pool.error() == kv.KV_ERR_OUT_OF_PAGES
    assert f.lens_d.tolist() == [23, 0, 20]


def test_stale_partly_filled_page(kv):
    f = Filled(kv, [3, 20], seed=29, spare=8, extra_width=8)
    f.tags_d[0, 0] = 5
    new = [4, 4]
    host, dev = _inputs(f, new, 4, 128, 1, 30)
    out = _call(f, new, 4, dev, False)
    assert f.pool.error() == kv.KV_ERR_TAG_MISMATCH
    assert bool((out == 7.0).all()) and f.lens_d.tolist() == [3, 20]


def test_rows_beyond_the_inputs(kv):
    """new_indptr past total_new: an error, and none of that request's rows."""
    f = Filled(kv, [0, 0], seed=31, spare=8, extra_width=8)
    host, dev = _inputs(f, [4, 4], 4, 128, 1, 32)
    before = f.pool.k_cache.clone()
    ind = torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda")
    out = _call(f, [4, 4], 4, dev, False, max_new=8, ind=ind)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    assert bool((out[4:] == 7.0).all())
    p0 = int(f.table_d[0, 0])
    keep = torch.ones(before.shape[0], dtype=torch.bool)
    keep[p0] = False
    assert torch.equal(before.cpu()[keep], f.pool.k_cache.cpu()[keep])


@pytest.mark.parametrize("ind", [[0, 4, 12], [-4, 4, 8], [100000, 100004, 100008], [0, 4, 2]])
def test_rows_outside_the_inputs_are_not_served(kv, ind):
    """No page is popped and no length grows for a request with rows outside the inputs, nor for
    those behind it."""
    f = Filled(kv, [3, 5], seed=47, spare=8, extra_width=8)
    host, dev = _inputs(f, [4, 4], 4, 128, 1, 48)
    before = [x.clone() for x in (f.pool.k_cache, f.pool.v_cache, f.pool.tags, f.table_d)]
    out = _call(f, [4, 4], 4, dev, False, max_new=8, ind=torch.tensor(ind, dtype=torch.int32, device="cuda"))
    first = ind[0] == 0  # request 0 is in order
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    assert f.lens_d.tolist() == [7 if first else 3, 5]
    assert int(f.pool.ctl[0]) == f.free_head
    assert bool((out[4 if first else 0:] == 7.0).all())
    for x, y in zip(before, (f.pool.k_cache, f.pool.v_cache, f.pool.tags, f.table_d)):
        if not (first and x.dim() == 4):
            assert torch.equal(x, y)


def test_axis_out_of_range(kv):
    f = Filled(kv, [0], seed=33, spare=8, extra_width=8)
    host, dev = _inputs(f, [4], 4, 32, 1, 34)
    dev[4][3] = 9
    _call(f, [4], 4, dev, False)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG


def test_captured_and_replayed(kv):
    """A graph of the append, replayed: each replay appends its rows again."""
    f = Filled(kv, [7, 0], hkv=2, seed=35, spare=30, extra_width=10)
    ref = Filled(kv, [7, 0], hkv=2, seed=35, spare=30, extra_width=10)
    new = [9, 20]
    host, dev = _inputs(f, new, 4, 128, 2, 36)
    out = torch.zeros_like(dev[0])
    ind = indptr(new).cuda()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(f, new, 4, dev, False, ind=ind, q_out=out)
    for _ in range(2):
        g.replay()
        _call(ref, new, 4, dev, False, ind=ind)
    torch.cuda.synchronize()
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    assert torch.equal(raw(f.pool.k_cache), raw(ref.pool.k_cache))
    assert torch.equal(raw(f.pool.v_cache), raw(ref.pool.v_cache))
    assert f.lens_d.tolist() == [25, 40] and torch.equal(f.table_d, ref.table_d)
    assert math.isclose(float(out.float().abs().sum()),
                        float(_call(ref, new, 4, dev, False, ind=ind).float().abs().sum()))
