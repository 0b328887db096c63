"""paged_prefill_attn where values are extreme: rows that are no numbers, V scales of zero and
near fp32's ends, weights far below a row's largest, weights of a bf16 pool that nearly cancel.

Bound of an output o = sum_j p_j v_j / sum_j p_j against the 64-bit form, A = sum_j p_j |v_j| /
sum_j p_j, S = the row's largest sum over dims of |q k| in log2 units (after scaling), L the
length:
  bf16 output       2^-8 |o|, and half the smallest step, 2^-134
  weights (e4m3)    f16: 2^-11 of each, or half of f16's smallest step (2^-25) where that is more:
                    the reference is 2^6 or more below a row's largest p * (V scale), so at most
                    2^-31 of that largest, for every key, times its code
  weights (bf16)    two bf16 parts: 2^-8 of the second, which is 2^-8 of the weight: 2^-16 A
  scores            128 products of exact factors (e4m3: f16 holds both; bf16) summed in fp32, and
                    three roundings of the exponent: 132 * 2^-24 S; ln 2 times that is the
                    weight's, and the sum's again; exp2 adds 2^-22, twice: 2^-21
  smallest weights  fp32 has no normal values below 2^-126, and exp2 gives zero there: a weight
                    below 2^-125 of the sum (which is at least half of its own reference) may be
                    left out: 2^-125 |v_j| for every key
  sums              L terms, each at most 2^-23 off its sum (the tensor cores may cut), in o and
                    in the sum of the weights; 64 more for rescaling and merging: (L + 64) 2^-22
"""
import math

import pytest
import torch

from promptref import Filled, attention, e4m3_values, indptr

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _queries(new, hq, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((sum(new), hq, 128), generator=g) * scale).to(torch.bfloat16)


def _load(f):
    """The pool's device copies of what a test has changed."""
    f.pool.k_cache.copy_(f.k)
    f.pool.v_cache.copy_(f.v)
    if f.fp8:
        f.pool.k_scale.copy_(f.ks)
        f.pool.v_scale.copy_(f.vs)


def _run(f, q, new, copies=1):
    """The outputs; with `copies`, [copies][rows][heads][dim] of as many requests that share the
    pages of f's one (so many items that few are cut)."""
    q = q.repeat(copies, 1, 1)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((f.pool.prefill_workspace_size(f.B * copies, q.shape[1], q.shape[0]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(f.B * copies, q.shape[1], q.cuda(), indptr(new * copies).cuda(),
                        f.table_d.repeat(copies, 1), f.lens_d.repeat(copies), None, SCALE, out, ws)
    got = out.cpu().double()
    assert f.pool.error() == 0
    return got if copies == 1 else got.unflatten(0, (copies, -1))


def _codes(f, b):
    """|V| of request b in units of its pages' scales, [L][heads][dim]."""
    at = torch.arange(f.lens[b])
    c = f.v[f.table[b].long()[at // 16], :, :, at % 16]
    return e4m3_values()[c.long()].abs()


def _check(f, q, new, got, rows=None):
    """`rows`: a truth value for each (query row, head) that is looked at."""
    ind = indptr(new)
    for b in range(f.B):
        lo, hi = int(ind[b]), int(ind[b + 1])
        if lo == hi:
            continue
        qb, k, v, L = q[lo:hi].double(), f.rows(b, "k"), f.rows(b, "v"), f.lens[b]
        old = L - (hi - lo)
        ref, mag = attention(qb, k, v, SCALE, old), attention(qb, k, v.abs(), SCALE, old)
        g = q.shape[1] // f.hkv
        big = torch.einsum("nhd,lhd->hnl", qb.abs(), k.abs().repeat_interleave(g, 1)).amax(-1)
        S = big.t()[..., None] * SCALE / math.log(2)  # [n][Hq][1]
        c = (2 * math.log(2) * 132 * 2.0 ** -24 * S + 2.0 ** -21 + (L + 64) * 2.0 ** -22
             + (2.0 ** -11 if f.fp8 else 2.0 ** -16))
        bound = 2.0 ** -8 * ref.abs() + c * mag + 2.0 ** -134
        if f.fp8:
            s = torch.einsum("nhd,lhd->hnl", qb, k.repeat_interleave(g, 1)) * SCALE
            see = torch.arange(L)[None] <= old + torch.arange(hi - lo)[:, None]
            s = s.masked_fill(~see[None], -math.inf)
            vs = f.vs[f.table[b].long()[torch.arange(L) // 16]].double()
            p = torch.softmax(s, -1)
            top = (p * vs.t().repeat_interleave(g, 0)[:, None]).amax(-1).t()[..., None]  # [n][Hq][1]
            codes = torch.einsum("nl,lhd->nhd", see.double(), _codes(f, b)).repeat_interleave(g, 1)
            values = torch.einsum("nl,lhd->nhd", see.double(), v.abs()).repeat_interleave(g, 1)
            bound = bound + 2.0 ** -31 * top * codes + 2.0 ** -125 * values
        err = (got[..., lo:hi, :, :] - ref).abs() / bound
        if rows is not None:
            err = err[rows[lo:hi]]
        assert bool((err <= 1.0).all()), (b, float(err.max()))


# (lengths with the new tokens, new tokens, query heads, kv heads): an item of one tile, of two,
# and items that are cut over CTAs
KINDS = {
    "one tile": ([300], [16], 8, 1),
    "two tiles": ([290], [64], 8, 2),
    "two requests": ([200, 70], [3, 40], 8, 2),
    "single token, cut": ([9000], [1], 8, 1),
    "cut": ([2600], [130], 16, 2),
    "a query head each": ([400], [300], 2, 2),
}


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("kind", list(KINDS))
def test_queries_that_are_no_numbers(kv, kind, fp8):
    """A query of NaN or infinities has weights that are no numbers: its row is NaN, whole, and
    every other is right."""
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, fp8=fp8, seed=201)
    q = _queries(new, hq, 202)
    t = q.shape[0]
    bad = torch.zeros(t, hq, dtype=torch.bool)
    for i, (row, head, x) in enumerate(((0, 1, math.nan), (t // 2, hq - 1, math.inf), (t - 1, hq // 2, -math.inf))):
        q[row, head, 5 * i] = x
        bad[row, head] = True
    got = _run(f, q, new)
    assert bool(torch.isnan(got[bad]).all())
    clean = q.clone()
    clean[bad] = 0
    _check(f, clean, new, got, ~bad)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("what", ["key", "scale"])
@pytest.mark.parametrize("at", [0, 70, 130, -3])
@pytest.mark.parametrize("kind", list(KINDS))
def test_keys_that_are_no_numbers(kv, kind, at, what, fp8):
    """One key with a NaN, or a page whose K scale is one: the rows that see it are NaN, whole, and
    the others are right."""
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, fp8=fp8, seed=203)
    at = at % lens[0]
    page, head = int(f.table[0, at // 16]), hkv - 1
    clean = (f.k.clone(), None if f.ks is None else f.ks.clone())
    if what == "key":
        f.k[page, head, at % 16, 9] = 0x7F if fp8 else math.nan
    elif fp8:
        f.ks[page, head] = math.nan
        at = at // 16 * 16
    else:
        pytest.skip("a bf16 pool has no scales")
    _load(f)
    q = _queries(new, hq, 204)
    got = _run(f, q, new)
    g = hq // hkv
    bad = torch.zeros(q.shape[0], hq, dtype=torch.bool)
    sees = torch.arange(new[0]) + lens[0] - new[0] >= at
    bad[:new[0], head * g:] = sees[:, None]
    assert bool(bad.any()) and bool(torch.isnan(got[bad]).all())
    f.k, f.ks = clean
    _check(f, q, new, got, ~bad)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -130, 1e-38, 1e-20, 1e34])
@pytest.mark.parametrize("first", [64, 304])
@pytest.mark.parametrize("lead", [1.0, 30.0])
@pytest.mark.parametrize("kind", list(KINDS))
def test_scales_of_leading_pages(kv, kind, lead, first, scale):
    """V scales of zero, below and near fp32's smallest, or near its largest over whole units of
    pages at a request's begin, whose keys score like the others' or far higher and lower: their
    weights count in the sum whatever their values are."""
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, seed=205)
    for b in range(f.B):
        pages = f.table[b, :min(first, (lens[b] - 1) // 16 * 16) // 16].long()
        f.vs[pages] = scale
        f.ks[pages] *= lead
    _load(f)
    q = _queries(new, hq, 206)
    _check(f, q, new, _run(f, q, new))


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -130, 1e-37, 1e-20, 1e34])
@pytest.mark.parametrize("kind", list(KINDS))
def test_scales_of_every_page(kv, kind, scale):
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, seed=207)
    f.vs.fill_(scale)
    _load(f)
    q = _queries(new, hq, 208)
    _check(f, q, new, _run(f, q, new))


@pytest.mark.parametrize("kind", list(KINDS))
def test_scales_far_apart_anywhere(kv, kind):
    """Scales of every size from 2^-130 to 2^110, page by page in any order."""
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, seed=209)
    g = torch.Generator().manual_seed(210)
    f.vs = torch.exp2(torch.randint(-130, 111, f.vs.shape, generator=g).float())
    f.ks *= torch.exp2(torch.randint(-3, 5, f.ks.shape, generator=g).float())
    _load(f)
    q = _queries(new, hq, 211)
    _check(f, q, new, _run(f, q, new))


@pytest.mark.parametrize("nats", [10.0, 18.0])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("at", [0, 2500])
def test_a_key_far_above_the_rest(kv, at, new, nats):
    """A key of value zero that leads by 10 or 18 nats: what the others, 2^-26 of it each, add up to
    is the whole output."""
    L = 6000
    f = Filled(kv, [L], hkv=1, seed=213)
    f.k[f.table[0, :L // 16].long(), :, :, 0] = 0  # no other key has a part of dim 0
    f.ks.fill_(1e-4)
    page = int(f.table[0, at // 16])
    f.k[page] = 0
    f.k[page, 0, at % 16, 0] = 0x38  # 1.0
    f.ks[page] = 1.0
    f.v &= 0x7F  # all other values are positive
    f.v[f.v == 0x7F] = 0x7E
    f.v[page, :, :, at % 16] = 0
    f.vs.fill_(0.01)
    _load(f)
    q = _queries([new], 8, 214, 0.01)
    q[..., 0] = nats / SCALE
    _check(f, q, [new], _run(f, q, [new], copies=152))


@pytest.mark.parametrize("at", [3, 400])
def test_a_page_of_a_large_scale(kv, at):
    """A page whose scale one outlier has made 2^12 times the others'."""
    f = Filled(kv, [6000], hkv=1, seed=215)
    page = int(f.table[0, at // 16])
    f.vs.fill_(0.01)
    f.vs[page] = 0.01 * 2 ** 12
    f.v[page] = 0x08  # 2^-6: as large as the others' there
    f.v[page, 0, 7, at % 16] = 0x7E
    _load(f)
    q = _queries([50], 8, 216, 2.0)
    _check(f, q, [50], _run(f, q, [50]))


@pytest.mark.parametrize("new", [1, 16, 60])
@pytest.mark.parametrize("steps", [-16.8, -2.8, -0.9, 1.8])
def test_bf16_weights_that_nearly_cancel(kv, new, steps):
    """Two kinds of keys whose weights lie less than half a bf16 step apart, with values +1 and -1:
    the output is the difference."""
    L = 320
    f = Filled(kv, [L], hkv=1, fp8=False, seed=217)
    for j in range(L):
        page = int(f.table[0, j // 16])
        f.k[page, 0, j % 16] = 0
        f.v[page, 0, :, j % 16] = 1.0 if j % 2 else -1.0
        if j % 2:
            f.k[page, 0, j % 16, 0] = 1.0
    _load(f)
    q = torch.zeros((new, 8, 128), dtype=torch.bfloat16)
    q[..., 0] = math.log1p(steps * 2.0 ** -9) / SCALE
    _check(f, q, [new], _run(f, q, [new]))


@pytest.mark.parametrize("what", ["nan", "inf", "scale nan", "scale inf"])
@pytest.mark.parametrize("back", [1, 7, 15])
@pytest.mark.parametrize("kind", [k for k in KINDS if k != "single token, cut"])
@pytest.mark.parametrize("fp8", [True, False])
def test_values_behind_the_mask(kv, fp8, kind, back, what):
    """A value that is not finite reaches its own dim of the rows that see its position, and nothing
    of the rows before it; nor does a page's V scale that is not."""
    if (what == "inf") if fp8 else ("scale" in what):
        pytest.skip("e4m3 has no infinities, a bf16 pool no scales")
    lens, new, hq, hkv = KINDS[kind]
    b = len(lens) - 1
    f = Filled(kv, lens, hkv=hkv, fp8=fp8, seed=219)
    at = lens[b] - back
    if "scale" in what:
        at = (lens[b] - 1) // 16 * 16  # the last page's first token
    page, head, g = int(f.table[b, at // 16]), hkv - 1, hq // hkv
    clean = (f.v.clone(), None if f.vs is None else f.vs.clone())
    if "scale" in what:
        f.vs[page, head] = math.nan if "nan" in what else math.inf
    else:
        f.v[page, head, 77, at % 16] = 0x7F if fp8 else math.nan if what == "nan" else math.inf
        f.v[page, head, 3, at % 16] = 0xFF if fp8 else -math.inf
    _load(f)
    q = _queries(new, hq, 220)
    got = _run(f, q, new)
    f.v, f.vs = clean
    sees = torch.arange(new[b]) + lens[b] - new[b] >= at
    rows = torch.zeros(q.shape[0], hq, dtype=torch.bool)
    rows[-new[b]:, head * g:] = sees[:, None]
    assert bool(rows.any()) and not bool(rows.all())
    _check(f, q, new, got, ~rows)
    if "scale" in what:
        assert bool(torch.isnan(got[rows]).all())
        return
    assert not bool(torch.isfinite(got[rows][:, [3, 77]]).any())
    got[..., [3, 77]] = 0  # every other dim is right
    f.v[:, :, [3, 77]] = 0
    _check(f, q, new, got, rows)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("kind", list(KINDS))
def test_values_anywhere_that_are_not_finite(kv, kind, fp8):
    """Values that are not finite at several positions, one of them seen by (nearly) every row, three
    dims of a head at each: an output is finite where its row sees none of its dim, and right."""
    lens, new, hq, hkv = KINDS[kind]
    f = Filled(kv, lens, hkv=hkv, fp8=fp8, seed=221)
    g = torch.Generator().manual_seed(222)
    clean = f.v.clone()
    first = torch.full((f.B, hkv, 128), 1 << 30)  # the first such position of each dim
    for b in range(f.B):
        backs = [k for k in (1, 4, 11, 30, 77, 130, 290) if k == 1 or k <= new[b]]
        for at in [*(lens[b] - k for k in backs), lens[b] // 3]:
            h, d = int(torch.randint(0, hkv, (), generator=g)), torch.randint(0, 128, (3,), generator=g)
            page = int(f.table[b, at // 16])
            f.v[page, h, d, at % 16] = 0x7F if fp8 else math.nan if at % 2 else -math.inf
            clean[page, h, d, at % 16] = 0
            first[b, h, d] = torch.clamp_max(first[b, h, d], at)
    _load(f)
    q = _queries(new, hq, 223)
    got = _run(f, q, new)
    f.v = clean
    ind = indptr(new)
    bad = torch.zeros(got.shape, dtype=torch.bool)
    for b in range(f.B):
        last = torch.arange(new[b]) + lens[b] - new[b]  # the last position each row sees
        bad[ind[b]:ind[b + 1]] = (first[b] <= last[:, None, None]).repeat_interleave(hq // hkv, 1)
    assert bool(bad.any()) and not bool(bad.all())
    assert not bool(torch.isfinite(got[bad]).any())
    assert bool(torch.isfinite(got[~bad]).all())
    # (where they belong, the reference takes their place)
    _check(f, q, new, torch.where(bad, _reference(f, q, new), got))


def _reference(f, q, new):
    ind = indptr(new)
    return torch.cat([attention(q[ind[b]:ind[b + 1]].double(), f.rows(b, "k"), f.rows(b, "v"), SCALE,
                                f.lens[b] - new[b]) for b in range(f.B)])
