"""Decode attention over 4-bit pools where keys, values or queries are no numbers: what reaches a
row, whatever part of its positions a warp has.  Rows that nothing reaches keep the bound of
test_e2m1_attn_gpu."""
import pytest
import torch

from e2m1ref import PLACES, Filled4
from promptref import attention
from test_e2m1_attn_gpu import _queries, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


# query heads, kv heads: 8 rows a warp; 16 (of one, two and three blocks); 32 (of one and two)
SHAPES = [(8, 1), (8, 2), (64, 8), (16, 1), (24, 2), (64, 2), (48, 1), (128, 4), (128, 2)]


def _bounded_rows(f, b, got, q, scale, rows):
    """The bound over the (token, head) pairs of the mask `rows`."""
    n, T = f.lens[b], q.shape[0]
    k, v = f.rows(b, "k"), f.rows(b, "v")
    ref, mag = (attention(torch.where(rows[..., None], q.double(), 0.0), k, x, scale, n - T)
                for x in (v, v.abs()))
    bad = (got.double() - ref).abs() > 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 1e-30
    assert not bool((bad | torch.isnan(got))[rows].any())


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("n", [1, 17, 33, 65, 700])
def test_a_newest_key_that_is_no_number(kv, hq, hkv, n):
    """The newest token's key has a NaN: it may be the only position of a warp's part, or of the
    request.  The kv head's rows are NaN; other heads', and the other request's, are not."""
    f = Filled4(kv, [n, 40], hkv=hkv, seed=41)
    q = _queries(2, 1, hq, 42, 0.5)
    p, slot = int(f.table[0, (n - 1) // 16]), (n - 1) % 16
    f.cache["k"][p, hkv - 1, PLACES["k"][2][slot, 5]] = 0x7F
    f.to_device()
    got = _run(f, q, 0.09)
    assert f.pool.error() == 0
    G = hq // hkv
    assert bool(torch.isnan(got[0, :, -G:]).all())
    f.cache["k"][p, hkv - 1, PLACES["k"][2][slot, 5]] = 0x30
    rows = torch.ones((1, hq), dtype=torch.bool)
    _bounded_rows(f, 1, got[1], q[1], 0.09, rows)
    rows[:, -G:] = False
    _bounded_rows(f, 0, got[0], q[0], 0.09, rows)


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("n", [1, 33, 700])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_no_number(kv, hq, hkv, n, value):
    """Every score of such a row is NaN or infinite: the row is NaN, and no other."""
    f = Filled4(kv, [n, 40], hkv=hkv, seed=43)
    q = _queries(2, 1, hq, 44, 0.5)
    q[0, 0, hq // 2, 77] = value
    got = _run(f, q, 0.09)
    rows = torch.ones((1, hq), dtype=torch.bool)
    _bounded_rows(f, 1, got[1], q[1], 0.09, rows)
    assert bool(torch.isnan(got[0, 0, hq // 2]).all())
    rows[0, hq // 2] = False
    _bounded_rows(f, 0, got[0], q[0], 0.09, rows)


@pytest.mark.parametrize("hq,hkv", [(4, 2), (24, 2), (64, 4)])
def test_drafts_before_the_bad_key_and_rows_that_see_nothing(kv, hq, hkv):
    """Four tokens over three positions: the first sees none (zeros), the second and third do not
    see the newest key, which has a NaN; the last does."""
    f = Filled4(kv, [3], hkv=hkv, seed=45)
    q = _queries(1, 4, hq, 46, 0.5)
    q[0, 0, 0, 0] = float("nan")  # (a row that sees nothing is zero whatever its query is)
    p = int(f.table[0, 0])
    for h in range(hkv):
        f.cache["k"][p, h, PLACES["k"][2][2, 0]] = 0x7F
    f.to_device()
    got = _run(f, q, 0.09)[0]
    assert not got[0].any() and bool(torch.isnan(got[3]).all())
    for h in range(hkv):
        f.cache["k"][p, h, PLACES["k"][2][2, 0]] = 0x30
    rows = torch.zeros((4, hq), dtype=torch.bool)
    rows[1:3] = True
    _bounded_rows(f, 0, got, q[0], 0.09, rows)


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("exp", [40, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_keys_of_far_scores(kv, hq, hkv, exp, sign):
    """All keys are alike and every score is 1.5 * 2^exp (as a power of 2's exponent), to which no page's
    V block scale can be added in fp32: each position has the same weight, whatever part it is in."""
    n = 1600
    f = Filled4(kv, [n], hkv=hkv, seed=48)
    for j, p in enumerate(f.table[0, :n // 16]):
        f.cache["k"][p][:, :1024] = 0x22  # 1
        f.cache["k"][p][:, 1024:] = 0x38  # times 1
        f.scale["k"][p] = 1.0
        f.scale["v"][p] = 2.0 ** (-20 if j < 40 else 0 if j < 70 else 15)
    f.to_device()
    q = torch.full((1, 1, hq, 128), sign * 2.0 ** 20, dtype=torch.bfloat16)
    got = _run(f, q, 1.5 * 2.0 ** (exp - 20 - 7) * 0.6931471805599453)
    G = hq // hkv
    v = f.rows(0, "v")
    ref, mag = (x.mean(0).repeat_interleave(G, 0) for x in (v, v.abs()))
    assert bool(((got[0, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag).all())


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("n", [1, 40, 700])
def test_scores_next_to_the_lowest(kv, hq, hkv, n):
    """All keys are alike and every score is -1.5 * 2^127 (as a power of 2's exponent; fp32's lowest is
    -2 * 2^127): each position has the same weight."""
    f = Filled4(kv, [n], hkv=hkv, seed=47)
    for p in f.table[0, :-(-n // 16)]:
        f.cache["k"][p][:, :1024] = 0x22  # 1
        f.cache["k"][p][:, 1024:] = 0x38  # times 1
        f.scale["k"][p] = 2.0 ** 13
    f.to_device()
    q = torch.full((1, 1, hq, 128), -2.0 ** 100, dtype=torch.bfloat16)
    got = _run(f, q, 1.5 * 2.0 ** (127 - 100 - 13 - 7) * 0.6931471805599453)
    G = hq // hkv
    v = f.rows(0, "v")
    ref, mag = (x.mean(0).repeat_interleave(G, 0) for x in (v, v.abs()))
    assert bool(((got[0, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag).all())


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("which,value", [("k", float("nan")), ("v", float("nan")), ("v", float("inf")), ("v", -1.0)])
@pytest.mark.parametrize("page", [0, 20, 43])
def test_a_block_scale_that_is_no_number(kv, hq, hkv, which, value, page):
    """The kv head's rows, which all see the page, are NaN, and no others."""
    f = Filled4(kv, [700, 40], hkv=hkv, seed=49)
    q = _queries(2, 1, hq, 50, 0.5)
    p, G = int(f.table[0, page]), hq // hkv
    was = f.scale[which][p, 0]
    f.scale[which][p, 0] = value
    f.to_device()
    got = _run(f, q, 0.09)
    f.scale[which][p, 0] = was
    assert bool(torch.isnan(got[0, 0, :G]).all())
    rows = torch.ones((1, hq), dtype=torch.bool)
    _bounded_rows(f, 1, got[1], q[1], 0.09, rows)
    rows[0, :G] = False
    _bounded_rows(f, 0, got[0], q[0], 0.09, rows)
