"""4-bit decode attention over pages whose V block scales lie far apart.

A V block scale says nothing about a token's weight, so the bound of test_e2m1_attn_gpu holds for
each dim by itself: weights in f16 are relative to the row's largest weight alone, a code times its
group's scale is exact with any of the powers of two that bring pages together, and so is moving
sums from one such power to another.  Pages 2^60 below the largest keep all of this.  What lies
further below may be left out, as much as 2^-56 of the largest value (and is off by no more)."""
import numpy as np
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


SHAPES = [(8, 1), (16, 2), (16, 1), (48, 1), (128, 4)]


def _check(f, q, got, left_out=0.0):
    for b, n in enumerate(f.lens):
        k, v = f.rows(b, "k"), f.rows(b, "v")
        ref, mag = (attention(q[b].double(), k, x, 0.09, n - q.shape[1]) for x in (v, v.abs()))
        err = (got[b].double() - ref).abs()
        bound = 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + left_out * v.abs().max()
        assert bool((err <= bound).all()), (b, float((err / bound).nan_to_num(0).max()))


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("exp", [-12, -18, -27, -50])
@pytest.mark.parametrize("which", ["one", "some", "last"])
def test_pages_of_zeros(kv, hq, hkv, exp, which):
    """A page whose V rows are all zero has the block scale 1; it adds nothing but its weights."""
    f = Filled4(kv, [960, 100], hkv=hkv, seed=61, spread=1)
    f.scale["v"] *= np.float32(2.0 ** exp)
    zero = {"one": [0], "some": range(0, 60, 7), "last": [59]}[which]
    for j in zero:
        f.cache["v"][f.table[0, j]] = 0
        f.scale["v"][f.table[0, j]] = 1.0
    f.to_device()
    q = _queries(2, 1, hq, 62, 0.5)
    _check(f, q, _run(f, q, 0.09))


def _spread_pages(f, kinds, exps):
    """Page j of request 0 has block scale 2^exps[kind], and values other than zero in the first
    16, 32 or 128 dims for the kinds 0, 1 and 2."""
    scale = PLACES["v"][2]
    for j, kind in enumerate(kinds):
        p = f.table[0, j]
        f.scale["v"][p] = np.float32(2.0 ** exps[kind])
        for c in range((1, 2, 8)[kind], 8):
            f.cache["v"][p][:, scale[:, c]] = 0
    f.to_device()


def _kinds(order, pages, rng):
    kinds = rng.integers(0, 3, pages)
    return {"mixed": kinds, "up": np.sort(kinds)[::-1], "down": np.sort(kinds)}[order]


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("exps", [(0, -10, -20), (10, -5, -20), (0, -20, -58), (100, 70, 42), (-42, -70, -100)])
@pytest.mark.parametrize("order", ["mixed", "up", "down"])
def test_block_scales_far_apart(kv, hq, hkv, exps, order):
    rng = np.random.default_rng(63)
    f = Filled4(kv, [1600], hkv=hkv, seed=64)
    _spread_pages(f, _kinds(order, 100, rng), exps)
    q = _queries(1, 1, hq, 65, 0.5)
    _check(f, q, _run(f, q, 0.09))


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("order", ["mixed", "up", "down"])
def test_block_scales_further_apart(kv, hq, hkv, order):
    rng = np.random.default_rng(66)
    f = Filled4(kv, [1600], hkv=hkv, seed=67)
    _spread_pages(f, _kinds(order, 100, rng), (110, 0, -100))
    q = _queries(1, 1, hq, 68, 0.5)
    _check(f, q, _run(f, q, 0.09), 2.0 ** -56)


@pytest.mark.parametrize("hq,hkv", SHAPES)
def test_block_scales_at_the_ends(kv, hq, hkv):
    """All of a request's V at 2^121 (values up to 2^127) or at 2^-100: no sum leaves fp32."""
    for exp in (121, -100):
        f = Filled4(kv, [700, 1], hkv=hkv, seed=69)
        f.scale["v"][:] = np.float32(2.0 ** exp)
        if exp > 0:  # group scales up to 10: 6 * 10 * 2^121
            sc = PLACES["v"][2]
            f.cache["v"][:, :, sc] = np.where(f.cache["v"][:, :, sc] == 0x7F, 0x7F, f.cache["v"][:, :, sc] + 0x13)
        f.to_device()
        q = _queries(2, 1, hq, 70, 0.5)
        got = _run(f, q, 0.09)
        assert bool(torch.isfinite(got).all())
        _check(f, q, got)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (128, 4)])
def test_far_scales_and_a_value_that_is_no_number(kv, hq, hkv):
    """Whatever power of two a page is brought by: NaN stays in its group's dims."""
    rng = np.random.default_rng(71)
    f = Filled4(kv, [1600], hkv=hkv, seed=72)
    _spread_pages(f, _kinds("mixed", 100, rng), (90, 0, -90))
    f.cache["v"][f.table[0, 50], 0, PLACES["v"][2][3, 6]] = 0x7F
    f.to_device()
    got = _run(f, _queries(1, 1, hq, 73, 0.5), 0.09)[0, 0]
    want = torch.zeros((hq, 128), dtype=torch.bool)
    want[:hq // hkv, 96:112] = True
    assert torch.equal(torch.isnan(got), want)


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("exp", [-10, -12, -13, -14, -15, -16, -17])
def test_the_smallest_values_of_pages_below_others(kv, hq, hkv, exp):
    """Pages 2^exp below the others with the smallest group scales, subnormal ones among them: the
    others are zero there, so every bit of those values counts."""
    rng = np.random.default_rng(74)
    f = Filled4(kv, [1600], hkv=hkv, seed=75)
    _spread_pages(f, np.arange(100) % 3 // 2 * 2, (0, 0, exp))  # every third
    scale = PLACES["v"][2]
    for j in range(2, 100, 3):
        p = f.table[0, j]
        f.cache["v"][p][:, scale[:, 1:]] = rng.integers(0, 16, (hkv, 16, 7))
    f.to_device()
    q = _queries(1, 1, hq, 76, 0.5)
    _check(f, q, _run(f, q, 0.09))
