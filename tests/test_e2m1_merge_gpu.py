"""4-bit decode attention: a V that is no number reaches every row that sees it, however far below
the row's largest weight its own is, and whichever warp met it."""
import pytest
import torch

from e2m1ref import PLACES, Filled4
from test_e2m1_attn_gpu import _queries, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


@pytest.mark.parametrize("hq,hkv,row", [(8, 1, 3), (64, 8, 0), (16, 1, 9), (48, 1, 40), (128, 4, 17)])
@pytest.mark.parametrize("where", [0, 600, 999])
def test_weights_of_zero(kv, hq, hkv, row, where):
    """One row's weights are 1 for a key and below 2^-160 for all others, so that an fp32 factor
    between two parts of the request is 0."""
    f = Filled4(kv, [1000], hkv=hkv, seed=51, spread=0)
    p, slot = int(f.table[0, where // 16]), where % 16
    f.cache["k"][p, 0, PLACES["k"][2][slot]] = 0x50  # 8: the others are below 2
    far = (where + 500) % 1000
    f.cache["v"][int(f.table[0, far // 16]), 0, PLACES["v"][2][far % 16, 3]] = 0x7F
    f.to_device()
    q = _queries(1, 1, hq, 52, 0.02)
    keys = f.rows(0, "k")[:, 0]
    k = keys[where]
    q[0, 0, row] = (k * (300.0 / float(k @ k) / 0.09)).to(torch.bfloat16)
    score = keys @ q[0, 0, row].double() * 0.09
    top = float(score[where])
    score[where] = -1e9
    assert (top - float(score.max())) * 1.4427 > 160
    got = _run(f, q, 0.09)[0, 0]
    G = hq // hkv
    want = torch.zeros((hq, 128), dtype=torch.bool)
    want[:G, 48:64] = True
    assert torch.equal(torch.isnan(got), want)
    v = f.rows(0, "v")[where, 0]
    keep = [d for d in range(128) if not 48 <= d < 64]
    assert bool(((got[row].double() - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -10 * v.abs().max())[keep].all())
