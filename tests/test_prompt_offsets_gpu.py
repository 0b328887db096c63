"""Row offsets that run backwards in the middle of a batch, for the three prompt-side operators:
the requests before such a place get what they would get alone, that request and those behind it
nothing, and the error word says so.  Errors of a request do not depend on where its rows lie.

Bounds of the values are those of the operators' own tests."""
import pytest
import torch

import test_prompt_prefill_gpu as attn
import test_prompt_read_gpu as read
import test_prompt_rotary_gpu as rotary
from promptref import Filled, indptr
from test_prompt_read_gpu import kv  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# (offsets, requests served): decreases behind a request of many pages, to a negative entry, behind
# two requests, at once, and in a batch of more requests than a warp's lanes
BACKWARDS = [
    ([0, 200, 10, 20], 1),
    ([0, 200, 10, 200], 1),
    ([0, 64, -100, 40], 1),
    ([0, 100, 180, 3, 90], 2),
    ([0, 200, 200, 100, 100, 200], 2),
    ([150, 10, 200], 0),
    ([*range(0, 120, 3), 40, 50, 200], 39),
    ([*range(0, 150), 20, *range(30, 60), 200], 149),
]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("ind,served", BACKWARDS)
def test_rotary(kv, ind, served, fp8):  # noqa: F811
    B = len(ind) - 1
    f = Filled(kv, [3] * B, hkv=2, fp8=fp8, seed=301, spare=300, extra_width=20)
    new = [b - a for a, b in zip(ind, ind[1:])][:served]
    rows = [0] * B
    rows[0] = 200  # the inputs have 200 rows
    host, dev = rotary._inputs(f, rows, 4, 128, 2, 302)
    out = rotary._call(f, rows, 4, dev, False, max_new=200, ind=_i32(ind))
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    assert f.lens_d.tolist() == [3 + n for n in new] + [3] * (B - served)
    assert int(f.pool.ctl[kv.KV_CTL_APPEND_STOP]) == served
    rotary._check(f, new + [0] * (B - served), host, out, False, served=served)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("ind,served", BACKWARDS)
def test_read(kv, ind, served, fp8):  # noqa: F811
    B = len(ind) - 1
    f = Filled(kv, [200] * B, hkv=2, fp8=fp8, seed=303)
    k = torch.full((200, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    f.pool.read_rows(B, f.table_d, f.lens_d, None, _i32(ind), None, k, v)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    f.B = served
    read._check(f, [0] * served, torch.tensor(ind[:served + 1]) if served else indptr([0]), k, v)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [(8, 1), (2, 2)])
@pytest.mark.parametrize("ind,served", BACKWARDS)
def test_attention(kv, ind, served, heads, fp8):  # noqa: F811
    B, (hq, hkv) = len(ind) - 1, heads
    f = Filled(kv, [210] * B, hkv=hkv, fp8=fp8, seed=305)
    q = attn._queries(f, [200], hq, 306)
    out = torch.full((200, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(f.pool.prefill_workspace_size(B, hq, 200), dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(B, hq, q.cuda(), _i32(ind), f.table_d, f.lens_d, None, attn.SCALE, out, ws)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    f.B = served
    new = [b - a for a, b in zip(ind, ind[1:])][:served]
    attn._check(f, q, new, out)


@pytest.mark.parametrize("aborted", [[0, 0], [1, 0]])
@pytest.mark.parametrize("ind", [[0, 100000, 100040], [100000, 100000, 100040], [0, 0, 100040], [0, 80, 10 ** 9]])
def test_rows_far_behind_the_arrays(kv, ind, aborted):  # noqa: F811
    """A request whose rows begin or end behind every work item is reported, also behind one that is
    aborted or has no rows."""
    ab = torch.tensor(aborted, dtype=torch.uint8, device="cuda")
    f = Filled(kv, [60, 60], hkv=2, seed=307)
    k = torch.full((80, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    f.pool.read_rows(2, f.table_d, f.lens_d, None, _i32(ind), ab, k, v)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    assert bool((k == 7.0).all()) and bool((v == 7.0).all())
    f = Filled(kv, [90, 90], hkv=2, seed=308)
    q, out = torch.zeros((80, 4, 128), dtype=torch.bfloat16, device="cuda"), k.new_full((80, 4, 128), 7.0)
    ws = torch.empty(f.pool.prefill_workspace_size(2, 4, 80), dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(2, 4, q, _i32(ind), f.table_d, f.lens_d, ab, attn.SCALE, out, ws)
    assert f.pool.error() == kv.KV_ERR_INVALID_ARG
    assert bool((out[ind[1] if ind[1] <= 80 and not aborted[0] else 0:] == 7.0).all())


def test_aborted_requests_with_bad_rows_are_not_reported(kv):  # noqa: F811
    ab = torch.tensor([1, 0], dtype=torch.uint8, device="cuda")
    f = Filled(kv, [60, 60], hkv=2, seed=309)
    f.lens_d[0] = 10 ** 6
    k = torch.full((80, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    f.pool.read_rows(2, f.table_d, f.lens_d, None, _i32([0, 40, 80]), ab, k, v)
    assert f.pool.error() == 0 and bool((k[:40] == 7.0).all()) and not bool((k[40:] == 7.0).all())
    q, out = torch.zeros((80, 4, 128), dtype=torch.bfloat16, device="cuda"), k.new_full((80, 4, 128), 7.0)
    ws = torch.empty(f.pool.prefill_workspace_size(2, 4, 80), dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(2, 4, q, _i32([0, 40, 80]), f.table_d, f.lens_d, ab, attn.SCALE, out, ws)
    assert f.pool.error() == 0 and bool((out[:40] == 7.0).all()) and bool((out[40:60] != 7.0).any())
