"""Row offsets that run backwards in the middle of a batch, for the three prompt-side operators:
the requests before such a place get what they would get alone, that request and those behind it
nothing, and the error word says so.  Errors of a request do not depend on where its rows lie.

Bounds of the values are those of the operators' own tests."""
import pytest
import torch

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
