"""paged_prefill_attn's Python call takes q for what num_q_heads says, and no larger row."""
import pytest
import torch

from test_prompt_abi import Recorder, kv  # noqa: F401  (kv: the fixture)


@pytest.mark.parametrize("heads,dim", [(4, 128), (16, 128), (8, 64), (8, 256)])
def test_heads_other_than_the_rows(kv, monkeypatch, heads, dim):  # noqa: F811
    """num_q_heads 8 and rows of another width: rows would be taken from the wrong places."""
    monkeypatch.setattr(kv, "_lib", Recorder())
    monkeypatch.setattr(kv, "_device", lambda: -1)
    monkeypatch.setattr(kv, "_ptr", lambda t, dtype=None, name="": 0)
    i32 = dict(dtype=torch.int32)
    rest = (torch.zeros(3, **i32), torch.zeros(2, 4, **i32), torch.zeros(2, **i32), None, 0.1)
    ws = torch.zeros(256, dtype=torch.uint8)
    q = torch.zeros(6, heads, dim, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.paged_prefill_attn(0, 2, 8, q, *rest, q.clone(), ws, 0)
    for good in (torch.zeros(6, 8, 128, dtype=torch.bfloat16), torch.zeros(6, 1024, dtype=torch.bfloat16)):
        with pytest.raises(AssertionError, match="called"):
            kv.paged_prefill_attn(0, 2, 8, good, *rest, good.clone(), ws, 0)
