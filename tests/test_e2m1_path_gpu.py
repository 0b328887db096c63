"""The 4-bit pools' operators run together as a server runs them: prompts normalised, turned and
appended into a bf16 pool and attended there, handed to a 4-bit pool, decode turns of normalised
appends, tag check and attention over it (captured too), rows handed back, pages released and
taken again.

Each stage is held against the 64-bit form of its own inputs as they lie on the device, with the
bounds of its operator's own tests: attention over 4 bits as in test_e2m1_attn_gpu.py (its inputs'
scores: heads normalised with weights up to 2 in magnitude have norms of at most 2 * 128^0.5 and
the terms of a product sum to at most 2^9), over bf16 as in test_prompt_path_gpu.py, queries as in
test_norm_rotary_gpu.py."""
import numpy as np
import pytest
import torch

from e2m1ref import Filled4, values
from promptref import Filled, attention, indptr, rotate
from test_norm_rotary_gpu import _normed
from test_prompt_rotary_gpu import _pair_len

pytestmark = pytest.mark.gpu
SCALE, EPS = 128 ** -0.5, 1e-6


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


class Turn:
    """New tokens of every request, the queries, keys and values of one projection."""

    def __init__(self, new, hq, hkv, seed):
        g = torch.Generator().manual_seed(seed)
        t, width = sum(new), (hq + 2 * hkv) * 128
        self.new, self.hq = new, hq
        self.x = torch.randn((t, width), generator=g).to(torch.bfloat16).cuda()
        at = [0, hq * 128, (hq + hkv) * 128, width]
        self.q, self.k, self.v = (self.x[:, a:b].unflatten(1, (-1, 128)) for a, b in zip(at, at[1:]))
        self.w = [torch.empty(128).uniform_(-2.0, 2.0, generator=g).to(torch.bfloat16).cuda() for _ in "qk"]
        self.pos = torch.randint(0, 3000, (2, t), generator=g, dtype=torch.int32).cuda()
        self.axis = (torch.arange(64) % 2).to(torch.uint8).cuda()
        self.freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
        self.ind = indptr(new).cuda()
        self.q_out = torch.full((t, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")

    def append(self, f):
        f.pool.append_norm_rotary(f.B, self.hq, self.q, self.k, self.v, self.ind, max(self.new), self.pos,
                                  self.axis, self.freq, False, *self.w, EPS, self.q_out, f.table_d, f.tags_d,
                                  f.lens_d)

    def check_q(self):
        x = _normed(self.q.cpu(), self.w[0].cpu(), EPS)
        ref = rotate(x, self.pos.cpu(), self.axis.cpu(), self.freq.cpu(), False)
        err = (self.q_out.cpu().double() - ref).abs()
        assert bool((err <= 2.0 ** -18 * _pair_len(x, 128, False) + 2.0 ** -8 * ref.abs() + 1e-38).all())


def _rows4(f, b, which):
    """Request b's rows as the device holds them, fp64."""
    n = int(f.lens_d[b])
    pg = f.table_d[b, :-(-n // 16)].long()
    tile = getattr(f.pool, which + "_cache")[pg].cpu().numpy()
    x = values(tile, getattr(f.pool, which + "_scale")[pg].cpu().numpy(), which)
    return torch.from_numpy(x.transpose(0, 2, 1, 3).reshape(-1, f.hkv, 128)[:n].copy())


def _check4(f, got, q, live=None):
    for b in range(f.B):
        if live is not None and not live[b]:
            continue
        k, v = _rows4(f, b, "k"), _rows4(f, b, "v")
        ref, mag = (attention(q[b].double(), k, x, SCALE, k.shape[0] - q.shape[1]) for x in (v, v.abs()))
        err = (got[b].double() - ref).abs()
        assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 1e-30).all()), b


@pytest.mark.parametrize("hq,hkv", [(8, 2), (36, 3)])
def test_prompts_to_answers(kv, hq, hkv):
    lens = [300, 17, 1, 64]
    src = Filled(kv, [0] * 4, hkv=hkv, fp8=False, seed=1, spare=60, extra_width=30)
    p = Turn(lens, hq, hkv, 2)
    p.append(src)
    out = torch.zeros_like(p.q_out)
    ws = torch.empty(src.pool.prefill_workspace_size(4, hq, sum(lens)), dtype=torch.uint8, device="cuda")
    src.pool.prefill_attn(4, hq, p.q_out, p.ind, src.table_d, src.lens_d, None, SCALE, out, ws)
    p.check_q()
    assert src.pool.error() == 0 and src.lens_d.tolist() == lens and bool(torch.isfinite(out).all())

    f = Filled4(kv, [0] * 4, hkv=hkv, seed=3, spare=60, extra_width=30)
    f.pool.append_from_pool(4, src.pool, src.table_d, src.lens_d, f.table_d, f.tags_d, f.lens_d)
    # what the 4 bits leave of a key: a group's codes lie at most 6 steps of s apart, s off by 2^-4
    for b in range(4):
        pg = src.table_d[b, :-(-lens[b] // 16)].long()
        for which, dim in (("k", 2), ("v", 3)):
            rows = getattr(src.pool, which + "_cache")[pg].cpu().double().movedim(dim, 1)  # page, slot, ..
            rows = rows.reshape(-1, hkv, 128)[:lens[b]]
            got = _rows4(f, b, which)
            amax = rows.unflatten(-1, (8, 16)).abs().amax(-1).repeat_interleave(16, -1)
            # half of the widest step (1 of 2 s) with s up to amax / 6 (1 + 2^-4), and what saturates
            assert bool(((got - rows).abs() <= amax / 6 * (1 + 2.0 ** -4) + 2.0 ** -4 * amax).all())

    mask = torch.zeros(4, dtype=torch.uint8, device="cuda")
    ws = torch.empty(f.pool.workspace_size(4, hq, 1), dtype=torch.uint8, device="cuda")
    for i in range(3):
        t = Turn([1] * 4, hq, hkv, 10 + i)
        t.append(f)
        f.pool.verify(4, f.table_d, f.tags_d, f.lens_d, mask)
        q = t.q_out.view(4, 1, hq, 128)
        got = torch.zeros_like(q)
        f.pool.attn(4, hq, 1, q, f.table_d, f.lens_d, mask, SCALE, got, ws)
        t.check_q()
        assert mask.tolist() == [0] * 4 and f.lens_d.tolist() == [n + i + 1 for n in lens]
        _check4(f, got.cpu(), q.cpu())
        again, m2 = torch.zeros_like(q), torch.ones_like(mask)
        kv.paged_decode_attn_checked(f.pool.handle, 4, hq, 1, q, f.table_d, f.tags_d, f.lens_d, SCALE, again, m2, ws)
        assert torch.equal(again, got) and m2.tolist() == [0] * 4

    # a turn captured: its replays append a token more each
    t = Turn([1] * 4, hq, hkv, 20)
    q, got = t.q_out.view(4, 1, hq, 128), torch.zeros_like(t.q_out).view(4, 1, hq, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.append(f)
        f.pool.verify(4, f.table_d, f.tags_d, f.lens_d, mask)
        f.pool.attn(4, hq, 1, q, f.table_d, f.lens_d, mask, SCALE, got, ws)
    for i in range(18):  # over a page's end
        graph.replay()
    torch.cuda.synchronize()
    assert f.pool.error() == 0 and f.lens_d.tolist() == [n + 21 for n in lens]
    _check4(f, got.cpu(), q.cpu())

    # rows handed back, and the pages of two requests taken again by another's handoff
    n = f.lens_d.tolist()
    k, v = (torch.zeros((sum(n), hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    f.pool.read_rows(4, f.table_d, f.lens_d, None, indptr(n).cuda(), None, k, v)
    for which, x in (("k", k), ("v", v)):
        assert torch.equal(x.cpu().double(), torch.cat([_rows4(f, b, which) for b in range(4)]))
    keep = [_rows4(f, b, "k") for b in range(4)]
    old = f.table_d.clone(), f.tags_d.clone(), f.lens_d.clone()
    rel = torch.empty(kv.kv_release_workspace_size(4), dtype=torch.uint8, device="cuda")
    f.pool.release(4, f.table_d, f.tags_d, f.lens_d, torch.tensor([1, 0, 0, 1], dtype=torch.uint8).cuda(), rel)
    only = torch.tensor([lens[0], 0, 0, 0], dtype=torch.int32).cuda()
    f.pool.append_from_pool(4, src.pool, src.table_d, only, f.table_d, f.tags_d, f.lens_d)
    assert f.pool.error() == 0 and f.lens_d.tolist() == [lens[0], n[1], n[2], 0]
    for b in (1, 2):
        assert torch.equal(_rows4(f, b, "k"), keep[b])
    assert torch.equal(_rows4(f, 0, "k"), keep[0][:lens[0]])  # (as it was with more tokens behind it)
    f.pool.verify(4, *old, mask)
    assert mask.tolist()[0] != 0 and mask.tolist()[1:3] == [0, 0]


@pytest.mark.parametrize("hq", [8, 24])
def test_step_of_more_requests_than_the_plan_cache(kv, hq):
    """kv_decode_step writes the attention's plan in its append: the bits of the separate calls."""
    B = 1100
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, B).tolist()
    f, h = (Filled4(kv, lens, hkv=2, seed=6, spare=B, extra_width=2) for _ in range(2))
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn((B, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = (torch.randn((B, 1, hq, 128), generator=g) * 0.5).to(torch.bfloat16).cuda()
    ind = indptr([1] * B).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.empty(B, dtype=torch.uint8, device="cuda")
    ws = torch.empty(f.pool.step_workspace_size(B, hq, 1), dtype=torch.uint8, device="cuda")
    f.tags_d[700, 0] += 1  # stale where it has rows
    h.tags_d[700, 0] += 1
    stale = lens[700] > 0
    f.pool.step(B, hq, 1, None, k, v, ind, 1, f.table_d, f.tags_d, f.lens_d, q, SCALE, out, mask, 0, ws)
    assert f.pool.error() == 0
    assert stale and mask.nonzero().flatten().tolist() == [700]
    counts = [int(b != 700) for b in range(B)]
    rows = torch.tensor([b for b in range(B) if b != 700]).cuda()
    h.pool.append(B, k[rows].contiguous(), v[rows].contiguous(), indptr(counts).cuda(), 1, h.table_d, h.tags_d, h.lens_d)
    want = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws2 = torch.empty(h.pool.workspace_size(B, hq, 1), dtype=torch.uint8, device="cuda")
    h.pool.attn(B, hq, 1, q, h.table_d, h.lens_d, mask, SCALE, want, ws2)
    for a, b in ((f.pool.k_cache, h.pool.k_cache), (f.table_d, h.table_d), (f.lens_d, h.lens_d), (out, want)):
        assert torch.equal(a, b)
    assert bool((out[700] == 7.0).all())
    live = [b in (0, 1, 699, 701, 1023, 1024, 1099) for b in range(B)]
    _check4(f, out.cpu(), q.cpu(), live)


def test_appends_of_two_pools_at_once(kv):
    """Handoffs and normalised appends into two pools on two streams: the bits of one after the other."""
    lens = [700, 33, 257]
    src = Filled(kv, lens, hkv=2, fp8=False, seed=30)
    pools = [Filled4(kv, [0] * 3, hkv=2, seed=31, spare=80, extra_width=50) for _ in range(3)]
    turns = [Turn([5, 1, 40], 8, 2, 32) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def run(f, t):
        f.pool.append_from_pool(3, src.pool, src.table_d, src.lens_d, f.table_d, f.tags_d, f.lens_d)
        t.append(f)

    for f, t, s in zip(pools, turns, streams):
        with torch.cuda.stream(s):
            run(f, t)
    torch.cuda.synchronize()
    run(pools[2], turns[2])
    torch.cuda.synchronize()
    a = pools[2]
    for f, t in zip(pools[:2], turns):
        assert f.pool.error() == 0 and f.lens_d.tolist() == [705, 34, 297]
        assert torch.equal(t.q_out, turns[2].q_out)
        for x, y in ((f.pool.k_cache, a.pool.k_cache), (f.pool.v_cache, a.pool.v_cache), (f.table_d, a.table_d)):
            assert torch.equal(x, y)
