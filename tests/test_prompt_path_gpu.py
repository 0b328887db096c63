"""The prompt-side operators run together as a server runs them: rows appended
with kv_append_rotary, pages checked with kv_verify_tags, the new tokens'
attention with paged_prefill_attn, a decode step with paged_decode_attn behind
it, and the cached rows handed back with kv_read_rows.

Each stage is held against the 64-bit form of its own inputs as they lie on the
device (the turned queries, the quantised cache), so its bound is that of the
operator alone: attention as in test_prompt_prefill_gpu.py (2^-8 |o| + c A),
rows read back one bf16 half step and fp32's rounding."""
import pytest
import torch

from promptref import Filled, attention, e4m3_values, indptr, rotate

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _cached(f, b, n, which):
    """Request b's first n rows as the device holds them, fp64."""
    table = f.table_d[b].cpu().long()
    at = torch.arange(n)
    pg, slot = table[at // f.page], at % f.page
    c = (f.pool.k_cache if which == "k" else f.pool.v_cache).cpu()
    x = c[pg, :, slot] if which == "k" else c[pg, :, :, slot]
    if not f.fp8:
        return x.double()
    s = (f.pool.k_scale if which == "k" else f.pool.v_scale).cpu()[pg].double()
    return e4m3_values()[x.long()] * s[:, :, None]


def _bounded(f, got, q, k, v, old):
    ref, mag = attention(q, k, v, SCALE, old), attention(q, k, v.abs(), SCALE, old)
    c = 2.0 ** -9 if f.fp8 else 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10
    worst = float(((got.double() - ref).abs() / (2.0 ** -8 * ref.abs() + c * mag + 1e-30)).max())
    assert worst <= 1.0, worst


class Turn:
    """A batch's tensors of one turn: new tokens of every request."""

    def __init__(self, f, new, hq, seed, pad=0):
        g = torch.Generator().manual_seed(seed)
        t = sum(new) + pad
        width = (hq + 2 * f.hkv) * 128
        self.new, self.hq, self.x = new, hq, torch.randn((t, width), generator=g).to(torch.bfloat16).cuda()
        at = [0, hq * 128, (hq + f.hkv) * 128, width]  # one projection's output
        self.q, self.k, self.v = (self.x[:, a:b].unflatten(1, (-1, 128)) for a, b in zip(at, at[1:]))
        self.pos = torch.randint(0, 3000, (3, t), generator=g, dtype=torch.int32).cuda()
        self.axis = (torch.arange(64) % 3).to(torch.uint8).cuda()
        self.freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
        self.ind = indptr(new).cuda()
        self.q_out = torch.full((t, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = torch.full((t, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.abort = torch.zeros(f.B, dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(f.pool.prefill_workspace_size(f.B, hq, t), dtype=torch.uint8, device="cuda")

    def run(self, f, max_new=None):
        f.pool.append_rotary(f.B, self.hq, self.q, self.k, self.v, self.ind, max_new or max(self.new), self.pos,
                             self.axis, self.freq, False, self.q_out, f.table_d, f.tags_d, f.lens_d)
        f.pool.verify(f.B, f.table_d, f.tags_d, f.lens_d, self.abort)
        f.pool.prefill_attn(f.B, self.hq, self.q_out, self.ind, f.table_d, f.lens_d, self.abort, SCALE, self.out,
                            self.ws)

    def check(self, f, aborted=()):
        torch.cuda.synchronize()
        lens = f.lens_d.tolist()
        ind = self.ind.tolist()
        assert [int(x != 0) for x in self.abort.tolist()] == [int(b in aborted) for b in range(f.B)]
        for b in range(f.B):
            rows = slice(ind[b], ind[b + 1])
            if rows.start == rows.stop:
                continue
            if b in aborted:
                assert bool((self.out[rows] == 7.0).all())
                continue
            turned = rotate(self.q[rows].cpu(), self.pos[:, rows].cpu(), self.axis.cpu(), self.freq.cpu(), False)
            got = self.q_out[rows].cpu().double()
            # half a step of the value and 2^-19 of its pair (at most sqrt(2) of the larger)
            pair = self.q[rows].cpu().double().abs()
            pair = torch.maximum(pair, pair.roll(64, -1)) * 1.4143
            assert bool(((got - turned).abs() <= 2.0 ** -8 * turned.abs() + 2.0 ** -19 * pair).all())
            k, v = _cached(f, b, lens[b], "k"), _cached(f, b, lens[b], "v")
            _bounded(f, self.out[rows].cpu(), got, k, v, lens[b] - (rows.stop - rows.start))
        assert bool((self.out[ind[-1]:] == 7.0).all()) and bool((self.q_out[ind[-1]:] == 7.0).all())


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [(8, 2), (15, 3)])
def test_turns(kv, heads, fp8):
    """Prompts, a mixed batch behind them, one token each; then a decode step over the same cache
    gives what the attention of the last tokens gave, and the rows come back as they are cached."""
    hq, hkv = heads
    f = Filled(kv, [0, 0, 0, 0], hkv=hkv, fp8=fp8, seed=71, spare=200, extra_width=60)
    for i, new in enumerate(([300, 17, 1, 0], [1, 200, 1, 33], [1, 1, 1, 1])):
        t = Turn(f, new, hq, 72 + i, pad=5 if i == 1 else 0)  # (rows behind the last request's)
        t.run(f)
        t.check(f)
    assert f.pool.error() == 0 and f.lens_d.tolist() == [302, 218, 3, 34]
    # the last turn's tokens again, as a decode step
    dec = torch.zeros((4, 1, hq, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(f.pool.workspace_size(4, hq, 1), dtype=torch.uint8, device="cuda")
    f.pool.attn(4, hq, 1, t.q_out.view(4, 1, hq, 128), f.table_d, f.lens_d, t.abort, SCALE, dec, ws)
    lens = f.lens_d.tolist()
    for b in range(4):
        _bounded(f, dec[b].cpu(), t.q_out[b:b + 1].cpu().double(), _cached(f, b, lens[b], "k"),
                 _cached(f, b, lens[b], "v"), lens[b] - 1)
    # a window of each request's rows
    first = [10, 0, 1, 33]
    counts = [n - a for n, a in zip(lens, first)]
    k = torch.zeros((sum(counts), hkv, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    f.pool.read_rows(4, f.table_d, f.lens_d, torch.tensor(first, dtype=torch.int32).cuda(), indptr(counts).cuda(),
                     t.abort, k, v)
    at = 0
    for b in range(4):
        for which, got in (("k", k), ("v", v)):
            ref = _cached(f, b, lens[b], which)[first[b]:]
            x = got[at:at + counts[b]].cpu().double()
            assert bool(((x - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all())
        at += counts[b]
    assert f.pool.error() == 0


def test_a_request_whose_page_went_elsewhere(kv):
    """A tag that no longer fits: the request's attention rows stay untouched, the others' are right."""
    f = Filled(kv, [100, 64, 33], hkv=2, seed=81, spare=100, extra_width=20)
    t = Turn(f, [20, 30, 40], 8, 82)
    f.pool.tags[int(f.table_d[1, 2])] += 1  # page 2 of request 1 has a new owner
    t.run(f)
    t.check(f, aborted=(1,))


def test_captured_turn_follows_lengths(kv):
    """One captured turn (append, check, attention), replayed three times over a growing cache with
    other row counts, beside a second stream that reads rows of another pool."""
    f = Filled(kv, [0, 50], hkv=2, seed=91, spare=200, extra_width=80)
    t = Turn(f, [120, 40], 8, 92)
    other = Filled(kv, [700], hkv=2, seed=93)
    k = torch.zeros((700, 2, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ind = indptr([700]).cuda()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t.run(f, max_new=160)
    s = torch.cuda.Stream()
    want = [0, 50]
    for new in ([120, 40], [1, 159], [33, 0]):
        t.ind.copy_(indptr(new))
        t.out.fill_(7.0)
        t.q_out.fill_(7.0)
        s.wait_stream(torch.cuda.current_stream())
        g.replay()
        other.pool.read_rows(1, other.table_d, other.lens_d, None, ind, None, k, v, s)
        t.check(f)
        want = [a + n for a, n in zip(want, new)]
        assert f.lens_d.tolist() == want
    for which, got in (("k", k), ("v", v)):
        ref = other.rows(0, which)
        assert bool(((got.cpu().double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all())
    assert f.pool.error() == 0 and other.pool.error() == 0


@pytest.mark.parametrize("fp8", [True, False])
def test_queries_that_are_not_finite(kv, fp8):
    """A query of NaN or infinities spoils its own output row and no other, head and token apart."""
    f = Filled(kv, [400], hkv=2, fp8=fp8, seed=101)
    g = torch.Generator().manual_seed(102)
    q = torch.randn((200, 8, 128), generator=g).to(torch.bfloat16)
    q[3, 1, 5], q[77, 6, 0], q[130, 2, 9] = float("nan"), float("inf"), float("-inf")
    out = torch.zeros((200, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(f.pool.prefill_workspace_size(1, 8, 200), dtype=torch.uint8, device="cuda")
    f.pool.prefill_attn(1, 8, q.cuda(), indptr([200]).cuda(), f.table_d, f.lens_d, None, SCALE, out, ws)
    assert f.pool.error() == 0
    good = torch.ones(200, 8, dtype=torch.bool)
    good[3, 1] = good[77, 6] = good[130, 2] = False
    assert bool(torch.isfinite(out.cpu()[good]).all())
    clean = q.double()
    clean[~good] = 0
    k, v = f.rows(0, "k"), f.rows(0, "v")
    ref, mag = attention(clean, k, v, SCALE, 200), attention(clean, k, v.abs(), SCALE, 200)
    c = 2.0 ** -9 if fp8 else 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10
    err = (out.cpu().double() - ref).abs() / (2.0 ** -8 * ref.abs() + c * mag + 1e-30)
    assert float(err[good].max()) <= 1.0


def test_tensors_of_another_device_are_refused(kv, monkeypatch):
    f = Filled(kv, [20], hkv=2, seed=111)
    monkeypatch.setattr(kv, "_device", lambda: 1)
    k = torch.zeros((20, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        f.pool.read_rows(1, f.table_d, f.lens_d, None, indptr([20]).cuda(), None, k, k.clone())
    with pytest.raises(ValueError):
        kv.kv_read_rows(f.pool.handle, 1, f.table_d, f.lens_d, None, indptr([20]).cuda(), None, k,
                        k.clone(), 0)
