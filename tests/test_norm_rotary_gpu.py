"""kv_append_norm_rotary against the 64-bit form, in e4m3, bf16 and 4-bit pools.

Bounds.  A normalised value is x times a root that is off by at most 2^-21 (128 squares
summed in fp32 with a relative error of 2^-19 at most in pairs and chains of 16, halved by
the root, and two ulp of it), times a weight: two roundings.  2^-19 of the value in all;
the rotation adds 2^-19 of the pair's length (see test_prompt_rotary_gpu.py): 2^-18.  A bf16
output adds half a step, 2^-8; an e4m3 code half a step, 2^-4 of the value or 2^-10 scales;
a 4-bit code is one of the nearest values of its group."""
import numpy as np
import pytest
import torch

from promptref import Filled, e4m3_values, indptr, rotate
from test_prompt_rotary_gpu import _pair_len

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_fp8_kv_append_gb300 as kv

    return kv


def _normed(x, w, eps):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


class Case:
    def __init__(self, f, new, hq, rot, axes, interleaved, seed, dk=128, dv=128, norms="qk", eps=1e-6, mag=1.0):
        g = torch.Generator().manual_seed(seed)
        t, self.f, self.new, self.hq, self.il, self.eps = sum(new), f, new, hq, interleaved, eps
        width = (hq + f.hkv) * dk + f.hkv * dv + 8
        x = torch.randn((t, width), generator=g) * mag
        x *= torch.empty((t, 1)).uniform_(0.1, 10.0, generator=g)
        x = x.to(torch.bfloat16)
        xd = x.cuda()
        at = [0, hq * dk, (hq + f.hkv) * dk, width - 8]
        cut = lambda z, i, d: z[:, at[i]:at[i + 1]].unflatten(1, (-1, d)) if at[i + 1] > at[i] else None  # noqa: E731
        self.q, self.k, self.v = cut(x, 0, dk), cut(x, 1, dk), cut(x, 2, dv)
        self.dev = cut(xd, 0, dk), cut(xd, 1, dk), cut(xd, 2, dv)
        self.pos = torch.randint(-500, 4000, (axes, t), generator=g, dtype=torch.int32)
        self.axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.uint8)
        self.freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
        self.w = [torch.empty(dk).uniform_(-2.0, 2.0, generator=g).to(torch.bfloat16) if c in norms else None
                  for c in "qk"]

    def run(self, max_new=None, stream=None):
        f, (q, k, v) = self.f, self.dev
        self.q_out = None if q is None else torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        f.pool.append_norm_rotary(f.B, self.hq, q, k, v, indptr(self.new).cuda(),
                                  max(self.new) if max_new is None else max_new, self.pos.cuda(),
                                  self.axis.cuda(), self.freq.cuda(), self.il,
                                  *(None if w is None else w.cuda() for w in self.w), self.eps, self.q_out,
                                  f.table_d, f.tags_d, f.lens_d, stream)

    def turned(self, which):
        x = _normed(getattr(self, which), self.w["qk".index(which)], self.eps)
        return rotate(x, self.pos, self.axis, self.freq, self.il), _pair_len(x, 2 * len(self.freq), self.il)

    def check_q(self):
        ref, ln = self.turned("q")
        got = self.q_out.cpu().double()
        assert bool(((got - ref).abs() <= 2.0 ** -18 * ln + 2.0 ** -8 * ref.abs() + 1e-38).all())

    def places(self):
        """(row, page, slot) of every new row."""
        table, row = self.f.table_d.cpu(), 0
        for b, n in enumerate(self.new):
            for i in range(n):
                j, slot = divmod(self.f.lens[b] + i, self.f.page if hasattr(self.f, "page") else 16)
                yield row, int(table[b, j]), slot
                row += 1


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rot,axes,il", [(128, 3, False), (64, 2, True), (32, 1, False), (16, 1, True), (112, 2, False)])
@pytest.mark.parametrize("lens,new", [([0, 5, 16, 33], [16, 40, 1, 17]), ([3, 0], [1, 1])])
def test_pools_of_16x128(kv, fp8, rot, axes, il, lens, new):
    f = Filled(kv, lens, hkv=2, seed=rot, spare=24, extra_width=8, fp8=fp8)
    c = Case(f, new, 6, rot, axes, il, seed=rot)
    c.run()
    assert f.pool.error() == 0 and f.lens_d.tolist() == [a + b for a, b in zip(lens, new)]
    c.check_q()
    _check_kv(f, c)


def _check_kv(f, c):
    kr, ln = c.turned("k")
    vr = c.v.double()
    kc, vc = f.pool.k_cache.cpu(), f.pool.v_cache.cpu()
    for row, p, slot in c.places():
        for x, got, slack, scale in (
                (kr[row], kc[p, :, slot], 2.0 ** -18 * ln[row], f.pool.k_scale),
                (vr[row], vc[p, :, :, slot], torch.zeros(1), f.pool.v_scale)):
            if not f.fp8:
                assert bool(((got.double() - x).abs() <= slack + 2.0 ** -8 * x.abs()).all())
                continue
            s = scale[p].cpu().double()[:, None]
            x = x.clamp(-448 * s, 448 * s)  # (a partly filled page's scale is frozen)
            err = (e4m3_values()[got.long()] * s - x).abs()
            # (half a step of the value, and of a value that the slack moves across a border)
            assert bool((err <= slack + 2.0 ** -4 * (x.abs() + slack) + 2.0 ** -10 * s).all())


@pytest.mark.parametrize("dk,dv,page", [(64, 64, 16), (256, 256, 8), (32, 64, 16), (16, 16, 64), (512, 512, 4)])
def test_other_shapes(kv, dk, dv, page):
    f = Filled(kv, [0, 3], hkv=3, dk=dk, dv=dv, page=page, seed=dk, spare=32, extra_width=24)
    c = Case(f, [20, 33], 4, 16, 1, False, seed=dk, dk=dk, dv=dv)
    c.run()
    assert f.pool.error() == 0
    c.check_q()
    _check_kv(f, c)


@pytest.mark.parametrize("norms,hq", [("q", 4), ("k", 4), ("k", 0), ("", 4)])
def test_one_side_alone(kv, norms, hq):
    f = Filled(kv, [0, 7], hkv=2, seed=1, spare=16, extra_width=8)
    c = Case(f, [16, 30], hq, 64, 1, False, seed=2, norms=norms)
    c.run()
    assert f.pool.error() == 0
    if hq:
        c.check_q()
    _check_kv(f, c)


def test_without_weights_it_is_the_rotary_append(kv):
    got = []
    for plain in (False, True):
        f = Filled(kv, [0, 7], hkv=2, seed=1, spare=16, extra_width=8)
        c = Case(f, [33, 30], 4, 128, 2, False, seed=2, norms="")
        if plain:
            q, k, v = c.dev
            c.q_out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
            f.pool.append_rotary(2, 4, q, k, v, indptr(c.new).cuda(), 33, c.pos.cuda(), c.axis.cuda(),
                                 c.freq.cuda(), False, c.q_out, f.table_d, f.tags_d, f.lens_d)
        else:
            c.run()
        got.append((c.q_out, f.pool.k_cache, f.pool.v_cache, f.pool.k_scale, f.pool.v_scale))
    for a, b in zip(*got):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


@pytest.mark.parametrize("mag,eps", [(1e-4, 1e-6), (1e-4, 0.0), (3e3, 1e-5), (1e15, 1e-6), (1e-15, 0.0)])
def test_magnitudes(kv, mag, eps):
    f = Filled(kv, [0], hkv=2, seed=1, spare=16, extra_width=8, fp8=False)
    c = Case(f, [37], 4, 128, 1, False, seed=3, mag=mag, eps=eps)
    c.run()
    c.check_q()
    _check_kv(f, c)


def test_rows_of_zeros_and_rows_that_are_not_finite(kv):
    f = Filled(kv, [0], hkv=2, seed=1, spare=16, extra_width=8, fp8=False)
    c = Case(f, [32], 4, 64, 1, False, seed=4)
    for x in (c.q, c.dev[0]):
        x[3, 1] = 0
        x[5, 2, 77] = float("nan")
        x[6, 0, 3] = float("inf")
    c.run()
    out = c.q_out.cpu()
    assert not out[3, 1].any()
    assert bool(torch.isnan(out[5, 2]).all())
    assert bool(torch.isnan(out[6, 0, 3])) and not out[6, 0, 40:].any()  # a mean of infinity
    bad = torch.isnan(out)
    bad[5, 2] = bad[6, 0] = False
    assert not bad.any()


def test_in_place_and_captured(kv):
    f = Filled(kv, [0, 5], hkv=2, seed=1, spare=40, extra_width=20)
    c = Case(f, [20, 17], 4, 128, 1, False, seed=5)
    q = c.dev[0].contiguous()
    args = lambda: (2, 4, q, c.dev[1], c.dev[2], indptr(c.new).cuda(), 20, c.pos.cuda(), c.axis.cuda(),  # noqa: E731
                    c.freq.cuda(), False, c.w[0].cuda(), c.w[1].cuda(), 1e-6)
    held = args()
    f.pool.append_norm_rotary(*held, q, f.table_d, f.tags_d, f.lens_d)
    c.q_out = q.clone()
    c.check_q()
    _check_kv(f, c)
    out = torch.empty_like(q)
    q.copy_(c.dev[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.pool.append_norm_rotary(*held, out, f.table_d, f.tags_d, f.lens_d)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert f.pool.error() == 0 and f.lens_d.tolist() == [60, 56]
    assert torch.equal(out, c.q_out)


def test_stops_leave_later_requests(kv):
    f = Filled(kv, [0, 5, 3], hkv=2, seed=1, spare=3, extra_width=8)
    c = Case(f, [30, 64, 1], 4, 128, 1, False, seed=5)
    c.run()
    assert f.pool.error() == kv.KV_ERR_OUT_OF_PAGES and int(f.pool.ctl[2]) == 1
    assert f.lens_d.tolist() == [30, 5, 3]
    assert bool((c.q_out[30:] == 7.0).all())
    c.new = [30, 0, 0]
    ref, ln = c.turned("q")
    assert bool(((c.q_out.cpu().double() - ref).abs() <= 2.0 ** -18 * ln + 2.0 ** -8 * ref.abs())[:30].all())


def test_python_refusals(kv):
    f = Filled(kv, [0], hkv=2, seed=1, spare=16, extra_width=8)
    c = Case(f, [5], 4, 128, 1, False, seed=5)
    good = list(c.w)
    strided = torch.ones(256, dtype=torch.bfloat16, device="cuda")[::2]  # (a copy from the host would pack it)
    for bad in (torch.ones(64, dtype=torch.bfloat16), torch.ones(128), strided):
        c.w = [bad, good[1]]
        with pytest.raises((TypeError, ValueError)):
            c.run()
    c.w = good
    c.eps = -1.0
    with pytest.raises(kv.KVError):
        c.run()
    assert f.lens_d.tolist() == [0]


@pytest.mark.parametrize("norms", ["qk", ""])
@pytest.mark.parametrize("rot,axes,il", [(128, 3, False), (64, 2, True), (16, 1, False), (112, 1, True), (48, 2, False)])
@pytest.mark.parametrize("lens,new", [([0, 5, 16, 33], [16, 40, 1, 17]), ([3, 0], [1, 1])])
def test_4_bit_pools(kv, norms, rot, axes, il, lens, new):
    from e2m1ref import VALUES, Filled4, block_scale, scale_place, values

    f = Filled4(kv, lens, hkv=2, seed=rot, spare=24, extra_width=8)
    before = {w: f.cache[w].copy() for w in "kv"}
    c = Case(f, new, 6, rot, axes, il, seed=rot, norms=norms)
    if norms:
        c.run()
    else:
        q, k, v = c.dev
        c.q_out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        f.pool.append_rotary(f.B, 6, q, k, v, indptr(new).cuda(), max(new), c.pos.cuda(), c.axis.cuda(),
                             c.freq.cuda(), il, c.q_out, f.table_d, f.tags_d, f.lens_d)
    assert f.pool.error() == 0
    c.check_q()
    kr, ln = (x.numpy() for x in c.turned("k"))
    vr = c.v.double().numpy()
    fresh = {}
    for row, p, slot in c.places():
        fresh.setdefault(p, []).append((row, slot))
    for which, x, slack in (("k", kr, 2.0 ** -18 * ln), ("v", vr, 0 * vr)):
        cache = getattr(f.pool, which + "_cache").cpu().numpy()
        scale = getattr(f.pool, which + "_scale").cpu().numpy()
        for p, rows in fresh.items():
            for h in range(2):
                S = float(scale[p, h])
                if rows[0][1] == 0:  # taken by this call (a border of floor(log2) is off by one step)
                    a = max(np.abs(x[r, h]).max() for r, _ in rows)
                    assert S in (block_scale(a * (1 - 2 ** -17)), block_scale(a * (1 + 2 ** -17)))
                got = values(cache[p, h], np.float32(S), which)
                for r, slot in rows:
                    for g in range(8):
                        d = slice(16 * g, 16 * g + 16)
                        s = float(torch.tensor(cache[p, h, scale_place(which, slot, g)]).view(
                            torch.float8_e4m3fn)) * S
                        want = np.abs(x[r, h, d]).max() / 6
                        assert abs(s - min(want, 448 * S)) <= 2.0 ** -4 * want * (1 + 2 ** -12) + 2.0 ** -10 * S
                        y = x[r, h, d]
                        near = np.abs(y[:, None] - np.concatenate([-VALUES, VALUES])[None] * s).min(1)
                        assert (np.abs(got[slot, d] - y) <= near + 2 * slack[r, h, d] + 2.0 ** -20 * np.abs(y)).all()
                # rows that were there stay
                if rows[0][1]:
                    old = values(before[which][p, h], np.float32(f.scale[which][p, h]), which)
                    assert np.array_equal(got[:rows[0][1]], old[:rows[0][1]])
