"""Measured cases of the 4-bit pools' operators, and of the append that normalises heads.

Four operators around a paged pool: rows quantised to 4 bits as they are written
(kv_append_quantize, kv_append_from_pool), decode attention over such a pool
(paged_decode_attn), its rows back as bf16 (kv_read_rows), and new rows whose heads are
normalised and rotated on their way into an e4m3 or bf16 pool (kv_append_norm_rotary).

`run` makes one pass: the plain torch form where `own` is false, the library's entry
points where it is true.  Both take the state of `prepare`, in the pool's layouts.

A 4-bit pool holds a tile of 1152 bytes for each (page of 16 tokens, kv head) of K and of V:
1024 bytes of e2m1 codes, then 128 of e4m3 group scales, one for 16 dims of a token; a
power-of-two fp32 scale for each (page, kv head) stands outside.  With group c = d / 16:
  K code   byte 64 slot + 16 (c % 4) + 8 (c / 4) + (d % 16) / 2, low half where d is even
  K scale  byte 1024 + 16 (slot % 8) + 4 (c % 4) + 2 (slot / 8) + c / 4
  V code   byte 512 (d % 16 / 8) + 64 c + 16 (slot % 8 / 2) + 4 (d % 8 / 2) + 2 (slot / 8) + d % 2,
           low half where slot is even
  V scale  byte 1024 + 16 c + 4 (slot % 8 / 2) + 2 (slot / 8) + slot % 2
"""
import math
import random

import torch

own = False

P = 16  # tokens a page
D = 128  # head dim
TILE = 1152  # bytes of a 4-bit tile
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a whole decode batch of long contexts, one token each
        dict(name="attn batch", op="attn", B=32, T=1, hq=64, hkv=8, len_min=4096, len_max=32768, shape=1),
        # one request at a very long context: its pages are spread over the whole card
        dict(name="attn one long", op="attn", B=1, T=1, hq=64, hkv=8, len_min=131071, len_max=131071, shape=2),
        # scoring 4 drafted tokens a request: 32 query rows a kv head
        dict(name="attn drafts", op="attn", B=24, T=4, hq=32, hkv=4, len_min=4, len_max=24001, shape=3),
        # 12 query heads a kv head, ragged shorter requests
        dict(name="attn ragged", op="attn", B=48, T=1, hq=96, hkv=8, len_min=301, len_max=8191, shape=4),
        # the smallest batch: a few short requests, where latency counts
        dict(name="attn tiny", op="attn", B=4, T=1, hq=8, hkv=2, len_min=37, len_max=255, shape=5),
        # one decode step's rows of every request
        dict(name="append decode", op="append", B=64, hkv=8, new_min=1, new_max=1, old_min=1000, old_max=4095, shape=6),
        # prompts join the batch, some behind a page that is partly filled
        dict(name="append prompts", op="append", B=8, hkv=8, new_min=1001, new_max=4096, old_min=0, old_max=100, shape=7),
        # prompts that a bf16 pool holds are handed to the decode pool
        dict(name="handoff", op="handoff", B=16, hkv=8, len_min=4096, len_max=32768, shape=8),
        # a decode batch leaves the pool, to a bf16 prefill or another worker
        dict(name="read batch", op="read", B=32, hkv=8, len_min=4096, len_max=32768, windows=False, shape=9),
        # parts of short requests from odd places
        dict(name="read windows", op="read", B=6, hkv=2, len_min=37, len_max=1023, windows=True, shape=10),
        # one decode step: heads normalised, half of each turned in neighbouring pairs, bf16 pool
        dict(name="norm decode", op="norm", B=64, hq=32, hkv=4, fp8=False, new_min=1, new_max=1, old_min=1000,
             old_max=4095, axes=1, rot=64, interleaved=True, shape=11),
        # prompts of images and text: heads normalised and turned on three axes, e4m3 pool
        dict(name="norm prompts", op="norm", B=8, hq=64, hkv=8, fp8=True, new_min=1001, new_max=4096, old_min=0,
             old_max=100, axes=3, rot=128, interleaved=False, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "handoff", "read", "norm"])
    hkv, shape = rng.choice([1, 2, 4, 8]), rng.randrange(1 << 30)
    if op == "attn":
        T = rng.choice([1, 1, 1, 2, 4])
        G = rng.choice([g for g in (1, 4, 5, 6, 8, 12, 16) if T * g <= 64])
        hi = _log(rng, T, 131072)
        B = min(_log(rng, 1, 64), max(1, 600000 // hi))
        return dict(op=op, B=B, T=T, hq=G * hkv, hkv=hkv, len_min=max(T, hi // 8), len_max=hi, shape=shape)
    if op == "handoff":
        hi = _log(rng, 1, 32768)
        return dict(op=op, B=min(_log(rng, 1, 64), max(1, 300000 // hi)), hkv=hkv, len_min=hi // 8, len_max=hi,
                    shape=shape)
    if op == "read":
        hi = _log(rng, 20, 32768)
        return dict(op=op, B=min(_log(rng, 1, 64), max(1, 600000 // hi)), hkv=hkv, len_min=max(1, hi // 8), len_max=hi,
                    windows=rng.random() < 0.5, shape=shape)
    hi = _log(rng, 1, 4096)
    case = dict(op=op, B=min(_log(rng, 1, 128), max(1, 24000 // hi)), hkv=hkv, new_min=max(1, hi // 4), new_max=hi,
                old_min=0, old_max=_log(rng, 1, 4000), shape=shape)
    if op == "norm":
        case.update(hq=hkv * rng.choice([4, 8]), fp8=rng.random() < 0.6, axes=rng.choice([1, 2, 3]),
                    rot=rng.choice([32, 64, 128]), interleaved=rng.random() < 0.4)
    return case


def _lens(case):
    """(cached before, new) of each request; a read's (first row, rows, cached)."""
    rng = random.Random(case["shape"])
    got = []
    for b in range(case["B"]):
        if case["op"] == "read":
            n = rng.randint(case["len_min"], case["len_max"])
            first = rng.randint(0, n - 1) if case["windows"] else 0
            got.append((first, rng.randint(1, n - first) if case["windows"] else n, n))
        elif case["op"] == "attn":
            got.append((rng.randint(case["len_min"], case["len_max"]), 0))
        elif case["op"] == "handoff":
            got.append((0, rng.randint(case["len_min"], case["len_max"])))
        else:
            got.append((rng.randint(case["old_min"], case["old_max"]), rng.randint(case["new_min"], case["new_max"])))
    if case["op"] == "handoff" and not sum(n for _, n in got):
        got[0] = (0, 1)
    return got


def work(case):
    lens, hkv = _lens(case), case["hkv"]
    row = 2 * hkv * D * 9 / 16  # K and V of a token in 4 bits, with the group scales
    if case["op"] == "attn":
        T, hq = case["T"], case["hq"]
        rows = sum(o for o, _ in lens)
        seen = sum(max(0, o - T + 1 + i) for o, _ in lens for i in range(T))
        return {"bytes": 4 * case["B"] * T * hq * D + rows * row + 8 * hkv * sum(-(-o // P) for o, _ in lens),
                "flops": 4 * hq * D * seen}
    if case["op"] == "read":
        rows = sum(n for _, n, _ in lens)
        return {"bytes": rows * (row + 4 * hkv * D), "flops": rows * 4 * hkv * D}
    new = sum(n for _, n in lens)
    if case["op"] != "norm":
        return {"bytes": new * (row + 4 * hkv * D), "flops": new * 6 * hkv * D}
    elem = 1 if case["fp8"] else 2
    return {"bytes": new * D * (4 * case["hq"] + 2 * hkv * (2 + elem)) + 4 * case["axes"] * new,
            "flops": new * ((4 * D + 3 * case["rot"]) * (case["hq"] + hkv) + 2 * hkv * D)}


# ---------------------------------------------------------------- the 4-bit form

def _layout():
    """Byte and shift of each [slot][dim] code, and byte of each [slot][group] scale, in a K and a V tile."""
    s, d = torch.arange(P, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    c = d // 16
    kb, ks = 64 * s + 16 * (c % 4) + 8 * (c // 4) + d % 16 // 2, (d % 2 * 4).expand(P, D)
    vb = 512 * (d % 16 // 8) + 64 * c + 16 * (s % 8 // 2) + 4 * (d % 8 // 2) + 2 * (s // 8) + d % 2
    vs, c = (s % 2 * 4).expand(P, D), torch.arange(D // 16, device="cuda")[None]
    kg = 1024 + 16 * (s % 8) + 4 * (c % 4) + 2 * (s // 8) + c // 4
    vg = 1024 + 16 * c + 4 * (s % 8 // 2) + 2 * (s // 8) + s % 2
    return dict(k=(kb, ks.to(torch.uint8), kg), v=(vb, vs.to(torch.uint8), vg), codes=torch.tensor(CODES, device="cuda"))


def _values(tiles, scale, lay, which):
    """The values [..., slot, dim] of tiles [..., 1152] with block scales [...]."""
    at, shift, group = lay[which]
    nib = (tiles[..., at] >> shift) & 15
    s = tiles[..., group].view(torch.float8_e4m3fn).float() * scale[..., None, None]
    return (lay["codes"][nib.int()].unflatten(-1, (D // 16, 16)) * s[..., None]).flatten(-2)


def _block_scale(amax):
    """2^(floor(log2 amax) - 6), in 2^-100 .. 2^121: the largest group's scale lies in [10.6, 21.4)."""
    e = ((amax.view(torch.int32) >> 23) - 133).clamp(-100, 121)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), 1.0)


def _codes(x, scale):
    """x [..., 128] in fp32 over block scales [...]: its codes (a byte each) and group scale bytes [..., 8]."""
    inv = (1.0 / scale)[..., None]  # a power of two
    g = x.unflatten(-1, (D // 16, 16))
    s = (g.abs().amax(-1) * inv * (1 / 6)).clamp_max(448).to(torch.float8_e4m3fn)
    f = torch.where(s.float() > 0, 1.0 / s.float(), 0.0) * inv
    q = g * f[..., None]
    a = q.abs()  # to the nearest value, ties to the even code
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
            + (torch.signbit(q).byte() << 3))
    return code.flatten(-2), s.view(torch.uint8)


def _write(cache, which, lay, pg, slot, code, group, even, odd):
    """Codes and group scales of rows into their places; `even` / `odd`: the rows of even and odd slots."""
    at, _, gat = lay[which]
    head = torch.arange(cache.shape[1], device="cuda")[None, :, None]
    cache[pg[:, None, None], head, gat[slot][:, None]] = group
    if which == "k":  # a byte holds two dims of the row
        cache[pg[:, None, None], head, at[slot][:, None, ::2]] = code[..., ::2] | (code[..., 1::2] << 4)
        return
    for rows, keep, shift in ((even, 0xF0, 0), (odd, 0x0F, 4)):  # a byte holds two slots of a dim
        i = (pg[rows][:, None, None], head, at[slot[rows]][:, None])
        cache[i] = (cache[i] & keep) | (code[rows] << shift)


# ---------------------------------------------------------------- inputs

def _fill4(g, pages, hkv, lay, which):
    """A pool's tiles and block scales: rows as a cache holds them, with a spread of its own for each channel."""
    tiles = torch.empty((pages, hkv, TILE), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, hkv), device="cuda")
    spread = torch.empty((1, hkv, 1, D), device="cuda").uniform_(0.5, 4.0, generator=g)
    at, shift, gat = lay[which]
    order = torch.argsort((at * 2 + shift // 4).flatten())  # the codes in the order of the tile's halves
    for lo in range(0, pages, 4096):
        x = torch.randn((min(4096, pages - lo), hkv, P, D), device="cuda", generator=g) * spread
        s = _block_scale(x.abs().amax((-1, -2)))
        code, group = _codes(x, s[..., None].expand(-1, -1, P))
        code = code.flatten(-2)[..., order]
        tiles[lo:lo + 4096, :, :1024] = code[..., ::2] | (code[..., 1::2] << 4)
        tiles[lo:lo + 4096, :, gat] = group
        scale[lo:lo + 4096] = s
    return tiles, scale


def _fill_other(g, pages, hkv, fp8):
    """The same for an e4m3 or bf16 pool."""
    out = []
    for shape, chan in (((pages, hkv, P, D), (1, hkv, 1, D)), ((pages, hkv, D, P), (1, hkv, D, 1))):
        x = torch.randn(shape, device="cuda", generator=g)
        x *= torch.empty(chan, device="cuda").uniform_(0.5, 4.0, generator=g)
        if fp8:
            s = x.abs().amax((-1, -2)) / 448
            out += [(x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s]
        else:
            out += [x.to(torch.bfloat16), None]
    return out


def _starts(counts):
    return [sum(counts[:b]) for b in range(len(counts) + 1)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, B, hkv, lens = case["op"], case["B"], case["hkv"], _lens(case)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bf16 = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cached = [x[2] if op == "read" else x[0] for x in lens]
    total = cached if op in ("attn", "read") else [o + n for o, n in lens]
    need, have = [-(-t // P) for t in total], [-(-c // P) for c in cached]
    pages = int(sum(need) * 1.1) + 8
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    width = max(need) + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    lay, four = _layout(), op != "norm"
    if four:
        kc, ks = _fill4(g, pages, hkv, lay, "k")
        vc, vs = _fill4(g, pages, hkv, lay, "v")
    else:
        kc, ks, vc, vs = _fill_other(g, pages, hkv, case["fp8"])
    tags = torch.zeros(pages, dtype=torch.int32, device="cuda")
    book = i32([at, 0, 0, 0] + cached)  # control words, then lengths
    st = dict(op=op, B=B, hkv=hkv, table=table, k_cache=kc, k_scale=ks, v_cache=vc, v_scale=vs, lay=lay, book=book,
              free=ids)  # pages in the order in which an append takes them: those in use come first
    new = [x[1] for x in lens]
    st["indptr"], st["new_max"], rows = i32(_starts(new)), max(new), sum(new)
    if op == "attn":
        st.update(hq=case["hq"], T=case["T"], len_max=max(total), scale=D ** -0.5,
                  q=torch.randn((B, case["T"], case["hq"], D), device="cuda", generator=g).to(torch.bfloat16))
        st["out"] = torch.empty_like(st["q"])
    elif op == "read":
        st.update(first=i32([x[0] for x in lens]), k_out=bf16(rows, hkv, D), v_out=bf16(rows, hkv, D))
    else:
        st["book0"] = book.clone()
        slots = [(o + i) % 2 for o, n in lens for i in range(n)]
        st["even"], st["odd"] = (torch.tensor([t for t, s in enumerate(slots) if s == half], device="cuda",
                                              dtype=torch.long) for half in (0, 1))
        spread = torch.empty((2, hkv, D), device="cuda").uniform_(0.5, 4.0, generator=g)
        if op == "append":
            st["k"], st["v"] = ((torch.randn((rows, hkv, D), device="cuda", generator=g) * s).to(torch.bfloat16)
                                for s in spread)
        elif op == "handoff":
            st["src_k"], _, st["src_v"], _ = _fill_other(g, pages, hkv, False)
            st["src_lens"] = i32(new)
            st["src_table"] = torch.full_like(table, -1)
            perm, at = torch.randperm(pages, device="cuda", generator=g).to(torch.int32), 0
            for b in range(B):
                st["src_table"][b, :need[b]] = perm[at:at + need[b]]
                at += need[b]
        else:
            hq, rot, axes = case["hq"], case["rot"], case["axes"]
            qkv = torch.randn((rows, hq + 2 * hkv, D), device="cuda", generator=g)
            qkv *= torch.empty((1, hq + 2 * hkv, 1), device="cuda").uniform_(0.2, 5.0, generator=g)
            qkv = qkv.to(torch.bfloat16)  # one projection's output, its parts side by side
            # time, height and width of a token: text has all three alike, an image's differ
            pos = i32([p for o, n in lens for p in range(o, o + n)]).repeat(axes, 1)
            pos[1:] += torch.randint(0, 64, pos[1:].shape, device="cuda", generator=g, dtype=torch.int32)
            pos += torch.randint(0, 100000, (1,), device="cuda", generator=g, dtype=torch.int32)
            st.update(hq=hq, rot=rot, interleaved=case["interleaved"], fp8=case["fp8"], q=qkv[:, :hq],
                      k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos,
                      axis=(torch.arange(rot // 2, device="cuda") * axes // (rot // 2)).to(torch.uint8),
                      freq=10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot),
                      q_norm=torch.empty(D, device="cuda").uniform_(0.3, 2.0, generator=g).to(torch.bfloat16),
                      k_norm=torch.empty(D, device="cuda").uniform_(0.3, 2.0, generator=g).to(torch.bfloat16),
                      eps=1e-6, q_out=bf16(rows, hq, D))
    if own:
        import paged_fp8_kv_append_gb300 as kv

        dtype = kv.KV_DTYPE_E2M1 if four else kv.KV_DTYPE_E4M3 if case["fp8"] else kv.KV_DTYPE_BF16
        st["pool"] = kv.KVPool(pages, P, hkv, D, D, dtype=dtype, tags=tags, free_list=ids, ctl=book[:kv.KV_CTL_WORDS],
                               k_cache=kc, k_scale=ks, v_cache=vc, v_scale=vs)
        st["exp_tags"] = torch.zeros_like(table)
        if op == "attn":
            n = st["pool"].workspace_size(B, case["hq"], case["T"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if op == "handoff":
            st["src"] = kv.KVPool(pages, P, hkv, D, D, dtype=kv.KV_DTYPE_BF16, k_cache=st["src_k"], v_cache=st["src_v"])
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return {"attn": _attn, "read": _read, "append": _append, "handoff": _append, "norm": _norm}[st["op"]](st)


def _attn(st):
    B, T, hq, hkv, lens = st["B"], st["T"], st["hq"], st["hkv"], st["book"][4:]
    if own:
        st["pool"].attn(B, hq, T, st["q"], st["table"], lens, None, st["scale"], st["out"], st["workspace"])
        return st["out"]
    G = hq // hkv
    pg = st["table"][:, :-(-st["len_max"] // P)].long().clamp_min(0)
    k = _values(st["k_cache"][pg], st["k_scale"][pg], st["lay"], "k")  # [B, pages, hkv, slot, dim]
    v = _values(st["v_cache"][pg], st["v_scale"][pg], st["lay"], "v")
    k, v = k.permute(0, 2, 4, 1, 3).flatten(-2), v.transpose(1, 2).flatten(2, 3)
    q = st["q"].float().view(B, T, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, D)
    s = torch.matmul(q, k).mul_(st["scale"]).view(B, hkv, T, G, -1)
    # query i of a request sees positions 0 .. length - T + i
    see = torch.arange(k.shape[-1], device="cuda") <= (lens.long()[:, None] - T + torch.arange(T, device="cuda"))[..., None]
    s = s.masked_fill(~see[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    o = torch.matmul(s.view(B, hkv, T * G, -1), v).view(B, hkv, T, G, D) / s.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, hq, D).to(torch.bfloat16)


def _owners(ind, rows):
    """The request of each row, and the row's number within it."""
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(ind[1:], t, right=True)
    return b, t - ind[b]


def _read(st):
    if own:
        st["pool"].read_rows(st["B"], st["table"], st["book"][4:], st["first"], st["indptr"], None, st["k_out"],
                             st["v_out"])
        return [st["k_out"], st["v_out"]]
    b, at = _owners(st["indptr"].long(), st["k_out"].shape[0])
    at = at + st["first"].long()[b]
    pg, slot = st["table"].long()[b, at // P], at % P
    out = []
    for which in ("k", "v"):
        tiles, lay = st[which + "_cache"], st["lay"]
        where, shift, group = lay[which]
        head = torch.arange(st["hkv"], device="cuda")[None, :, None]
        nib = (tiles[pg[:, None, None], head, where[slot][:, None]] >> shift[slot][:, None]) & 15
        s = tiles[pg[:, None, None], head, group[slot][:, None]].view(torch.float8_e4m3fn).float()
        s = s * st[which + "_scale"][pg][..., None]
        x = lay["codes"][nib.int()].unflatten(-1, (D // 16, 16)) * s[..., None]
        out.append(x.flatten(-2).to(torch.bfloat16))
    return out


def _take_pages(st, rows):
    """Each request takes the pages that its new rows need, in order: page, slot and freshness of each row."""
    ind, lens = st["indptr"].long(), st["book"][4:]
    old, count = lens.long(), ind[1:] - ind[:-1]
    first = (old + P - 1) // P
    need = (old + count + P - 1) // P - first
    base = st["book"][0].long() + need.cumsum(0) - need
    b, at = _owners(ind, rows)
    at = at + old[b]
    j, slot = at // P, at % P
    fresh = j >= first[b]
    took = st["free"].long()[(base[b] + j - first[b]).clamp_(0, st["free"].shape[0] - 1)]
    pg = torch.where(fresh, took, st["table"].long()[b, j])
    st["table"][b, j] = pg.int()
    lens += count.int()
    st["book"][0] += need.sum()
    return pg, slot, fresh


def _block_scales(x, scale, pg, fresh, of_amax):
    """A page taken now gets the scale of its rows, another keeps what it has."""
    amax = torch.zeros_like(scale).index_reduce_(0, pg, x.abs().amax(-1), "amax")
    mine = torch.zeros_like(scale[:, 0]).index_reduce_(0, pg, fresh.float(), "amax")
    scale.copy_(torch.where((mine > 0)[:, None], of_amax(amax), scale))


def _append(st):
    st["book"].copy_(st["book0"])  # the rows of the pass before are taken back
    lens, back = st["book"][4:], [st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"], st["book"][4:]]
    if own:
        if st["op"] == "append":
            st["pool"].append(st["B"], st["k"], st["v"], st["indptr"], st["new_max"], st["table"], st["exp_tags"], lens)
        else:
            st["pool"].append_from_pool(st["B"], st["src"], st["src_table"], st["src_lens"], st["table"],
                                        st["exp_tags"], lens)
        return back
    rows = st["even"].shape[0] + st["odd"].shape[0]
    if st["op"] == "append":
        k, v = st["k"], st["v"]
    else:
        b, at = _owners(st["indptr"].long(), rows)
        pg, slot = st["src_table"].long()[b, at // P], at % P
        k, v = st["src_k"][pg, :, slot], st["src_v"][pg, :, :, slot]
    pg, slot, fresh = _take_pages(st, rows)
    for which, x in (("k", k.float()), ("v", v.float())):
        scale = st[which + "_scale"]
        _block_scales(x, scale, pg, fresh, _block_scale)
        code, group = _codes(x, scale[pg])
        _write(st[which + "_cache"], which, st["lay"], pg, slot, code, group, st["even"], st["odd"])
    return back


def _norm(st):
    st["book"].copy_(st["book0"])
    lens = st["book"][4:]
    if own:
        st["pool"].append_norm_rotary(st["B"], st["hq"], st["q"], st["k"], st["v"], st["indptr"], st["new_max"],
                                      st["pos"], st["axis"], st["freq"], st["interleaved"], st["q_norm"],
                                      st["k_norm"], st["eps"], st["q_out"], st["table"], st["exp_tags"], lens)
        q = st["q_out"]
    else:
        q = _norm_plain(st)
    cache = [x.view(torch.float8_e4m3fn) if st["fp8"] else x for x in (st["k_cache"], st["v_cache"])]
    scales = [st["k_scale"], st["v_scale"]] if st["fp8"] else []
    return [q, *cache, *scales, st["table"], lens]


def _norm_plain(st):
    angle = st["freq"] * st["pos"].t()[:, st["axis"].long()].double()  # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q, k = (_turn(_normed(st[x].float(), st[x + "_norm"].float(), st["eps"]), cos, sin, st) for x in ("q", "k"))
    v = st["v"].float()
    pg, slot, fresh = _take_pages(st, v.shape[0])
    if st["fp8"]:
        out = []
        for x, scale in ((k, st["k_scale"]), (v, st["v_scale"])):
            _block_scales(x, scale, pg, fresh, lambda a: torch.where(a > 0, a / 448, 1.0))
            x = (x / scale[pg][..., None]).clamp_(-448, 448)
            out.append(x.to(torch.float8_e4m3fn).view(torch.uint8))
        k, v = out
    st["k_cache"][pg, :, slot] = k.to(st["k_cache"].dtype)
    st["v_cache"][pg, :, :, slot] = v.to(st["v_cache"].dtype)
    return q.to(torch.bfloat16)


def _normed(x, weight, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight


def _turn(x, cos, sin, st):
    rot, r = st["rot"], st["rot"] // 2
    if st["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "read": _exact_read, "append": _exact_append, "handoff": _exact_append,
            "norm": _exact_norm}[case["op"]](case, st)


def _stored(tile, scale, which):
    """What tiles [n, 1152] with block scales [n] stand for: [n, slot, dim] in 64 bits."""
    n = tile.shape[0]
    nib = torch.stack((tile[:, :1024] & 15, tile[:, :1024] >> 4), -1)
    groups = tile[:, 1024:].view(torch.float8_e4m3fn).double()
    if which == "k":  # [slot, c % 4, c / 4, byte, half]; scales [slot % 8, c % 4, slot / 8, c / 4]
        nib = nib.view(n, 16, 4, 2, 8, 2).permute(0, 1, 3, 2, 4, 5)
        groups = groups.view(n, 8, 4, 2, 2).permute(0, 3, 1, 4, 2)
    else:  # [d % 16 / 8, c, slot % 8 / 2, d % 8 / 2, slot / 8, d % 2, half]; scales [c, slot % 8 / 2, slot / 8, slot % 2]
        nib = nib.view(n, 2, 8, 4, 4, 2, 2, 2).permute(0, 5, 3, 7, 2, 1, 4, 6)
        groups = groups.view(n, 8, 4, 2, 2).permute(0, 3, 2, 4, 1)
    nib = nib.reshape(n, 16, 8, 16).double()
    size = nib % 8
    e, m = (size / 2).floor(), size % 2
    x = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2) * torch.where(nib >= 8, -1.0, 1.0)
    return (x * groups.reshape(n, 16, 8, 1) * scale.double()[:, None, None, None]).reshape(n, 16, 128)


def _rows_of(st, b, h, n, which):
    """The first n cached rows of request b, kv head h."""
    pg = st["table"][b, :-(-n // P)].long()
    return _stored(st[which + "_cache"][pg, h], st[which + "_scale"][pg, h], which).reshape(-1, D)[:n]


def _exact_attn(case, st):
    T, G = case["T"], case["hq"] // case["hkv"]
    out = torch.zeros((case["B"], T, case["hq"], D), dtype=torch.float64, device="cuda")
    for b, (n, _) in enumerate(_lens(case)):
        for h in range(case["hkv"]):
            k, v = _rows_of(st, b, h, n, "k"), _rows_of(st, b, h, n, "v")
            for i in range(max(0, T - n), T):
                last = n - T + i + 1
                q = st["q"][b, i, h * G:(h + 1) * G].double()
                out[b, i, h * G:(h + 1) * G] = torch.softmax(q @ k[:last].t() * st["scale"], -1) @ v[:last]
    return out


def _exact_read(case, st):
    return [torch.cat([torch.stack([_rows_of(st, b, h, first + n, w)[first:] for h in range(case["hkv"])], 1)
                       for b, (first, n, _) in enumerate(_lens(case))]) for w in ("k", "v")]


def _exact_append(case, st):
    """Codes and pages are whole numbers and have no value here; block scales are 2^(floor(log2 amax) - 6)."""
    scales = [st["k_scale"].double(), st["v_scale"].double()]
    at, used = 0, int(st["book"][0])
    free = st["free"].tolist()
    for b, (old, new) in enumerate(_lens(case)):
        page = -(-old // P)
        while page * P < old + new:
            lo, hi = max(0, page * P - old), min(new, (page + 1) * P - old)
            for i, x in enumerate(("k", "v")):
                if case["op"] == "append":
                    rows = st[x][at + lo:at + hi].double()  # [rows, hkv, D]
                else:
                    rows = st["src_" + x][int(st["src_table"][b, page])].double()
                    rows = (rows[:, :hi - lo] if x == "k" else rows[..., :hi - lo].transpose(1, 2)).transpose(0, 1)
                amax = rows.abs().amax((0, 2))
                scales[i][free[used]] = torch.where(amax > 0, torch.exp2(torch.frexp(amax)[1] - 7.0), 1.0)
            used, page = used + 1, page + 1
            if used > 30000:
                return None  # page by page this takes too long
        at += new
    return [None, None, *scales, None, None]


def _exact_norm(case, st):
    half = case["rot"] // 2
    place = (lambda i, o: 2 * i + o) if case["interleaved"] else (lambda i, o: i + o * half)  # a pair's two dims
    i = torch.arange(half, device="cuda")
    angle = torch.stack([st["pos"][a] for a in st["axis"].tolist()], -1).double() * st["freq"]
    turned = []
    for name in ("q", "k"):
        x = st[name].double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + st["eps"]).sqrt() * st[name + "_norm"].double()
        z = torch.complex(x[..., place(i, 0)], x[..., place(i, 1)]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        x[..., place(i, 0)], x[..., place(i, 1)] = z.real, z.imag
        turned.append(x)
    fp8 = case["fp8"]
    cache = [x.view(torch.float8_e4m3fn).double() if fp8 else x.double() for x in (st["k_cache"], st["v_cache"])]
    scale = [st["k_scale"].double(), st["v_scale"].double()] if fp8 else []
    free, at = st["free"][int(st["book"][0]):].tolist(), 0
    for b, (old, new) in enumerate(_lens(case)):
        row = 0
        while row < new:
            page, slot = divmod(old + row, P)
            n = min(P - slot, new - row)
            pg = free.pop(0) if slot == 0 else int(st["table"][b, page])
            for c, x in enumerate((turned[1], st["v"].double())):
                x = x[at + row:at + row + n].transpose(0, 1)  # [hkv, rows, D]
                if fp8:
                    if slot == 0:
                        scale[c][pg] = x.abs().amax((1, 2)) / 448
                    x = (x / scale[c][pg][:, None, None]).clamp(-448, 448)
                if c == 0:
                    cache[0][pg, :, slot:slot + n] = x
                else:
                    cache[1][pg, :, :, slot:slot + n] = x.transpose(1, 2)
            row += n
        at += new
    return [turned[0], *cache, *scale, None, None]
