"""Measured cases of the pool's prompt-side operators.

Three operators around one paged pool: new rows rotated and quantised as they are
written (kv_append_rotary), attention of many new tokens over the cache
(paged_prefill_attn), and the cache's rows read back as bf16 (kv_read_rows).

`run` makes one pass: the plain torch form where `own` is false, the library's entry
points where it is true.  Both take the state of `prepare`, in the pool's layouts:
K [page][kv head][slot][dim], V [page][kv head][dim][slot], one fp32 scale per
(page, kv head) for e4m3; latent rows [page][slot][dim] with one scale per page.
"""
import math
import random

import torch

own = False

P = 16  # tokens a page (grouped heads)
D = 128  # head dim (grouped heads)
LATENT = {"page": 64, "dk": 576, "dv": 512}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a long prompt's first pass: the cache holds exactly the prompt
        dict(name="prefill prompt", op="prefill", B=1, hq=64, hkv=8, fp8=True, new_min=8192, new_max=8192,
             old_min=0, old_max=0, singles=0, shape=1),
        # chunked prompt processing far into two long contexts
        dict(name="prefill chunk", op="prefill", B=2, hq=64, hkv=8, fp8=True, new_min=2048, new_max=2048,
             old_min=30720, old_max=30720, singles=0, shape=2),
        # a batch of ragged prompts behind shared prefixes, bf16 cache, 12 query heads a kv head
        dict(name="prefill ragged bf16", op="prefill", B=4, hq=96, hkv=8, fp8=False, new_min=301, new_max=2900,
             old_min=0, old_max=1999, singles=0, shape=3),
        # a mixed step: a few prompt chunks among requests that decode one token
        dict(name="prefill mixed", op="prefill", B=24, hq=32, hkv=4, fp8=True, new_min=100, new_max=256,
             old_min=1000, old_max=7900, singles=20, shape=4),
        # scoring 16 drafted tokens for each request of the decode batch
        dict(name="prefill drafts", op="prefill", B=32, hq=64, hkv=8, fp8=True, new_min=16, new_max=16,
             old_min=4080, old_max=32752, singles=0, shape=5),
        # the smallest batch: a few short requests, where latency counts
        dict(name="prefill tiny", op="prefill", B=4, hq=8, hkv=2, fp8=True, new_min=1, new_max=33,
             old_min=3, old_max=222, singles=1, shape=6),
        # handing short requests to another worker
        dict(name="read tiny", op="read", latent=False, B=4, hkv=2, fp8=True, len_min=37, len_max=255, windows=False,
             shape=7),
        # a whole decode batch leaves the pool (to host memory or to a bf16 prefill)
        dict(name="read batch", op="read", latent=False, B=32, hkv=8, fp8=True, len_min=4096, len_max=32768,
             windows=False, shape=8),
        # parts of latent rows from odd places: a prefix that another request reuses
        dict(name="read latent windows", op="read", latent=True, B=16, hkv=1, fp8=True, len_min=8192,
             len_max=65536, windows=True, shape=9),
        # one decode step's rows of every request
        dict(name="append decode", op="append", B=64, hq=64, hkv=8, fp8=True, new_min=1, new_max=1, old_min=1000,
             old_max=4095, axes=3, rot=128, interleaved=False, shape=10),
        # prompts of images and text join the batch: positions of three axes
        dict(name="append prompts", op="append", B=8, hq=64, hkv=8, fp8=True, new_min=1001, new_max=4096,
             old_min=0, old_max=100, axes=3, rot=128, interleaved=False, shape=11),
        # bf16 cache, half of each head rotated in neighbouring pairs, two axes
        dict(name="append bf16 partial", op="append", B=16, hq=32, hkv=4, fp8=False, new_min=100, new_max=600,
             old_min=0, old_max=333, axes=2, rot=64, interleaved=True, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "read", "append"])
    hkv = rng.choice([1, 2, 4, 8])
    fp8 = rng.random() < 0.7
    shape = rng.randrange(1 << 30)
    if op == "prefill":
        hq = hkv * rng.choice([1, 4, 6, 8, 12, 16])
        new = _log(rng, 1, 8192)
        old = rng.choice([0, _log(rng, 1, 30000)])
        B = _log(rng, 1, 32)
        # the plain form's scores (padded) and the work stay below the largest listed case's
        while B > 1 and B * hq * new * (new + old) > 4e9:
            B -= 1
        while hq * new * (new + old) > 4e9:
            new = max(1, new // 2)
        return dict(op=op, B=B, hq=hq, hkv=hkv, fp8=fp8, new_min=max(1, new // 3), new_max=new, old_min=old // 3,
                    old_max=old, singles=rng.choice([0, B // 2]), shape=shape)
    if op == "read":
        latent = rng.random() < 0.35
        hi = _log(rng, 20, 65536 if latent else 32768)
        return dict(op=op, latent=latent, B=_log(rng, 1, 16 if latent else 32), hkv=1 if latent else hkv, fp8=fp8,
                    len_min=max(1, hi // 8), len_max=hi, windows=rng.random() < 0.5, shape=shape)
    hi = _log(rng, 1, 4096)
    B = min(_log(rng, 1, 128), max(1, 24000 // hi))
    return dict(op=op, B=B, hq=hkv * rng.choice([4, 8]), hkv=hkv, fp8=fp8, new_min=max(1, hi // 4), new_max=hi,
                old_min=0, old_max=_log(rng, 1, 4000), axes=rng.choice([1, 2, 3]), rot=rng.choice([32, 64, 128]),
                interleaved=rng.random() < 0.4, shape=shape)


def _lens(case):
    """(cached before, new) of each request; a read's (first row, rows, cached)."""
    rng = random.Random(case["shape"])
    got = []
    for b in range(case["B"]):
        if case["op"] == "read":
            n = rng.randint(case["len_min"], case["len_max"])
            first = rng.randint(0, n - 1) if case["windows"] else 0
            got.append((first, n - first if not case["windows"] else rng.randint(1, n - first), n))
        else:
            new = rng.randint(case["new_min"], case["new_max"])
            if case["op"] == "prefill" and b >= case["B"] - case["singles"]:
                new = 1
            got.append((rng.randint(case["old_min"], case["old_max"]), new))
    return got


def work(case):
    lens = _lens(case)
    elem = 1 if case["fp8"] else 2
    if case["op"] == "prefill":
        rows = sum(o + n for o, n in lens)
        new = sum(n for _, n in lens)
        seen = sum(n * o + n * (n + 1) // 2 for o, n in lens)
        scale = 2 * case["hkv"] * 4 * sum(-(-(o + n) // P) for o, n in lens) if case["fp8"] else 0
        return {"bytes": 2 * 2 * new * case["hq"] * D + 2 * rows * case["hkv"] * D * elem + scale,
                "flops": 4 * case["hq"] * D * seen}
    if case["op"] == "read":
        rows = sum(n for _, n, _ in lens)
        width = LATENT["dk"] if case["latent"] else 2 * case["hkv"] * D
        return {"bytes": rows * width * (elem + 2), "flops": rows * width}
    new = sum(n for _, n in lens)
    return {"bytes": new * D * (4 * case["hq"] + 2 * case["hkv"] * (2 + elem)) + 4 * case["axes"] * new,
            "flops": new * (3 * case["rot"] * (case["hq"] + case["hkv"]) + 2 * case["hkv"] * D)}


# ---------------------------------------------------------------- inputs

def _scaled_rows(g, shape, std):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(torch.bfloat16)


def _fill(g, pages, hkv, fp8, latent):
    """A pool's content: rows as a cache holds them, with a spread of its own for each channel."""
    if latent:
        x = torch.randn((pages, 1, LATENT["page"] * LATENT["dk"]), device="cuda", generator=g)
        kinds = [(x, (pages, LATENT["page"], LATENT["dk"]))]
    else:
        kinds = []
        for shape, chan in (((pages, hkv, P, D), (1, hkv, 1, D)), ((pages, hkv, D, P), (1, hkv, D, 1))):
            x = torch.randn(shape, device="cuda", generator=g)
            x *= torch.empty(chan, device="cuda").uniform_(0.5, 4.0, generator=g)
            kinds.append((x.reshape(pages, hkv, -1), shape))
    out = []
    for x, shape in kinds:
        if fp8:
            s = x.abs().amax(-1) / 448
            out += [(x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape),
                    s.reshape(pages) if latent else s]
        else:
            out += [x.to(torch.bfloat16).reshape(shape), None]
    return (out + [None, None])[:4]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    lens = _lens(case)
    op, B, hkv, fp8 = case["op"], case["B"], case["hkv"], case["fp8"]
    latent = bool(case.get("latent"))
    page = LATENT["page"] if latent else P
    dk, dv = (LATENT["dk"], LATENT["dv"]) if latent else (D, D)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cached = [x[2] if op == "read" else x[0] for x in lens]
    total = cached if op == "read" else [o + n for o, n in lens]
    need = [-(-t // page) for t in total]
    have = [-(-c // page) for c in (total if op == "prefill" else cached)]
    pages = int(sum(need) * 1.1) + 8
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    width = max(need) + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    kc, ks, vc, vs = _fill(g, pages, hkv, fp8, latent)
    st = dict(op=op, fp8=fp8, latent=latent, page=page, B=B, hkv=hkv, table=table, k_cache=kc, k_scale=ks,
              v_cache=vc, v_scale=vs, width=width)
    # pages in the order in which an append takes them: those in use come first
    free = ids
    tags = torch.zeros(pages, dtype=torch.int32, device="cuda")
    book = i32([at, 0, 0, 0] + (total if op == "prefill" else cached))  # control words, then lengths
    st["book"], st["free"] = book, free
    if op == "prefill":
        hq = case["hq"]
        new = [n for _, n in lens]
        st.update(hq=hq, indptr=i32([sum(new[:b]) for b in range(B + 1)]), new_max=max(new), len_max=max(total),
                  scale=D ** -0.5, q=_scaled_rows(g, (sum(new), hq, D), 1.0))
        st["out"] = torch.empty_like(st["q"])
    elif op == "read":
        n = [x[1] for x in lens]
        st.update(first=i32([x[0] for x in lens]), indptr=i32([sum(n[:b]) for b in range(B + 1)]))
        st["k_out"] = torch.empty((sum(n), dk) if latent else (sum(n), hkv, dk), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = None if latent else torch.empty((sum(n), hkv, dv), dtype=torch.bfloat16, device="cuda")
    else:
        hq, rot = case["hq"], case["rot"]
        new = [n for _, n in lens]
        t = sum(new)
        qkv = _scaled_rows(g, (t, hq + 2 * hkv, D), 1.0)  # one projection's output, its parts side by side
        # time, height and width of a token: text has all three alike, an image's differ
        pos = i32([p for o, n in lens for p in range(o, o + n)]).repeat(case["axes"], 1)
        pos[1:] += torch.randint(0, 64, pos[1:].shape, device="cuda", generator=g, dtype=torch.int32)
        pos += torch.randint(0, 100000, (1,), device="cuda", generator=g, dtype=torch.int32)
        axis = torch.arange(rot // 2, device="cuda") * case["axes"] // (rot // 2)
        st.update(hq=hq, rot=rot, interleaved=case["interleaved"], indptr=i32([sum(new[:b]) for b in range(B + 1)]),
                  new_max=max(new), q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos,
                  axis=axis.to(torch.uint8), book0=book.clone(),
                  freq=10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot),
                  q_out=torch.empty((t, hq, D), dtype=torch.bfloat16, device="cuda"))
    if own:
        import paged_fp8_kv_append_gb300 as kv

        pool = kv.KVPool(pages, page, hkv, dk, dv, dtype=kv.KV_DTYPE_E4M3 if fp8 else kv.KV_DTYPE_BF16,
                         layout=kv.KV_LAYOUT_LATENT if latent else kv.KV_LAYOUT_GQA, tags=tags, free_list=free,
                         ctl=book[:kv.KV_CTL_WORDS], k_cache=kc, k_scale=ks, v_cache=vc, v_scale=vs)
        st["pool"], st["exp_tags"] = pool, torch.zeros_like(table)
        if op == "prefill":
            n = pool.prefill_workspace_size(B, case["hq"], st["q"].shape[0])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return {"prefill": _prefill, "read": _read, "append": _append}[st["op"]](st)


def _prefill(st):
    if own:
        st["pool"].prefill_attn(st["B"], st["hq"], st["q"], st["indptr"], st["table"], st["book"][4:], None,
                                st["scale"], st["out"], st["workspace"])
        return st["out"]
    B, hq, hkv, n, L = st["B"], st["hq"], st["hkv"], st["new_max"], st["len_max"]
    G, lens, ind = hq // hkv, st["book"][4:].long(), st["indptr"].long()
    count = ind[1:] - ind[:-1]
    i = torch.arange(n, device="cuda")
    q = st["q"][(ind[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)].float()  # [B, n, hq, D]
    q = q.view(B, n, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * n, D)
    pg = st["table"][:, :-(-L // P)].long().clamp_min(0)
    k, v = _values(st["k_cache"][pg], st["fp8"]), _values(st["v_cache"][pg], st["fp8"])
    if st["fp8"]:
        k *= st["k_scale"][pg][..., None, None]
        v *= st["v_scale"][pg][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(B, hkv, D, -1)  # [B, hkv, D, L]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, hkv, -1, D)
    # query i of a request sees positions 0 .. length - new + i
    see = torch.arange(k.shape[-1], device="cuda") <= (lens - count)[:, None, None] + i[:, None]  # [B, n, L]
    s = torch.matmul(q, k).mul_(st["scale"]).view(B, hkv, G, n, -1)
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, hkv, G * n, -1), v).view(B, hkv, G, n, D) / total.clamp_min(1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, D).to(torch.bfloat16)
    b, at = _owners(ind, st["q"].shape[0])
    return o[b, at]


def _values(x, fp8):
    return x.view(torch.float8_e4m3fn).float() if fp8 else x.float()


def _owners(ind, rows):
    """The request of each row, and the row's number within it."""
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(ind[1:], t, right=True)
    return b, t - ind[b]


def _read(st):
    if own:
        st["pool"].read_rows(st["B"], st["table"], st["book"][4:], st["first"], st["indptr"], None, st["k_out"],
                             st["v_out"])
        return [st["k_out"]] if st["latent"] else [st["k_out"], st["v_out"]]
    b, at = _owners(st["indptr"].long(), st["k_out"].shape[0])
    at = at + st["first"].long()[b]
    pg, slot = st["table"].long()[b, at // st["page"]], at % st["page"]
    if st["latent"]:
        k = _values(st["k_cache"][pg, slot], st["fp8"])
        if st["fp8"]:
            k *= st["k_scale"][pg][:, None]
        return [k.to(torch.bfloat16)]
    k, v = _values(st["k_cache"][pg, :, slot], st["fp8"]), _values(st["v_cache"][pg, :, :, slot], st["fp8"])
    if st["fp8"]:
        k *= st["k_scale"][pg][..., None]
        v *= st["v_scale"][pg][..., None]
    return [k.to(torch.bfloat16), v.to(torch.bfloat16)]


def _append(st):
    st["book"].copy_(st["book0"])  # the rows of the pass before are taken back
    lens = st["book"][4:]
    if own:
        st["pool"].append_rotary(st["B"], st["hq"], st["q"], st["k"], st["v"], st["indptr"], st["new_max"],
                                 st["pos"], st["axis"], st["freq"], st["interleaved"], st["q_out"], st["table"],
                                 st["exp_tags"], lens)
        q = st["q_out"]
    else:
        q = _append_plain(st, lens)
    cache = [x.view(torch.float8_e4m3fn) if st["fp8"] else x for x in (st["k_cache"], st["v_cache"])]
    scales = [st["k_scale"], st["v_scale"]] if st["fp8"] else []
    return [q, *cache, *scales, st["table"], lens]


def _append_plain(st, lens):
    ind = st["indptr"].long()
    angle = st["freq"] * st["pos"].t()[:, st["axis"].long()].double()  # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q, k, v = _turn(st["q"].float(), cos, sin, st), _turn(st["k"].float(), cos, sin, st), st["v"].float()
    # pages: each request takes what its new rows need, in order
    old, count = lens.long(), ind[1:] - ind[:-1]
    first = (old + P - 1) // P
    need = (old + count + P - 1) // P - first
    base = st["book"][0].long() + need.cumsum(0) - need
    b, at = _owners(ind, k.shape[0])
    at = at + old[b]
    j, slot = at // P, at % P
    fresh = j >= first[b]
    took = st["free"].long()[(base[b] + j - first[b]).clamp_(0, st["free"].shape[0] - 1)]
    pg = torch.where(fresh, took, st["table"].long()[b, j])
    st["table"][b, j] = pg.int()
    lens += count.int()
    st["book"][0] += need.sum()
    if st["fp8"]:
        k, v = _scaled(k, st["k_scale"], pg, fresh), _scaled(v, st["v_scale"], pg, fresh)
        k, v = k.to(torch.float8_e4m3fn).view(torch.uint8), v.to(torch.float8_e4m3fn).view(torch.uint8)
    st["k_cache"][pg, :, slot] = k.to(st["k_cache"].dtype)
    st["v_cache"][pg, :, :, slot] = v.to(st["v_cache"].dtype)
    return q.to(torch.bfloat16)


def _turn(x, cos, sin, st):
    rot, r = st["rot"], st["rot"] // 2
    if st["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _scaled(x, scale, pg, fresh):
    """x over its page's scale: a page taken now gets amax / 448 of its rows, another keeps what it has."""
    amax = torch.zeros_like(scale).index_reduce_(0, pg, x.abs().amax(-1), "amax")
    new = torch.where(amax > 0, amax / 448, 1.0)
    scale.copy_(torch.where(torch.zeros_like(scale[:, 0], dtype=torch.bool).index_fill_(0, pg[fresh], True)[:, None],
                            new, scale))
    return (x / scale[pg][..., None]).clamp_(-448, 448)


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "prefill" and work(case)["flops"] > 9e12:
        return None
    st = prepare(case, seed)
    return {"prefill": _exact_prefill, "read": _exact_read, "append": _exact_append}[case["op"]](case, st)


def _stored(st, which):
    """The values that a cache stands for, in 64 bits, as it is laid out."""
    x = st[which + "_cache"]
    if not st["fp8"]:
        return x.double()
    s = st[which + "_scale"].double()
    return x.view(torch.float8_e4m3fn).double() * s.reshape(s.shape + (1,) * (x.dim() - s.dim()))


def _exact_prefill(case, st):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    G, at = case["hq"] // case["hkv"], 0
    kd, vd = _stored(st, "k"), _stored(st, "v")
    for b, (old, new) in enumerate(_lens(case)):
        rows = torch.arange(old + new, device="cuda")
        pg, slot = st["table"][b].long()[rows // P], rows % P
        for h in range(case["hq"]):
            k, v = kd[pg, h // G, slot], vd[pg, h // G, :, slot]
            for lo in range(0, new, 2048):
                hi = min(new, lo + 2048)
                s = st["q"][at + lo:at + hi, h].double() @ k.t() * st["scale"]
                s += torch.full_like(s, -math.inf).triu(old + lo + 1)
                out[at + lo:at + hi, h] = torch.softmax(s, -1) @ v
        at += new
    return out


def _exact_read(case, st):
    got = []
    for which in ("k",) if case["latent"] else ("k", "v"):
        x = _stored(st, which)
        rows = []
        for b, (first, n, _) in enumerate(_lens(case)):
            at = torch.arange(first, first + n, device="cuda")
            pg, slot = st["table"][b].long()[at // st["page"]], at % st["page"]
            rows.append(x[pg, slot] if case["latent"] else x[pg, :, slot] if which == "k" else x[pg, :, :, slot])
        got.append(torch.cat(rows))
    return got


def _exact_append(case, st):
    half = case["rot"] // 2
    place = (lambda i, o: 2 * i + o) if case["interleaved"] else (lambda i, o: i + o * half)  # a pair's two dims
    i = torch.arange(half, device="cuda")
    angle = torch.stack([st["pos"][a] for a in st["axis"].tolist()], -1).double() * st["freq"]
    turned = []
    for x in (st["q"], st["k"]):
        x = x.double()
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
