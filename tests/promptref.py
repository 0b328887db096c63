"""Plain 64-bit forms of the prompt-side operators, and a small pool filled
directly (no append), for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch


def e4m3_values() -> torch.Tensor:
    """The 256 codes' values (fp64, NaN for 0x7F / 0xFF)."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


class Filled:
    """A GQA or latent pool whose requests' rows are drawn directly into
    shuffled pages; every other byte of the cache is NaN."""

    def __init__(self, kv, lens, hkv=2, dk=128, dv=128, page=16, fp8=True, latent=False, seed=0,
                 spare=8, extra_width=1, scale_mode=0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.lens, self.page, self.hkv, self.dk, self.dv = kv, lens, page, hkv, dk, dv
        self.fp8, self.latent, self.B = fp8, latent, len(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        ids = torch.randperm(pages, generator=g)
        width = max(need + [1]) + extra_width
        self.table = torch.full((self.B, width), -1, dtype=torch.int32)
        kshape = (pages, page, dk) if latent else (pages, hkv, page, dk)
        vshape = (pages, hkv, dv, page)
        if fp8:
            def fill(shape):
                x = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
                return torch.where((x & 0x7F) == 0x7F, x - 1, x)  # no NaN code
            junk = 0x7F
        else:
            def fill(shape):
                return torch.randn(shape, generator=g).to(torch.bfloat16)
            junk = math.nan
        k, v = fill(kshape), None if latent else fill(vshape)
        heads = (pages,) if latent else (pages, hkv)
        self.ks = torch.rand(heads, generator=g) * 0.01 + 1e-3 if fp8 else None
        self.vs = torch.rand(heads, generator=g) * 0.01 + 1e-3 if fp8 and not latent else None
        at = 0
        used = torch.zeros(pages, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                p = int(ids[at])
                at += 1
                used[p] = True
                self.table[b, j] = p
                left = min(page, n - j * page)
                if latent:
                    k[p, left:] = junk
                else:
                    k[p, :, left:] = junk
                    v[p, :, :, left:] = junk
        k[~used] = junk
        if v is not None:
            v[~used] = junk
        self.k, self.v = k, v
        self.free_list, self.free_head = ids.to(torch.int32), at
        dev = "cuda"
        ctl = torch.zeros(kv.KV_CTL_WORDS, dtype=torch.int32)
        ctl[0] = at
        cu = lambda t: None if t is None else t.to(dev)  # noqa: E731
        self.pool = kv.KVPool(pages, page, hkv, dk, dv,
                              dtype=kv.KV_DTYPE_E4M3 if fp8 else kv.KV_DTYPE_BF16,
                              layout=kv.KV_LAYOUT_LATENT if latent else kv.KV_LAYOUT_GQA,
                              free_list=self.free_list, k_cache=cu(k), v_cache=cu(v),
                              k_scale=cu(self.ks), v_scale=cu(self.vs), ctl=cu(ctl),
                              scale_mode=scale_mode)
        self.table_d = self.table.to(dev)
        self.tags_d = torch.zeros((self.B, width), dtype=torch.int32, device=dev)
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device=dev)

    def rows(self, b, which):
        """Request b's cached K or V rows, [n][heads][dim] ([n][dim] latent), in fp64."""
        n = self.lens[b]
        at = torch.arange(n)
        pg, slot = self.table[b].long()[at // self.page], at % self.page
        c = self.k if which == "k" else self.v
        x = c[pg, slot] if self.latent else c[pg, :, slot] if which == "k" else c[pg, :, :, slot]
        if not self.fp8:
            return x.double()
        s = (self.ks if which == "k" else self.vs)[pg].double()
        return e4m3_values()[x.long()] * s.reshape(s.shape + (1,) * (x.dim() - s.dim()))


def indptr(counts):
    out = np.zeros(len(counts) + 1, np.int32)
    out[1:] = np.cumsum(counts)
    return torch.from_numpy(out)


def attention(q, k, v, scale, old):
    """q [n][Hq][D], k / v [L][Hkv][D] in fp64; query i sees positions 0 .. old + i (rows that
    see none are zero)."""
    n, hq, _ = q.shape
    g = hq // k.shape[1]
    kx, vx = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("nhd,lhd->hnl", q, kx) * scale
    see = torch.arange(k.shape[0])[None] <= old + torch.arange(n)[:, None]
    s = s.masked_fill(~see[None], -math.inf)
    m = s.amax(-1, keepdim=True) if k.shape[0] else torch.zeros(hq, n, 1, dtype=torch.float64)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(s - m)
    return torch.einsum("hnl,lhd->nhd", p / p.sum(-1, keepdim=True).clamp_min(1e-300), vx)


def rotate(x, pos, axis, freq, interleaved):
    """x [n][heads][D] in fp64, pos [axes][n], pair i turned by pos[axis[i]] * freq[i]."""
    x = x.double().clone()
    half = len(freq)
    angle = pos.double()[axis.long()].t() * freq  # [n][half]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    x0, x1 = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
    return x
