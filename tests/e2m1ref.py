"""The 4-bit pools' form written out from its definition, in fp32 where the
definition says fp32 and in fp64 elsewhere, and a small pool filled directly."""
from __future__ import annotations

import math

import numpy as np
import torch

P, D, TILE = 16, 128, 1152
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SIXTH = np.float32(1.0) / np.float32(6.0)


def code_place(which, slot, d):
    """(byte, whether the high half) of a code in a tile."""
    c = d // 16
    if which == "k":
        return 64 * slot + 16 * (c % 4) + 8 * (c // 4) + (d % 16) // 2, d % 2
    return (512 * (d % 16 // 8) + 64 * c + 16 * (slot % 8 // 2) + 4 * (d % 8 // 2) + 2 * (slot // 8)
            + d % 2, slot % 2)


def scale_place(which, slot, c):
    if which == "k":
        return 1024 + 16 * (slot % 8) + 4 * (c % 4) + 2 * (slot // 8) + c // 4
    return 1024 + 16 * c + 4 * (slot % 8 // 2) + 2 * (slot // 8) + slot % 2


def _places(which):
    code = np.array([[code_place(which, s, d) for d in range(D)] for s in range(P)])
    scale = np.array([[scale_place(which, s, c) for c in range(D // 16)] for s in range(P)])
    return code[..., 0], code[..., 1], scale


PLACES = {w: _places(w) for w in "kv"}
_E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def values(tiles, block, which):
    """What tiles [..., 1152] with block scales [...] stand for: fp64 [..., slot, dim]."""
    byte, high, scale = PLACES[which]
    nib = (tiles[..., byte] >> (4 * high).astype(np.uint8)) & 15
    x = VALUES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = _E4M3[tiles[..., scale]] * block.astype(np.float64)[..., None, None]
    return x * np.repeat(s, 16, -1)


def block_scale(amax):
    """2^(floor(log2 amax) - 6), its exponent in -100 .. 121; 1 for nothing."""
    if not amax > 0:
        return np.float32(1.0)
    return np.float32(2.0) ** np.float32(min(max(math.frexp(float(amax))[1] - 7, -100), 121))


def e4m3_bytes(x):
    """fp32 (finite, >= 0) to e4m3, to nearest even, saturating."""
    t = torch.from_numpy(np.minimum(x, np.float32(448.0)).astype(np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def quantise(x, block):
    """Rows [..., 128] (fp32 values) over a block scale: codes [..., 128] and scale bytes [..., 8].
    Groups with a value that is not finite get the byte 0x7F and codes of no meaning."""
    x = x.astype(np.float32)
    inv = np.float32(1.0) / np.float32(block)
    g = x.reshape(x.shape[:-1] + (8, 16))
    amax = np.abs(g).max(-1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        finite = np.isfinite(g).all(-1)
        sc = e4m3_bytes(np.where(finite, amax * inv * SIXTH, 0).astype(np.float32))
        s = _E4M3[sc].astype(np.float32)
        f = np.where(s > 0, np.float32(1.0) / s, np.float32(0.0)) * inv
        q = (g * f[..., None]).astype(np.float32)
        a = np.abs(q).astype(np.float64)
        mids = (VALUES[1:] + VALUES[:-1]) / 2
        code = np.zeros(q.shape, np.uint8)
        for i, m in enumerate(mids):  # a tie goes to the even code
            code += (a > m) | ((a == m) & ((i + 1) % 2 == 0))
        code |= np.signbit(q).astype(np.uint8) << 3
    return code.reshape(x.shape), np.where(finite, sc, 0x7F).astype(np.uint8), finite


def write(tile, which, slot, codes, scales):
    """One row's codes and scale bytes into a tile [1152] (in place)."""
    byte, high, scale = PLACES[which]
    for d in range(D):
        b, h = byte[slot, d], high[slot, d]
        tile[b] = (tile[b] & 0x0F) | (codes[d] << 4) if h else (tile[b] & 0xF0) | codes[d]
    tile[scale[slot]] = scales


class Model:
    """A 4-bit pool's host twin: appends as the definition says, page by page."""

    def __init__(self, pages, hkv, free_list, tags, cache_k, cache_v, ks, vs, width, B):
        self.pages, self.hkv = pages, hkv
        self.free, self.head, self.tags = free_list.copy(), 0, tags.copy()
        self.cache = {"k": cache_k.copy(), "v": cache_v.copy()}
        self.scale = {"k": ks.copy(), "v": vs.copy()}
        self.table = np.full((B, width), -1, np.int32)
        self.exp = np.zeros((B, width), np.uint32)
        self.lens = np.zeros(B, np.int32)
        # nibbles / bytes whose codes have no meaning (groups that are not finite)
        self.loose = {"k": np.zeros(cache_k.shape, bool), "v": np.zeros(cache_v.shape, bool)}

    def append(self, k, v, counts):
        """k, v: fp32 [rows][hkv][128]; every request is served."""
        at = 0
        for r, n in enumerate(counts):
            row = 0
            while row < n:
                L = int(self.lens[r]) + row
                j, slot = divmod(L, P)
                m = min(P - slot, n - row)
                if slot == 0:
                    p = int(self.free[self.head])
                    self.head += 1
                    self.tags[p] = np.uint32((int(self.tags[p]) + 1) & 0xFFFFFFFF)
                    self.table[r, j], self.exp[r, j] = p, self.tags[p]
                p = int(self.table[r, j])
                for which, x in (("k", k), ("v", v)):
                    for h in range(self.hkv):
                        rows = x[at + row:at + row + m, h]
                        if slot == 0:
                            fin = np.isfinite(rows.reshape(m, 8, 16)).all(-1)
                            a = np.where(fin, np.abs(np.where(np.isfinite(rows), rows, 0)).reshape(
                                m, 8, 16).max(-1), 0).max()
                            self.scale[which][p, h] = block_scale(a)
                        code, sc, fin = quantise(rows, self.scale[which][p, h])
                        for i in range(m):
                            write(self.cache[which][p, h], which, slot + i, code[i], sc[i])
                            for c in np.nonzero(~fin[i])[0]:
                                self.loose[which][p, h, PLACES[which][0][slot + i,
                                                                         16 * c:16 * c + 16]] = True
                row += m
            at += n
            self.lens[r] += n


class Filled4:
    """A 4-bit pool whose requests' rows are drawn directly into shuffled pages; every
    other group scale of the cache is NaN, and so are unused pages' block scales."""

    def __init__(self, kv, lens, hkv=2, seed=0, spare=8, extra_width=1, spread=3):
        rng = np.random.default_rng(seed)
        self.kv, self.lens, self.hkv, self.B = kv, list(lens), hkv, len(lens)
        need = [-(-n // P) for n in lens]
        pages = sum(need) + spare
        ids = rng.permutation(pages).astype(np.int32)
        width = max(need + [1]) + extra_width
        self.table = np.full((self.B, width), -1, np.int32)
        self.cache, self.scale = {}, {}
        used = np.full(pages, 0)
        at = 0
        for b, n in enumerate(lens):
            for j in range(need[b]):
                self.table[b, j] = ids[at]
                used[ids[at]] = min(P, n - P * j)
                at += 1
        for which in "kv":
            tile = rng.integers(0, 256, (pages, hkv, TILE), dtype=np.uint8)
            byte, _, scale = PLACES[which]
            live = np.arange(P)[None, :] < used[:, None]  # [page, slot]
            sc = rng.integers(0x20, 0x40, (pages, hkv, P, 8), dtype=np.uint8)  # 1/32 .. 1.9
            sc = np.where(live[:, None, :, None], sc, 0x7F).astype(np.uint8)
            tile[:, :, scale] = sc
            self.cache[which] = tile
            s = 2.0 ** rng.integers(-spread, spread + 1, (pages, hkv)) * 0.25
            self.scale[which] = np.where((used > 0)[:, None], s, np.nan).astype(np.float32)
        self.free_list, self.free_head = ids, at
        self.to_device()

    def to_device(self):
        kv, pages = self.kv, self.cache["k"].shape[0]
        cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        ctl = np.zeros(kv.KV_CTL_WORDS, np.int32)
        ctl[0] = self.free_head
        self.pool = kv.KVPool(pages, P, self.hkv, D, D, dtype=kv.KV_DTYPE_E2M1,
                              free_list=self.free_list, k_cache=cu(self.cache["k"]),
                              v_cache=cu(self.cache["v"]), k_scale=cu(self.scale["k"]),
                              v_scale=cu(self.scale["v"]), ctl=cu(ctl))
        self.table_d = cu(self.table)
        self.tags_d = torch.zeros(self.table.shape, dtype=torch.int32, device="cuda")
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def rows(self, b, which, n=None):
        """Request b's first n cached rows, fp64 [n][hkv][128]."""
        n = self.lens[b] if n is None else n
        pg = self.table[b, :-(-n // P)]
        x = values(self.cache[which][pg], self.scale[which][pg], which)  # [pages, hkv, slot, dim]
        return torch.from_numpy(x.transpose(0, 2, 1, 3).reshape(-1, self.hkv, D)[:n].copy())
