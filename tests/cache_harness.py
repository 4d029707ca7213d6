"""Plain models of what happens to a paged cache: the 4-bit format, rotary positions, and a
pool of pages. NumPy and lists, no code of the package.

Bounds of attention over 4 bits, beside those of rows_harness: keys, values and (within
2^-25 of the row's largest element, where fp16 runs out of exponents) queries enter the
products as they are; a probability is rounded to fp16, 2^-11 of it, in product and sum, and
below 2^-31 of the largest one is lost.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import rows as R
from rows_harness import U, np64, prob_bound

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])        # 0 .. 448, by code


def nearest(x, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    up = (x - table[lo] > table[hi] - x) | ((x - table[lo] == table[hi] - x) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x, gain):
    """x [..., d] float32, gain float32 -> (codes [..., d/2] uint8, scales [..., d/16] uint8)."""
    with np.errstate(all="ignore"):
        y = (x.astype(np.float32) / np.float32(gain)).reshape(*x.shape[:-1], -1, 16)
        top = np.abs(y).max(-1)
        bad = ~np.isfinite(y).all(-1)
        s = nearest(np.minimum(np.where(bad, 0, top) / np.float32(6), np.float32(448)).astype(np.float64), E4M3)
        z = y / E4M3[s].astype(np.float32)[..., None]
        z = np.where((s == 0)[..., None] | bad[..., None], np.float32(0), z)
        code = nearest(np.minimum(np.abs(z), 6).astype(np.float64), LEVELS)
        code = code + 8 * (np.signbit(z))
    code = code.reshape(*x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0x7f, s).astype(np.uint8)


def values(codes, scales, gain):
    """What codes and scales stand for, fp64."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    return v * np.repeat(table[scales], 16, -1) * np.float64(gain)


class Fp4Paged:
    """One layer's cache in 4 bits, shuffled pages; every row that no sequence has is NaN."""

    def __init__(self, n, hkv, d, page, seed, cap=None, kv=None):
        g = torch.Generator().manual_seed(seed)
        cols = max(1, -(-(cap or max(n)) // page))
        pages = len(n) * cols + 3
        self.page, self.n = page, list(n)
        self.table = torch.randperm(pages, generator=g)[:len(n) * cols].to(torch.int32).view(len(n), cols)
        self.gain = [(0.05 + torch.rand(hkv, generator=g)).float().numpy() for _ in range(2)]
        self.codes = [np.full((pages, hkv, page, d // 2), 0x97, np.uint8) for _ in range(2)]
        self.scales = [np.full((pages, hkv, page, d // 16), 0x7f, np.uint8) for _ in range(2)]
        self.rows = []     # per sequence: K, V [n, H_kv, d] fp64
        for b, m in enumerate(n):
            both = []
            for w in range(2):
                x = kv(b, w, m) if kv else torch.randn(m, hkv, d, generator=g) * (1 + w)
                val = np.zeros((m, hkv, d))
                r = np.arange(m)
                at = self.table[b].numpy()[r // page]
                for h in range(hkv):
                    c, s = quantise(x[:, h].numpy(), self.gain[w][h])
                    self.codes[w][at, h, r % page], self.scales[w][at, h, r % page] = c, s
                    val[:, h] = values(c, s, self.gain[w][h])
                both.append(val)
            self.rows.append(both)

    def caches(self):
        from dynamic_sparse_kv_gb300 import Fp4Cache
        out = []
        for w in range(2):
            p, h, s, half = self.codes[w].shape
            c = Fp4Cache(1, p, h, s, 2 * half, gain=torch.from_numpy(self.gain[w])[None], device="cuda")
            c.codes.copy_(torch.from_numpy(self.codes[w])[None])
            c.scales.view(torch.uint8).copy_(torch.from_numpy(self.scales[w])[None])
            out.append(c)
        return out

    def decoder(self, q_heads, **kw):
        from dynamic_sparse_kv_gb300 import DecodeAttention
        dec = DecodeAttention(*self.caches(), self.table.cuda(), q_heads=q_heads, **kw)
        dec.set_seq_len(torch.tensor(self.n, dtype=torch.int32, device="cuda"))
        return dec


def logit_bound(q, K):
    """prob_bound plus what tiny elements of a query lose: c of every row and head."""
    c = prob_bound(q, K, q.shape[-1])
    if K.shape[0] == 0:
        return c
    d, g = q.shape[-1], q.shape[1] // K.shape[1]
    top = np.abs(q).max(-1)
    for h in range(q.shape[1]):
        c[:, h] += 2 * math.sqrt(d) * 2.0 ** -25 * top[:, h] * np.abs(K[:, h // g]).max()
    return c


def check_out4(got, q, K, V, where=""):
    """got, q [T, H_q, d] against attention over the values K, V [N, H_kv, d]."""
    out, p, mag = R.attend_all(q, K, V)
    c = logit_bound(q, K)
    tol = (c + K.shape[0] * 2.0 ** -24 + 2 * 2.0 ** -11)[..., None] * mag + U[torch.bfloat16] * np.abs(out)
    if K.shape[0]:
        tol += K.shape[0] * 2.0 ** -31 * np.abs(V).max()
    err = np.abs(np64(got) - out)
    assert np.isfinite(np64(got)).all(), f"{where}: not finite"
    worst = np.max(err - tol, initial=-1.0)
    assert worst <= 1e-30, f"{where}: error {err.max():.3g} is over its bound by {worst:.3g}"
    return p, c


# ---------------------------------------------------------------- rotary positions


def table(positions, rotary_dim, base):
    """cos, sin [positions, rotary_dim / 2] float32 of angles in 64 bits (base: a number, or a
    frequency for every pair)."""
    half = rotary_dim // 2
    f = base if np.ndim(base) else float(base) ** -(np.arange(half) / half)
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rotate(x, pos, axis, cos, sin, adjacent):
    """x [T, H, d] float32, pos [axes, T]; every product and sum rounded to float32."""
    half = cos.shape[1]
    x = x.copy()
    for i in range(half):
        p = np.clip(pos[axis[i]], 0, cos.shape[0] - 1)
        c, s = cos[p, i][:, None], sin[p, i][:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        x0, x1 = x[..., a].copy(), x[..., b].copy()
        x[..., a] = x0 * c - x1 * s
        x[..., b] = x1 * c + x0 * s
    return x


# ---------------------------------------------------------------- a pool of pages


class Pool:
    """Pages as lists; data[page] is what the page holds (any value)."""

    def __init__(self, batch, pages, page, cap_pages):
        self.page, self.pages, self.cap = page, pages, cap_pages
        self.rows = [[] for _ in range(batch)]
        self.len = [0] * batch
        self.data = list(range(pages))

    def refs(self):
        r = [0] * self.pages
        for row in self.rows:
            for x in row:
                r[x] += 1
        return r

    def reserve(self, want):
        """want[b]: rows; returns how many pages are missing."""
        refs, ps = self.refs(), self.page
        free = [i for i in range(self.pages) if refs[i] == 0]
        asked = []      # (sequence, column) that are looked at
        for b, n in enumerate(want):
            need = -(-min(max(n, 0), self.cap * ps) // ps)
            asked += [(b, c) for c in range(min(self.len[b] // ps, len(self.rows[b])), need)]
        wanted = {}
        for b, c in asked:
            if c < len(self.rows[b]):
                wanted.setdefault(self.rows[b][c], []).append((b, c))
        take = []
        for b, c in asked:
            if c < len(self.rows[b]):
                x = self.rows[b][c]
                if refs[x] == 1 or (len(wanted[x]) == refs[x] and wanted[x][0] == (b, c)):
                    continue
            take.append((b, c))
        if len(take) > len(free):
            return len(take) - len(free)
        old = list(self.data)
        for (b, c), x in zip(take, free):
            if c < len(self.rows[b]):
                if c * ps < self.len[b]:
                    self.data[x] = old[self.rows[b][c]]
                self.rows[b][c] = x
            else:
                self.rows[b].append(x)
        return 0

    def fork(self, src, dst):
        new = [(list(self.rows[s][:-(-self.len[s] // self.page)]), self.len[s]) for s in src]
        for d, (row, n) in zip(dst, new):
            self.rows[d], self.len[d] = row, n

    def release(self, seqs):
        for b in seqs:
            self.rows[b], self.len[b] = [], 0

    def trim(self):
        for b, n in enumerate(self.len):
            self.rows[b] = self.rows[b][:-(-n // self.page)]

    def compact(self):
        refs = self.refs()
        used = sum(r > 0 for r in refs)
        holes = [i for i in range(used) if refs[i] == 0]
        late = [i for i in range(used, self.pages) if refs[i] > 0]
        to = dict(zip(late, holes))
        for a, b in to.items():
            self.data[b] = self.data[a]
        self.rows = [[to.get(x, x) for x in row] for row in self.rows]
        return used
