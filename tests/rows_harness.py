"""Small paged cases for the shared-prefix, cross, weighing and eviction calls,
and the error bounds their outputs are held to.

Bounds, per output element, from the arithmetic alone (u = half a step):
a logit is a sum of d fp32 products, off by at most (d + 4) 2^-24 scale sum|q k|
(+ 3 roundings of its own size); a probability by twice that (itself and the sum
it is divided by) plus the exponential's 2^-21 twice and n 2^-24 for the sum's
additions: c. An output is sum p v, so off by c * sum p|v| + n 2^-24 sum p|v|;
bf16 rounds every probability (u = 2^-8) before the product, sums rounded or
unrounded ones, and rounds the result: (2u) sum p|v| + u |out| more.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import rows as R

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Paged:
    """One layer's cache with shuffled pages; rows are addressed by (sequence, row)."""

    def __init__(self, batch, cap, hkv, d, page, dtype, seed, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        cols = -(-cap // page)
        self.page, self.hkv, self.d = page, hkv, d
        extra = 3                                  # pages that no table names
        n = batch * cols + extra
        self.table = torch.randperm(n, generator=g)[:batch * cols].to(torch.int32).view(batch, cols)
        self.k = torch.randn(n, hkv, page, d, generator=g).to(dtype).to(device)
        self.v = torch.randn(n, hkv, page, d, generator=g).to(dtype).to(device)
        self.device = device

    def gpu_table(self):
        return self.table.to(self.device)

    def rows(self, b, lo, hi, k=None, v=None):
        """K, V of rows [lo, hi) of sequence b: [n, H_kv, d] fp64."""
        r = torch.arange(lo, hi)
        pages = self.table[b][r // self.page].long()
        k = self.k if k is None else k
        v = self.v if v is None else v
        return np64(k.cpu()[pages, :, r % self.page]), np64(v.cpu()[pages, :, r % self.page])


def prob_bound(q, K, scale_d):
    """c of every query row [T, H_q] (relative error of a probability)."""
    T, n_q, d = q.shape
    n = max(K.shape[0], 1)
    c = np.zeros((T, n_q))
    if K.shape[0] == 0:
        return c
    g = n_q // K.shape[1]
    for h in range(n_q):
        s = (np.abs(q[:, h]) @ np.abs(K[:, h // g]).T).max(-1) / math.sqrt(scale_d)
        c[:, h] = 2 * (d + 7) * 2.0 ** -24 * s
    return c + 2 * 2.0 ** -21 + n * 2.0 ** -24


def check_out(got, q, K, V, dtype, where=""):
    """got [T, H_q, d] against full attention over K, V; returns (probabilities, their bound)."""
    out, p, mag = R.attend_all(q, K, V)
    c = prob_bound(q, K, q.shape[-1])
    tol = (c + K.shape[0] * 2.0 ** -24)[..., None] * mag + U[dtype] * np.abs(out)
    if dtype == torch.bfloat16:
        tol += 2 * U[dtype] * mag
    err = np.abs(np64(got) - out)
    worst = np.max(err - tol, initial=-1.0)
    assert np.isfinite(np64(got)).all(), f"{where}: not finite"
    assert worst <= 1e-30, f"{where}: error {err.max():.3g} is over its bound by {worst:.3g}"
    return p, c
