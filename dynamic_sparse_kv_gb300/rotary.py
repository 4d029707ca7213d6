"""Rotary positions with several axes: the tables that DecodeAttention.write_layer turns
queries and keys by."""
from __future__ import annotations

import torch

from . import _native as N


class Rotary:
    """Angles of positions 0 .. positions - 1: pair i of a head turns by p_a * f_i, p_a the
    token's position on the pair's axis a.

    axes: how many pairs belong to each axis, e.g. (16, 24, 24) for time, height and
    width; (d / 2,) is the usual rotary embedding. They take the pairs in order, or with
    interleaved=True in turn (0, 1, 2, 0, 1, 2, ..., an axis that has its pairs left
    out). f_i = base ** (-2 i / rotary_dim), or with per_axis=True every axis counts its
    own pairs (base ** (-j / n) for the j-th of n). The first rotary_dim dimensions of a
    head turn (default all; a multiple of 32): pair i is dimensions i and
    i + rotary_dim / 2, or with adjacent=True 2i and 2i + 1.

    Cosines and sines are formed in 64 bits and kept in 32: positions * rotary_dim * 4
    bytes on the device.
    """

    def __init__(self, head_dim: int, axes, *, positions: int, base: float = 10000.0, rotary_dim: int | None = None,
                 adjacent: bool = False, interleaved: bool = False, per_axis: bool = False, device=None):
        rotary_dim = head_dim if rotary_dim is None else int(rotary_dim)
        axes = tuple(int(n) for n in axes)
        half = rotary_dim // 2
        if rotary_dim < 32 or rotary_dim % 32 or rotary_dim > head_dim:
            raise ValueError(f"rotary_dim must be a multiple of 32 of at most {head_dim}, not {rotary_dim}")
        if not 1 <= len(axes) <= 4 or min(axes) < 1 or sum(axes) != half:
            raise ValueError(f"axes must be 1 to 4 counts of pairs that add up to {half}, not {axes}")
        if positions < 1 or not base > 0:
            raise ValueError("positions must be at least 1 and base above 0")
        if interleaved:
            left, axis = list(axes), []
            while len(axis) < half:
                for a, n in enumerate(left):
                    if n:
                        axis.append(a)
                        left[a] -= 1
        else:
            axis = [a for a, n in enumerate(axes) for _ in range(n)]
        self.head_dim, self.rotary_dim, self.axes, self.positions = head_dim, rotary_dim, len(axes), int(positions)
        self.axis = torch.tensor(axis, dtype=torch.int8, device=device)
        exponent = torch.arange(half, dtype=torch.float64, device=device) / half
        if per_axis:
            seen, own = [0] * len(axes), []
            for a in axis:
                own.append(seen[a] / axes[a])
                seen[a] += 1
            exponent = torch.tensor(own, dtype=torch.float64, device=device)
        freq = float(base) ** -exponent
        angle = torch.arange(self.positions, dtype=torch.float64, device=device)[:, None] * freq
        self.cos_sin = torch.stack([torch.cos(angle), torch.sin(angle)], dim=-1).float().contiguous()
        self.c = N.fastocr_rotary(self.cos_sin.data_ptr(), self.axis.data_ptr(), self.positions, rotary_dim,
                                  self.axes, int(adjacent))
