"""Keys or values of a stack of layers held in 4 bits (FASTOCR_DTYPE_FP4).

A row is d codes (e2m1, two a byte) and d / 16 scales (e4m3, one a group of 16
dimensions); an element stands for e2m1 * e4m3 * gain of its layer and KV head: 4.5
bits instead of 16, so an attention layer that reads the cache reads 0.28 of it.
DecodeAttention.write_layer fills it and read_layer gives its values back.
"""
from __future__ import annotations

import torch


class Fp4Cache:
    """codes [layers, num_pages, H_kv, page_size, d / 2] uint8, scales [..., d / 16]
    float8_e4m3fn, gain [layers, H_kv] fp32 (a number, or a tensor that is copied).

    A group's scale is its largest magnitude / (6 gain), which e4m3 holds to 1 part in
    16 from 2^-6 to 448 and coarser below: a gain around the largest magnitude of the
    head / 2688 uses all of that range, 1 suits magnitudes of 0.1 to 2688.
    """

    fp4 = True
    dtype = torch.bfloat16   # of the queries, keys and values that go with it

    def __init__(self, layers: int, num_pages: int, kv_heads: int, page_size: int, head_dim: int, *, gain=1.0,
                 device=None):
        if head_dim % 16:
            raise ValueError("head_dim must be a multiple of 16")
        rows = (layers, num_pages, kv_heads, page_size)
        self.shape = torch.Size((*rows, head_dim))
        self.codes = torch.zeros(*rows, head_dim // 2, dtype=torch.uint8, device=device)
        self.scales = torch.zeros(*rows, head_dim // 16, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        gain = torch.as_tensor(gain, dtype=torch.float32).to(self.codes.device)
        if tuple(gain.shape) not in ((), (layers, kv_heads)):
            raise ValueError(f"gain must be a number or have shape ({layers}, {kv_heads})")
        if not bool((torch.isfinite(gain) & (gain > 0)).all()):
            raise ValueError("gain must be finite and above 0")
        self.gain = gain.expand(layers, kv_heads).clone(memory_format=torch.contiguous_format)

    @property
    def device(self):
        return self.codes.device

    @property
    def is_cuda(self):
        return self.codes.is_cuda

    def check(self):
        """Refuse tensors put in place of the cache's own that the library would read wrongly."""
        for name, dt, width in (("codes", torch.uint8, 2), ("scales", torch.float8_e4m3fn, 16)):
            t, want = getattr(self, name), (*self.shape[:4], self.shape[4] // width)
            if tuple(t.shape) != want or t.dtype != dt or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {want} on {self.device}")
        g = self.gain
        if tuple(g.shape) != (self.shape[0], self.shape[2]) or g.dtype != torch.float32 or g.device != self.device \
                or not g.is_contiguous():
            raise ValueError("gain must be a contiguous float32 tensor of shape [layers, H_kv]")

    def __getitem__(self, l):
        """Layer l: (codes, scales, gain)."""
        return self.codes[l], self.scales[l], self.gain[l]
