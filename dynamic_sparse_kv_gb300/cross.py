"""Cross attention of decoder layers to an encoder's states over the C ABI.

The states' keys and values sit in the same paged layout as a decoder's own
cache (fastocr_cross_attend): each sequence has a length of its own, 0 included,
and any number of query tokens, packed without padding.
"""
from __future__ import annotations

import torch

from . import _native as N


class CrossAttention:
    """Attention of packed queries to encoder states, for a stack of layers.

    k_cache, v_cache: [layers, num_pages, H_kv, page_size, d] (bf16 or fp32)
    block_table: [B, pages_per_seq] int32; state_len: int or [B] int32, states a
    sequence has (a device int32 tensor is taken as it is and may change).
    max_rows: query tokens of the largest call, for the workspace (None: any).
    max_states: about the longest sequence's states, for the split choices only;
    None takes it from state_len, or, where that is on the device, the capacity
    of block_table.
    """

    def __init__(self, k_cache, v_cache, block_table, state_len, *, q_heads: int,
                 max_rows: int | None = None, max_states: int | None = None):
        self.batch = block_table.shape[0]
        if isinstance(state_len, int):
            state_len = torch.full((self.batch,), state_len, dtype=torch.int32)
        if block_table.dim() != 2 or tuple(state_len.shape) != (self.batch,):
            raise ValueError(f"block_table must be [B, pages], state_len an int or [B], not "
                             f"{tuple(block_table.shape)} and {tuple(state_len.shape)}")
        dtype = N.check_caches(k_cache, v_cache)
        if dtype == N.FASTOCR_DTYPE_FP4:
            raise ValueError("cross attention needs states in bf16 or fp32, not in 4 bits")
        assert k_cache.is_cuda
        self.k_cache, self.v_cache = k_cache, v_cache
        self.layers, _, self.kv_heads, self.page_size, self.head_dim = k_cache.shape
        self.q_heads = q_heads
        dev = k_cache.device
        self.block_table = block_table.to(device=dev, dtype=torch.int32).contiguous()
        self.state_len = state_len.to(device=dev, dtype=torch.int32).contiguous()
        self.handle = N.fastocr_create(self.batch, q_heads, self.kv_heads, self.head_dim, dtype,
                                       self.page_size, self.block_table.shape[1], 0, self.layers)
        self.kv = [N.make_kv(k_cache[l], v_cache[l], self.block_table, self.state_len)
                   for l in range(self.layers)]
        if max_states is None and not state_len.is_cuda:
            max_states = int(state_len.max())
        capacity = self.block_table.shape[1] * self.page_size
        N.fastocr_set_length_hint(self.handle, min(max(0, max_states or 0), capacity))
        # the workspace stops growing where the rows of a sequence fill a row tile
        n = N.fastocr_rows_workspace(self.handle, max(1, 256 if max_rows is None else max_rows))
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)

    def close(self):
        if self.handle:
            N.fastocr_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def attend(self, l, q, q_start, out, stream=None):
        """Layer l: q, out [rows, H_q, d]; q_start [B + 1] int32, query tokens
        q_start[b] .. q_start[b+1]-1 are sequence b's. All contiguous and on the
        caches' device."""
        rows, dev = q.shape[0], self.k_cache.device
        shape = (rows, self.q_heads, self.head_dim)
        N.check_tensor(q, "q", shape, self.k_cache.dtype, dev)
        N.check_tensor(out, "out", shape, self.k_cache.dtype, dev)
        N.check_tensor(q_start, "q_start", (self.batch + 1,), torch.int32, dev)
        if rows == 0:
            return
        N.fastocr_cross_attend(self.handle, q, self.kv[l], q_start, rows, out, self.ws,
                               self.ws.numel(), stream)

    def device_status(self, stream=None) -> int:
        return N.fastocr_device_status(self.handle, stream)
