"""Per-step schedule of FastOCR decode attention over the C ABI.

FastOCR (gist.science technical summary, "Focal-Guided Pruning" and
"Cross-Step Fixation Reuse"):
  * warm-up: w steps of full attention in every layer while the library
    accumulates each layer's image-attention mass; the |C| layers with the
    most image mass become the focal set C (fastocr_profiler_select);
  * each later step: layers in C call fastocr_focal_attend (full cache,
    head-summed image scores, top ceil(tau*N_img)); the selection is handed
    to the following non-focal layers (fastocr_sparse_attend);
  * non-focal layers before the first focal layer reuse F_last, the previous
    step's selection of the deepest focal layer;
  * adaptive layer selection (named there as future work): ProfileSchedule
    re-runs the warm-up window every `period` steps and re-chooses C.
Unlimited OCR (R-SWA): every layer calls fastocr_rswa_attend; with
ring_block_table a sequence's cache holds only the prefix and a ring of
window pages.
Beside those, for generated text that grows long and for batches that read one
document: share_prefix + shared_step (a prefix read once for a group of
sequences) and track_weights + weighed_step + evict_step (every row's attention
weight added up, the rows of least weight dropped), alone or together.

The selection never leaves the GPU: every focal layer writes into its own
fixed device buffer, and F_last *is* the deepest focal layer's buffer, which
that layer overwrites only after all of this step's earlier readers ran. All
buffers have fixed addresses, so a whole step can be captured in a CUDA
graph and replayed (fastocr calls allocate nothing).

This module only sequences library calls; all arithmetic is in the kernels.
"""
from __future__ import annotations

import math
import weakref

import torch

from . import _native as N


def keep_capacity(tau: float, n_img: int) -> int:
    """Columns needed for a selection buffer: an upper bound of ceil(tau*N_img)."""
    return max(1, min(n_img, int(math.ceil(tau * n_img)) + 1)) if n_img > 0 else 1


def ring_block_table(batch: int, prefix_len: int, window: int, page_size: int, max_tokens: int,
                     first_page: int = 0):
    """Block table that keeps an R-SWA cache in bounded memory (Unlimited OCR
    page, "R-SWA": the attend set is the global prefix plus a sliding window,
    so only those tokens need storage).

    Logical page j of sequence b maps to physical page
    first_page + b*P + (j if j < P0 else P0 + (j - P0) % R), with P0 =
    ceil(prefix_len / page_size) prefix pages, R = max(1, ceil(window /
    page_size)) ring pages and P = P0 + R pages per sequence, whatever
    max_tokens is. The caller writes token p's K/V to
    (table[b, p // page_size], p % page_size) as usual. Token p shares its
    row only with tokens p +- m*R*page_size, and R*page_size >= window, so a
    row is overwritten only after its token has left the window
    [N_t - window, N_t); the R-SWA kernels read nothing else outside the
    prefix. Returns (table [batch, ceil(max_tokens / page_size)] int32 on the
    CPU, P).
    """
    p0 = -(-prefix_len // page_size)
    ring = max(1, -(-window // page_size))
    per = p0 + ring
    n_pages = -(-max_tokens // page_size)
    j = torch.arange(n_pages, dtype=torch.int64)
    local = torch.where(j < p0, j, p0 + (j - p0) % ring)
    table = first_page + torch.arange(batch, dtype=torch.int64)[:, None] * per + local[None, :]
    return table.to(torch.int32), per


class ProfileSchedule:
    """Which decode steps profile the layers and which run the steady step.

    A profiling step runs full attention in every layer and adds each layer's
    image-attention mass to the profile; the last step of a window chooses the
    focal set C and F_last (FastOCR, "Focal-Guided Pruning": focal layer
    selection by a light warm-up). period None: one window, steps
    [0, window) -- the published method. A period P > window re-runs the
    window in steps [m*P, m*P + window) and re-chooses C each time, the
    plainest form of the adaptive layer selection that the FastOCR summaries
    name as future work; each window's profile starts from zero.
    """

    def __init__(self, window: int, period: int | None = None):
        if window < 0 or (period is not None and period <= window):
            raise ValueError("need 0 <= window < period")
        self.window, self.period = int(window), period

    def position(self, t: int) -> int:
        """Position of step t in its profiling window, -1 for a steady step."""
        pos = t if self.period is None else t % self.period
        return pos if pos < self.window else -1


class _Weights(dict):
    """What track_weights made; a dict that can be held weakly."""


class DecodeAttention:
    """Decode attention of a stack of layers over a paged KV cache.

    k_cache, v_cache: [layers, num_pages, H_kv, page_size, d] (bf16 or fp32)
    block_table: [B, pages_per_seq] int32; img_range: [B, 2] int32 (focal modes).
    """

    def __init__(self, k_cache, v_cache, block_table, *, q_heads: int, img_range=None,
                 max_img: int = 0, tau: float = 1.0, mode: str = "fastocr",
                 rswa_prefix: int = 0, rswa_window: int = 0, splits=None, variants=None,
                 score_reduce=None):
        dtype = N.check_caches(k_cache, v_cache)
        assert k_cache.is_cuda
        self.k_cache, self.v_cache = k_cache, v_cache
        self.layers, self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_cache.shape
        self.batch = block_table.shape[0]
        self.q_heads = q_heads
        self.mode = mode
        self.tau = float(tau)
        self.rswa_prefix, self.rswa_window = rswa_prefix, rswa_window
        dev = k_cache.device
        self.block_table = block_table.to(device=dev, dtype=torch.int32).contiguous()
        self.img_range = (img_range.to(device=dev, dtype=torch.int32).contiguous()
                          if img_range is not None else None)
        self.max_img = int(max_img)
        self.handle = N.fastocr_create(self.batch, q_heads, self.kv_heads, self.head_dim, dtype,
                                       self.page_size, self.block_table.shape[1], self.max_img,
                                       self.layers)
        if splits:
            for m, s in splits.items():
                N.fastocr_set_splits(self.handle, m, s)
        if variants:   # {mode slot: VARIANT_*}; tuning and tests only
            for m, v in variants.items():
                N.fastocr_set_variant(self.handle, m, v)
        self.seq_len = torch.zeros(self.batch, dtype=torch.int32, device=dev)
        self.kv = [N.make_kv(k_cache[l], v_cache[l], self.block_table, self.seq_len)
                   for l in range(self.layers)]
        self.stride = keep_capacity(self.tau, self.max_img)
        self.focal: tuple = ()
        self.sel = {}          # focal layer -> (idx [B, stride], k [B])
        self.warm_idx = None   # [layers, B, stride] selections made during warm-up
        self.warm_k = None
        self.has_f_last = False
        # Head-sharded focal layers: score_reduce(sigma) sums the [B, max_img]
        # fp32 score shares of all GPUs that hold this sequence's heads, in
        # place (e.g. an all-reduce); focal layers then score, reduce and
        # select in three steps instead of one call.
        self.score_reduce = score_reduce
        self.sigma = (torch.zeros(self.batch, max(self.max_img, 1), dtype=torch.float32,
                                  device=dev) if score_reduce is not None else None)
        self.hint = 0          # length the split choices assume (0: the cache's capacity)
        self.groups = None     # share_prefix
        self.weights = None    # track_weights
        self._tracked = []     # weak references to all weights still in use, captured steps' among them

    def close(self):
        if self.handle:
            N.fastocr_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------ set-up
    def _set_hint(self, n):
        self.hint = n
        N.fastocr_set_length_hint(self.handle, n)

    def set_seq_len(self, n_t):
        """N_t of the current step, int (all sequences) or [B] tensor. An int
        also becomes the handle's length hint (split choice only), which
        begin_token and evict_step carry on."""
        if isinstance(n_t, int):
            self.seq_len.fill_(n_t)
            self._set_hint(n_t)
        else:
            self.seq_len.copy_(n_t, non_blocking=True)

    def _per_sequence(self, x, name):
        """int or [B] -> [B] int32 on the cache's device (a tensor that is that is taken as it is)."""
        dev = self.k_cache.device
        if isinstance(x, int):
            return torch.full((self.batch,), x, dtype=torch.int32, device=dev)
        x = torch.as_tensor(x).to(device=dev, dtype=torch.int32).contiguous()
        if tuple(x.shape) != (self.batch,):
            raise ValueError(f"{name} must have one value a sequence, shape ({self.batch},)")
        return x

    def share_prefix(self, group_start, prefix_len, max_prefix: int | None = None):
        """Sequences group_start[i] .. group_start[i+1]-1 share rows [0, prefix_len)
        of group_start[i]'s pages (group_start from 0 to B; prefix_len int or
        [B], the same within a group). max_prefix: about the longest, for the
        split choice only; None takes it from prefix_len (which then
        synchronises, if it is on the device). Call it again when the groups
        change; a CapturedStep goes on with the groups it was captured with."""
        start = torch.as_tensor(group_start).to(torch.int32)
        if start.dim() != 1 or not 2 <= start.numel() <= self.batch + 1:
            raise ValueError("group_start must hold 2 .. B+1 offsets")
        if not start.is_cuda:
            s = start.tolist()
            if s[0] != 0 or s[-1] != self.batch or sorted(s) != s:
                raise ValueError(f"group_start must ascend from 0 to {self.batch}")
        prefix = self._per_sequence(prefix_len, "prefix_len")
        if max_prefix is None:
            max_prefix = prefix_len if isinstance(prefix_len, int) else int(prefix.max())
        start = start.to(self.k_cache.device).contiguous()
        ws_bytes = N.fastocr_rows_workspace(self.handle, 0)
        ws = (self.groups["ws"] if self.groups else
              torch.empty(ws_bytes, dtype=torch.uint8, device=self.k_cache.device))
        self.groups = {"start": start, "prefix_len": prefix, "ws": ws,
                       "c": N.make_groups(start, prefix, max_prefix)}

    def track_weights(self, rows: int, protect, *, mass=None, pos=None, seen=None):
        """Weights of up to `rows` rows behind protect (int or [B]: the prompt,
        the image, a shared prefix) in every layer, for weighed_step and evict_step.

        mass, pos: [layers, B, H_kv, rows] fp32 / int32, seen: [B] int32, taken as
        they are if given (e.g. with a prompt's weights in them); otherwise
        no weight, every row at its own position, and the tokens of seq_len
        (a prompt that is already in the cache). begin_token advances seen. A
        CapturedStep goes on with the weights it was captured with, whose seen
        begin_token advances too. A protect on the device is read back once."""
        if rows < 1:
            raise ValueError("rows must be at least 1")
        dev = self.k_cache.device
        shape = (self.layers, self.batch, self.kv_heads, rows)
        given = protect
        protect = self._per_sequence(protect, "protect")
        most = given if isinstance(given, int) else int(torch.as_tensor(given).max())
        if mass is None:
            mass = torch.zeros(shape, dtype=torch.float32, device=dev)
        if pos is None:
            pos = (protect[:, None, None] + torch.arange(rows, dtype=torch.int32, device=dev)
                   ).expand(shape).contiguous()
        if seen is None:
            seen = self.seq_len.clone()
        for x, want, dt in ((mass, shape, torch.float32), (pos, shape, torch.int32),
                            (seen, (self.batch,), torch.int32)):
            if tuple(x.shape) != want or x.dtype != dt or x.device != dev or not x.is_contiguous():
                raise ValueError(f"need a contiguous {dt} tensor of shape {want} on {dev}")
        logits = torch.empty((self.batch, self.kv_heads, rows, 8), dtype=torch.float32, device=dev)
        self.weights = _Weights(mass=mass, pos=pos, seen=seen, protect=protect, logits=logits,
                                new_len=torch.zeros_like(self.seq_len), most_protect=most,
                                c=[N.make_weights(mass[l], pos[l], protect, seen, logits)
                                   for l in range(self.layers)])
        self._tracked = [r for r in self._tracked if r() is not None] + [weakref.ref(self.weights)]

    def begin_token(self):
        """One more token in every sequence: N_t and, with weights, seen go up by
        one (on the device; write its K/V to row N_t - 1)."""
        self.seq_len.add_(1)
        if self.hint > 0:
            self._set_hint(self.hint + 1)
        seen = [w["seen"] for w in (r() for r in self._tracked) if w is not None]
        for x in {t.data_ptr(): t for t in seen}.values():   # one counter may serve several
            x.add_(1)

    def set_focal_layers(self, focal):
        self.focal = tuple(sorted(int(l) for l in focal))
        dev = self.k_cache.device
        self.sel = {l: (torch.zeros(self.batch, self.stride, dtype=torch.int32, device=dev),
                        torch.zeros(self.batch, dtype=torch.int32, device=dev))
                    for l in self.focal}

    def begin_warmup(self, stream=None):
        dev = self.k_cache.device
        self.warm_idx = torch.zeros(self.layers, self.batch, self.stride, dtype=torch.int32,
                                    device=dev)
        self.warm_k = torch.zeros(self.layers, self.batch, dtype=torch.int32, device=dev)
        N.fastocr_profiler_reset(self.handle, stream)

    def warmup_step(self, q, out, stream=None, hook=None, select=True):
        """Full attention in every layer, profiling image mass. select=False
        (what scheduled_step runs) only profiles (fastocr_profile_attend: one
        kernel a layer, no logits, scores or top-k), and finish_warmup(q=...)
        then selects on the deepest chosen layer alone; select=True also keeps
        every layer's selection, for finish_warmup to take F_last from."""
        for l in range(self.layers):
            if hook:
                hook(l, True)
            if select:
                N.fastocr_focal_attend(self.handle, q[l], self.kv[l], self.img_range, self.tau,
                                       out[l], self.warm_idx[l], self.stride, self.warm_k[l],
                                       profile_layer=l, stream=stream)
            else:
                N.fastocr_profile_attend(self.handle, q[l], self.kv[l], self.img_range, out[l],
                                         l, stream)
            if hook:
                hook(l, False)

    def finish_warmup(self, n_focal: int, stream=None, q=None):
        """Choose C from the profile; F_last = the last warm-up step's selection
        of max(C). q: that step's queries, when it only profiled (then the
        deepest chosen layer's selection is made now, by one focal call on
        the same queries and cache, so the step must directly precede this
        call); None when it selected in every layer (warmup_step(select=True))."""
        focal, mass = N.fastocr_profiler_select(self.handle, n_focal, self.layers, stream)
        self.set_focal_layers(focal)
        deepest = max(self.focal)
        idx, k = self.sel[deepest]
        if q is None:
            idx.copy_(self.warm_idx[deepest])
            k.copy_(self.warm_k[deepest])
        else:
            scratch = torch.empty_like(q[deepest])   # the step's output of this layer is in out
            N.fastocr_focal_attend(self.handle, q[deepest], self.kv[deepest], self.img_range,
                                   self.tau, scratch, idx, self.stride, k, -1, stream)
        self.has_f_last = True
        return focal, mass

    def scheduled_step(self, t: int, q, out, schedule: ProfileSchedule, n_focal: int,
                       stream=None):
        """Decode step t under `schedule`: a profiling step (the first of a window
        resets the profile, the last chooses C and F_last, synchronising the
        host) or the steady step. Returns C when this step chose it, else
        None; a CapturedStep of the steady step must then be captured anew,
        since it holds the previous focal layers."""
        pos = schedule.position(t)
        if pos < 0:
            self.step(q, out, stream)
            return None
        if pos == 0:
            self.begin_warmup(stream)
        # every step of the window only profiles; at its end the deepest
        # chosen layer selects on the last step's queries (F_last)
        self.warmup_step(q, out, stream, select=False)
        if pos == schedule.window - 1:
            return self.finish_warmup(n_focal, stream, q=q)[0]
        return None

    # ------------------------------------------------------------ checkpoint
    def state_dict(self, stream=None) -> dict:
        """The method's state between decode steps, on the host: the focal set
        C, the selections of the focal layers (the deepest one is F_last, the
        next step's carried selection) and, while a warm-up window is open, the
        profiler's accumulated image mass (with the per-layer selection buffers
        of warmup_step(select=True), which the scheduled window leaves unused);
        and the rows' weights and positions, if they are tracked.
        Synchronises the stream. The KV cache is the caller's and not part of it."""
        if stream is not None:
            stream.synchronize()
        else:
            torch.cuda.synchronize(self.k_cache.device)
        st = {"batch": self.batch, "layers": self.layers, "stride": self.stride,
              "tau": self.tau, "max_img": self.max_img, "focal": tuple(self.focal),
              "has_f_last": self.has_f_last,
              "sel": {l: (idx.cpu(), k.cpu()) for l, (idx, k) in self.sel.items()},
              "warm": None, "weights": None}
        if self.weights is not None:
            st["weights"] = {x: self.weights[x].cpu() for x in ("mass", "pos", "seen", "protect")}
        if self.warm_idx is not None:
            st["warm"] = (self.warm_idx.cpu(), self.warm_k.cpu(),
                          N.fastocr_profiler_read(self.handle, self.layers, stream))
        return st

    def load_state_dict(self, st: dict, stream=None) -> None:
        """Resume from state_dict() of a decoder over the same shapes and tau, and
        with as many weighed rows if it has any (ValueError, and nothing changes).
        With the same focal set the selection buffers keep their addresses
        (a CapturedStep of this decoder stays valid); another focal set gets
        new buffers, so a step must then be captured anew."""
        for key in ("batch", "layers", "stride", "tau", "max_img"):
            if st[key] != getattr(self, key):
                raise ValueError(f"checkpoint {key}={st[key]!r}, decoder has {getattr(self, key)!r}")
        weights = st.get("weights")   # looked at before anything is changed
        if weights is not None and (self.weights is None or any(self.weights[x].shape != t.shape
                                                                for x, t in weights.items())):
            raise ValueError("checkpoint has weights: call track_weights with as many rows first")
        if tuple(st["focal"]) != tuple(self.focal):
            if st["focal"]:
                self.set_focal_layers(st["focal"])
            else:
                self.focal, self.sel = (), {}
        for l, (idx, k) in st["sel"].items():
            self.sel[l][0].copy_(idx)
            self.sel[l][1].copy_(k)
        for x, t in (weights or {}).items():
            self.weights[x].copy_(t)
        self.has_f_last = bool(st["has_f_last"])
        if st["warm"] is None:
            self.warm_idx = self.warm_k = None
        else:
            warm_idx, warm_k, mass = st["warm"]
            dev = self.k_cache.device
            self.warm_idx = warm_idx.to(dev).contiguous()
            self.warm_k = warm_k.to(dev).contiguous()
            N.fastocr_profiler_load(self.handle, mass, stream)
        torch.cuda.synchronize(self.k_cache.device)

    # ------------------------------------------------------------ steps
    def focal_layer(self, l, q_l, out_l, idx, k, stream=None):
        """One focal layer: attention, image scores and the top-k selection."""
        if self.score_reduce is None:
            N.fastocr_focal_attend(self.handle, q_l, self.kv[l], self.img_range, self.tau,
                                   out_l, idx, self.stride, k, -1, stream)
            return
        N.fastocr_focal_scores(self.handle, q_l, self.kv[l], self.img_range, out_l, self.sigma,
                               self.sigma.shape[1], stream)
        self.score_reduce(self.sigma)
        N.fastocr_select(self.handle, self.kv[l], self.img_range, self.sigma,
                         self.sigma.shape[1], self.tau, idx, self.stride, k, stream)

    def step(self, q, out, stream=None, only=None, hook=None):
        """One steady FastOCR decode step over all layers (q, out: [L, B, H_q, d]).

        The first gather layer after a focal layer is told that the kernel
        right before it writes its selection (FASTOCR_SELECTION_PENDING: it
        lays the selection out after its wait); the step's first layer, which
        may follow the previous step's last selection kernel, checks the
        selection it staged early; every other gather layer is told that its
        selection is final (FASTOCR_SELECTION_FINAL).

        only="focal" / "sparse": issue just that kind's calls, with the same
        flags (per-kind timing). hook(l, before): called on the host right
        before and right after layer l's calls are issued (CapturedStep uses
        it to order per-layer host copies against the layers)."""
        cur = self.sel[max(self.focal)] if self.has_f_last else None
        flags = 0   # first layer: stage F_last early, check it after the wait
        for l in range(self.layers):
            if hook:
                hook(l, True)
            if l in self.sel:
                idx, k = self.sel[l]
                if only != "sparse":
                    self.focal_layer(l, q[l], out[l], idx, k, stream)
                cur = (idx, k)
                flags = N.SELECTION_PENDING
            else:
                if only == "focal":
                    pass
                elif cur is None:
                    N.fastocr_full_attend(self.handle, q[l], self.kv[l], out[l], stream)
                else:
                    N.fastocr_sparse_attend_ex(self.handle, q[l], self.kv[l], self.img_range,
                                               cur[0], self.stride, cur[1], out[l], flags, stream)
                flags = N.SELECTION_FINAL
            if hook:
                hook(l, False)
        if only is None:
            self.has_f_last = True

    def dense_step(self, q, out, stream=None, hook=None):
        for l in range(self.layers):
            if hook:
                hook(l, True)
            N.fastocr_full_attend(self.handle, q[l], self.kv[l], out[l], stream)
            if hook:
                hook(l, False)

    def rswa_step(self, q, out, stream=None, hook=None):
        for l in range(self.layers):
            if hook:
                hook(l, True)
            N.fastocr_rswa_attend(self.handle, q[l], self.kv[l], self.rswa_prefix,
                                  self.rswa_window, out[l], stream)
            if hook:
                hook(l, False)

    def _check_layer(self, q_l, out_l):
        shape = (self.batch, self.q_heads, self.head_dim)
        N.check_tensor(q_l, "q", shape, self.k_cache.dtype, self.k_cache.device)
        N.check_tensor(out_l, "out", shape, self.k_cache.dtype, self.k_cache.device)

    def shared_layer(self, l, q_l, out_l, stream=None):
        """Layer l of a step over shared prefixes (share_prefix); adds the rows'
        weights if they are tracked. q_l, out_l: [B, H_q, d], contiguous."""
        g = self.groups
        if g is None:
            raise RuntimeError("share_prefix has not been called")
        self._check_layer(q_l, out_l)
        N.fastocr_shared_attend(self.handle, q_l, self.kv[l], g["c"], out_l, g["ws"],
                                g["ws"].numel(), self.weights["c"][l] if self.weights else None,
                                stream)

    def shared_step(self, q, out, stream=None, hook=None):
        """Full attention in every layer, every group's prefix read once."""
        for l in range(self.layers):
            if hook:
                hook(l, True)
            self.shared_layer(l, q[l], out[l], stream)
            if hook:
                hook(l, False)

    def weigh_layer(self, l, q_l, out_l, stream=None):
        """Layer l of a step that adds every row's attention weight. q_l, out_l:
        [B, H_q, d], contiguous."""
        if self.weights is None:
            raise RuntimeError("track_weights has not been called")
        self._check_layer(q_l, out_l)
        N.fastocr_weigh_attend(self.handle, q_l, self.kv[l], self.weights["c"][l], out_l, stream)

    def weighed_step(self, q, out, stream=None, hook=None):
        """Full attention in every layer, adding every row's attention weight."""
        for l in range(self.layers):
            if hook:
                hook(l, True)
            self.weigh_layer(l, q[l], out[l], stream)
            if hook:
                hook(l, False)

    def evict_layer(self, l, budget, recent, new_len=None, stream=None):
        """Cut layer l's rows behind protect to `budget` a KV head, the `recent`
        newest among them; new_len [B] int32 gets the rows left. Something else
        (evict_step copies new_len) must run before the layer attends again."""
        if self.weights is None:
            raise RuntimeError("track_weights has not been called")
        if new_len is not None:
            N.check_tensor(new_len, "new_len", (self.batch,), torch.int32, self.k_cache.device)
        N.fastocr_evict(self.handle, self.kv[l], self.weights["c"][l], budget, recent, new_len,
                        stream)

    def evict_step(self, budget: int, recent: int, stream=None):
        """Cut every layer's rows and set seq_len (on the device) to the rows left."""
        if self.weights is None:
            raise RuntimeError("track_weights has not been called")
        new_len = self.weights["new_len"]
        for l in range(self.layers):
            self.evict_layer(l, budget, recent, new_len if l == self.layers - 1 else None, stream)
        if isinstance(stream, int):   # 0 is the default stream, which ExternalStream does not know
            dev = self.k_cache.device
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):   # None: the current one
            self.seq_len.copy_(new_len)
        left = max(1, self.weights["most_protect"] + budget)   # rows of the longest sequence, at most
        if self.hint > left:
            self._set_hint(left)

    def launches_per_step(self, kind: str) -> int:
        """Kernels one step of `kind` launches: one attend kernel per layer,
        plus the selection kernel of every focal (or profiling) layer, and two
        a layer over shared prefixes."""
        if kind == "fastocr":
            return self.layers + len(self.focal)
        if kind == "profile":
            return 2 * self.layers
        if kind == "shared":
            return 2 * self.layers
        return self.layers   # "profile_mass", "dense", "rswa", "weighed": one kernel a layer

    def device_status(self, stream=None) -> int:
        return N.fastocr_device_status(self.handle, stream)


class CapturedStep:
    """One decode step of `dec` captured in a CUDA graph over static buffers.

    q, out: [L, B, H_q, d] device tensors owned by this object; write the
    step's queries into q (and N_t into dec.seq_len), then replay(). kind:
    "fastocr" (steady FastOCR step), "dense" (full attention in every layer),
    "profile" (the last step of a profiling window: full attention with
    scoring, selection and profile accumulation in every layer),
    "profile_mass" (an earlier step of the window: full attention and
    profile accumulation only), "rswa", "shared" (share_prefix) or "weighed"
    (track_weights); or any name with `fn`, a
    callable fn(q, out, stream) that issues the calls (e.g. a subset of the
    step's layers), and `launches`, the kernels it launches.

    The step runs once, on zero queries, before it is captured. The rows'
    weights and positions are put back after that run, so only replays add to
    them; what a callable of the caller's own does in it stays.

    host_io=True (step kinds only) adds page-locked host buffers q_host and
    out_host, and the graph itself moves the step's queries in and its
    outputs out: write the queries into q_host, replay(), and out_host holds
    the outputs once the stream reaches the replay's end. The queries come in
    through fastocr_copy, a kernel in the step's chain of programmatic
    dependent launches (the first layer stages its K/V while it runs; a copy
    node there would leave a launch gap before the first layer). When the
    queries past the first SIDE_SPLIT layers hold at least side_copy_bytes
    (default 2 MB: at the ~170 GB/s of a host link that copy outlasts the
    7-10 us that a cross-stream wait before a kernel costs), those go in on a
    copy engine of a side stream instead, waited for by layer SIDE_SPLIT
    only. The outputs go out on a copy engine of another stream in chunks of
    L/2, L/4, ... layers (the last chunk one layer), each started when its
    last layer's calls are done.
    """

    SIDE_SPLIT = 4

    def __init__(self, dec: DecodeAttention, kind: str = "fastocr", fn=None,
                 launches: int | None = None, host_io: bool = False,
                 side_copy_bytes: int = 2 << 20):
        self.dec, self.kind = dec, kind
        # the graph's own, should share_prefix or track_weights be called again
        self._groups, self._weights = dec.groups, dec.weights
        self.side_copy_bytes = int(side_copy_bytes)
        shape = (dec.layers, dec.batch, dec.q_heads, dec.head_dim)
        self.q = torch.zeros(shape, dtype=dec.k_cache.dtype, device=dec.k_cache.device)
        self.out = torch.zeros_like(self.q)
        self.q_host = self.out_host = None
        if host_io:
            if fn is not None:
                raise ValueError("host_io captures one of the step kinds, not a custom fn")
            self.q_host = torch.zeros(shape, dtype=self.q.dtype, pin_memory=True)
            self.out_host = torch.zeros(shape, dtype=self.q.dtype, pin_memory=True)
        if kind in ("profile", "profile_mass") and dec.warm_idx is None:
            dec.begin_warmup()
        kept = {}   # what the warm run may not change
        if fn is None and kind in ("shared", "weighed") and dec.weights is not None:
            kept = {x: dec.weights[x] for x in ("mass", "pos")}
        if fn is None:   # otherwise fn(q, out, stream) issues the calls and `launches` counts them
            fn = {"fastocr": dec.step, "dense": dec.dense_step, "rswa": dec.rswa_step,
                  "shared": dec.shared_step, "weighed": dec.weighed_step,
                  "profile": dec.warmup_step,
                  "profile_mass": lambda q, out, stream=None, hook=None:
                      dec.warmup_step(q, out, stream, hook, select=False)}[kind]
            launches = dec.launches_per_step(kind)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            saved = {x: t.clone() for x, t in kept.items()}
            fn(self.q, self.out)             # warm run outside the capture
            for x, t in kept.items():
                t.copy_(saved[x])
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        if host_io:
            self._copy_in, self._copy_out = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.graph(self.graph):
            if host_io:
                self._issue_with_host_io(fn)
            else:
                fn(self.q, self.out)
        self.launches = launches

    @staticmethod
    def output_chunks(layers: int) -> list:
        """Last layer of each output chunk: chunks of half the layers left,
        the last one a single layer (28 layers: 13, 20, 23, 25, 26, 27)."""
        ends, a = [], 0
        while a < layers:
            n = max(1, (layers - a) // 2)
            ends.append(a + n - 1)
            a += n
        return ends

    def _issue_with_host_io(self, fn):
        main = torch.cuda.current_stream()
        s_in, s_out = self._copy_in, self._copy_out
        L = self.q.shape[0]
        per = self.q[0].numel() * self.q.element_size()
        k = min(self.SIDE_SPLIT, L)
        rest = None
        if k < L and (L - k) * per >= self.side_copy_bytes:   # 0 forces the side copy
            N.fastocr_copy(self.q[:k], self.q_host[:k], k * per)
            s_in.wait_stream(main)
            with torch.cuda.stream(s_in):
                self.q[k:].copy_(self.q_host[k:], non_blocking=True)
                rest = torch.cuda.Event()
                rest.record(s_in)
        else:
            N.fastocr_copy(self.q, self.q_host, L * per)
        s_out.wait_stream(main)
        ends = set(self.output_chunks(L))
        done, first = [], [0]

        def hook(l, before):
            if before:
                if rest is not None and l == k:
                    main.wait_event(rest)
                return
            if l not in ends:
                return
            ev = torch.cuda.Event()
            ev.record(main)
            done.append(ev)
            s_out.wait_event(ev)
            a = first[0]
            with torch.cuda.stream(s_out):
                self.out_host[a:l + 1].copy_(self.out[a:l + 1], non_blocking=True)
            first[0] = l + 1

        fn(self.q, self.out, hook=hook)
        if rest is not None:
            main.wait_stream(s_in)
        main.wait_stream(s_out)
        self._events = done + ([rest] if rest is not None else [])   # alive with the graph

    def replay(self):
        self.graph.replay()
