"""ctypes binding of libfastocr.so: the C ABI of include/fastocr.h, same names.

Argument marshalling only -- every step of the decode-attention path runs in
the library's CUDA kernels. Tensors are PyTorch tensors on the GPU; their
data pointers are handed to the library as they are (no copies, no casts).
If the library is missing this module raises at import: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfastocr.so")

FASTOCR_OK = 0
FASTOCR_ERR_NULL = -1
FASTOCR_ERR_INVALID = -2
FASTOCR_ERR_UNSUPPORTED = -3
FASTOCR_ERR_CUDA = -4
FASTOCR_ERR_NO_DEVICE = -5
FASTOCR_ERR_ALIGN = -6
FASTOCR_DTYPE_F32 = 0
FASTOCR_DTYPE_BF16 = 1
FASTOCR_DTYPE_FP4 = 2
DEV_BAD_PAGE, DEV_BAD_SEQLEN, DEV_BAD_IMG, DEV_BAD_SELECTION, DEV_INTERNAL = 1, 2, 4, 8, 16
DEV_BAD_GROUP, DEV_BAD_WEIGHTS = 32, 64
DEV_BAD_POSITION, DEV_NO_PAGES, DEV_BAD_POOL = 128, 256, 512


class fastocr_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("max_img_tokens", ctypes.c_int32),
                ("num_layers", ctypes.c_int32)]


class fastocr_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_gain", ctypes.c_void_p), ("v_gain", ctypes.c_void_p)]


class fastocr_rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("axis", ctypes.c_void_p),
                ("positions", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("adjacent", ctypes.c_int32)]


class fastocr_tokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("start", ctypes.c_void_p),
                ("tokens", ctypes.c_int32)]


class fastocr_pool(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("held", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_layer", ctypes.c_int64), ("v_layer", ctypes.c_int64),
                ("k_scale_layer", ctypes.c_int64), ("v_scale_layer", ctypes.c_int64),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_int64)]


class fastocr_groups(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("n", ctypes.c_int32), ("max_prefix", ctypes.c_int32)]


class fastocr_weights(ctypes.Structure):
    _fields_ = [("mass", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("protect", ctypes.c_void_p), ("seen", ctypes.c_void_p),
                ("logits", ctypes.c_void_p), ("stride", ctypes.c_int32)]


class FastOCRError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python dynamic_sparse_kv_gb300/build.py` "
            "(or __graft_entry__.build()) -- there is no CPU fallback")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    sigs = {
        "fastocr_abi_version": ([], I32),
        "fastocr_status_string": ([I32], ctypes.c_char_p),
        "fastocr_create": ([ctypes.POINTER(fastocr_dims), ctypes.POINTER(P)], I32),
        "fastocr_destroy": ([P], I32),
        "fastocr_full_attend": ([P, P, ctypes.POINTER(fastocr_kv), P, P], I32),
        "fastocr_focal_attend": ([P, P, ctypes.POINTER(fastocr_kv), P, F64, P, P, I32, P, I32, P],
                                 I32),
        "fastocr_focal_scores": ([P, P, ctypes.POINTER(fastocr_kv), P, P, P, I32, P], I32),
        "fastocr_profile_attend": ([P, P, ctypes.POINTER(fastocr_kv), P, P, I32, P], I32),
        "fastocr_select": ([P, ctypes.POINTER(fastocr_kv), P, P, I32, F64, P, I32, P, P], I32),
        "fastocr_sparse_attend": ([P, P, ctypes.POINTER(fastocr_kv), P, P, I32, P, P, P], I32),
        "fastocr_sparse_attend_ex": ([P, P, ctypes.POINTER(fastocr_kv), P, P, I32, P, P,
                                      ctypes.c_uint32, P], I32),
        "fastocr_rswa_attend": ([P, P, ctypes.POINTER(fastocr_kv), I32, I32, P, P], I32),
        "fastocr_rows_workspace": ([P, I64], I64),
        "fastocr_shared_attend": ([P, P, ctypes.POINTER(fastocr_kv),
                                   ctypes.POINTER(fastocr_groups),
                                   ctypes.POINTER(fastocr_weights), P, P, I64, P], I32),
        "fastocr_weigh_attend": ([P, P, ctypes.POINTER(fastocr_kv),
                                  ctypes.POINTER(fastocr_weights), P, P], I32),
        "fastocr_evict": ([P, ctypes.POINTER(fastocr_kv), ctypes.POINTER(fastocr_weights), I32,
                           I32, P, P], I32),
        "fastocr_cross_attend": ([P, P, ctypes.POINTER(fastocr_kv), P, I64, P, P, I64, P], I32),
        "fastocr_write_rows": ([P, ctypes.POINTER(fastocr_kv), ctypes.POINTER(fastocr_tokens),
                                ctypes.POINTER(fastocr_rotary), P], I32),
        "fastocr_read_rows": ([P, ctypes.POINTER(fastocr_kv), P, I32, P, P, I32, P], I32),
        "fastocr_pool_workspace": ([P, I64], I64),
        "fastocr_pool_reserve": ([P, ctypes.POINTER(fastocr_pool), P, I32, P, P], I32),
        "fastocr_pool_fork": ([P, ctypes.POINTER(fastocr_pool), P, P, I32, P], I32),
        "fastocr_pool_release": ([P, ctypes.POINTER(fastocr_pool), P, I32, P], I32),
        "fastocr_pool_trim": ([P, ctypes.POINTER(fastocr_pool), P], I32),
        "fastocr_pool_compact": ([P, ctypes.POINTER(fastocr_pool), P, P], I32),
        "fastocr_pool_copy": ([P, ctypes.POINTER(fastocr_pool), P, P, I32, P], I32),
        "fastocr_profiler_reset": ([P, P], I32),
        "fastocr_profiler_select": ([P, I32, ctypes.POINTER(I32), ctypes.POINTER(F64), P], I32),
        "fastocr_profiler_read": ([P, ctypes.POINTER(F64), P], I32),
        "fastocr_profiler_load": ([P, ctypes.POINTER(F64), P], I32),
        "fastocr_device_status": ([P, ctypes.POINTER(I32), P], I32),
        "fastocr_set_splits": ([P, I32, I32], I32),
        "fastocr_set_variant": ([P, I32, I32], I32),
        "fastocr_set_length_hint": ([P, I32], I32),
        "fastocr_read_probe": ([P, ctypes.c_int64, P, P], I32),
        "fastocr_copy": ([P, P, ctypes.c_int64, P], I32),
        "fastocr_focal_attend_noalloc": ([ctypes.POINTER(fastocr_dims), P,
                                          ctypes.POINTER(fastocr_kv), P, F64, P, P, I32, P, P, P],
                                         I32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.fastocr_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != FASTOCR_OK:
        raise FastOCRError(fn, status)


def check_tensor(t, name, shape, dtype, device) -> None:
    """Refuse a tensor that the library would read or write wrongly: it gets the bare address."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}, not {t.dtype} {tuple(t.shape)} on {t.device}"
                         + ("" if t.is_contiguous() else f" with strides {t.stride()}"))


def check_caches(k, v) -> int:
    """The dtype code of a stack's caches [layers, pages, H_kv, page, d] (two tensors or two
    Fp4Cache); refuses what the kernels would read wrongly. Layers may lie apart, each must
    be contiguous."""
    if getattr(k, "fp4", False) or getattr(v, "fp4", False):
        if not (getattr(k, "fp4", False) and getattr(v, "fp4", False)) or k.shape != v.shape or k.device != v.device:
            raise ValueError("k_cache and v_cache must be alike: two Fp4Cache of one shape and device")
        k.check()
        v.check()
        return FASTOCR_DTYPE_FP4
    if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
        raise ValueError("k_cache and v_cache must be alike, [layers, pages, H_kv, page_size, d]")
    if k.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"caches must be bfloat16 or float32, not {k.dtype}")
    if not (k[0].is_contiguous() and v[0].is_contiguous()):
        raise ValueError("a layer's cache must be contiguous")
    return FASTOCR_DTYPE_BF16 if k.dtype == torch.bfloat16 else FASTOCR_DTYPE_F32


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:   # the current stream without the Stream object around it (0.3 us, not 2.9)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fastocr_abi_version() -> int:
    return lib.fastocr_abi_version()


def fastocr_create(batch, num_q_heads, num_kv_heads, head_dim, dtype, page_size,
                   max_pages_per_seq, max_img_tokens, num_layers) -> int:
    dims = fastocr_dims(batch, num_q_heads, num_kv_heads, head_dim, dtype, page_size,
                        max_pages_per_seq, max_img_tokens, num_layers)
    h = ctypes.c_void_p()
    _check("fastocr_create", lib.fastocr_create(ctypes.byref(dims), ctypes.byref(h)))
    return h.value


def fastocr_destroy(handle: int) -> None:
    _check("fastocr_destroy", lib.fastocr_destroy(handle))


def make_kv(k, v, block_table, seq_len) -> fastocr_kv:
    """One layer's cache descriptor; keeps no reference to the tensors. k, v: two tensors,
    or what an Fp4Cache gives for a layer."""
    if isinstance(k, tuple):   # codes, scales, gain
        return fastocr_kv(_ptr(k[0]), _ptr(v[0]), _ptr(block_table), _ptr(seq_len), int(k[0].shape[0]),
                          _ptr(k[1]), _ptr(v[1]), _ptr(k[2]), _ptr(v[2]))
    return fastocr_kv(_ptr(k), _ptr(v), _ptr(block_table), _ptr(seq_len), int(k.shape[0]))


def fastocr_full_attend(handle, q, kv: fastocr_kv, out, stream=None) -> None:
    _check("fastocr_full_attend",
           lib.fastocr_full_attend(handle, _ptr(q), ctypes.byref(kv), _ptr(out), _stream(stream)))


def fastocr_focal_attend(handle, q, kv: fastocr_kv, img_range, tau, out, idx, idx_stride, k_out,
                         profile_layer=-1, stream=None) -> None:
    _check("fastocr_focal_attend",
           lib.fastocr_focal_attend(handle, _ptr(q), ctypes.byref(kv), _ptr(img_range),
                                    float(tau), _ptr(out), _ptr(idx), int(idx_stride),
                                    _ptr(k_out), int(profile_layer), _stream(stream)))


def fastocr_profile_attend(handle, q, kv: fastocr_kv, img_range, out, profile_layer,
                           stream=None) -> None:
    """Full attention that adds the layer's image mass to the profiler; no selection."""
    _check("fastocr_profile_attend",
           lib.fastocr_profile_attend(handle, _ptr(q), ctypes.byref(kv), _ptr(img_range),
                                      _ptr(out), int(profile_layer), _stream(stream)))


def fastocr_focal_scores(handle, q, kv: fastocr_kv, img_range, out, sigma, sigma_stride,
                         stream=None) -> None:
    _check("fastocr_focal_scores",
           lib.fastocr_focal_scores(handle, _ptr(q), ctypes.byref(kv), _ptr(img_range), _ptr(out),
                                    _ptr(sigma), int(sigma_stride), _stream(stream)))


def fastocr_select(handle, kv: fastocr_kv, img_range, sigma, sigma_stride, tau, idx, idx_stride,
                   k_out, stream=None) -> None:
    _check("fastocr_select",
           lib.fastocr_select(handle, ctypes.byref(kv), _ptr(img_range), _ptr(sigma),
                              int(sigma_stride), float(tau), _ptr(idx), int(idx_stride),
                              _ptr(k_out), _stream(stream)))


def fastocr_sparse_attend(handle, q, kv: fastocr_kv, img_range, idx, idx_stride, k, out,
                          stream=None) -> None:
    _check("fastocr_sparse_attend",
           lib.fastocr_sparse_attend(handle, _ptr(q), ctypes.byref(kv), _ptr(img_range),
                                     _ptr(idx), int(idx_stride), _ptr(k), _ptr(out),
                                     _stream(stream)))


SELECTION_FINAL = 1     # FASTOCR_SELECTION_FINAL
SELECTION_PENDING = 2   # FASTOCR_SELECTION_PENDING


def fastocr_sparse_attend_ex(handle, q, kv: fastocr_kv, img_range, idx, idx_stride, k, out,
                             flags: int, stream=None) -> None:
    """fastocr_sparse_attend with flags; SELECTION_FINAL: idx and k were written
    before the kernel preceding this call on the stream began."""
    _check("fastocr_sparse_attend_ex",
           lib.fastocr_sparse_attend_ex(handle, _ptr(q), ctypes.byref(kv), _ptr(img_range),
                                        _ptr(idx), int(idx_stride), _ptr(k), _ptr(out),
                                        int(flags), _stream(stream)))


def fastocr_rswa_attend(handle, q, kv: fastocr_kv, prefix_len, window, out, stream=None) -> None:
    _check("fastocr_rswa_attend",
           lib.fastocr_rswa_attend(handle, _ptr(q), ctypes.byref(kv), int(prefix_len),
                                   int(window), _ptr(out), _stream(stream)))


def fastocr_rows_workspace(handle, rows) -> int:
    """Workspace bytes of fastocr_cross_attend over up to `rows` query tokens, or of
    fastocr_shared_attend (rows = 0)."""
    n = lib.fastocr_rows_workspace(handle, int(rows))
    if n < 0:
        raise FastOCRError("fastocr_rows_workspace", int(n))
    return n


def make_groups(start, prefix_len, max_prefix=0) -> fastocr_groups:
    """Groups of sequences that share a prefix; keeps no reference to the tensors."""
    return fastocr_groups(_ptr(start), _ptr(prefix_len), int(start.shape[0]) - 1, int(max_prefix))


def make_weights(mass, pos, protect, seen, logits) -> fastocr_weights:
    """One layer's weights; keeps no reference to the tensors."""
    return fastocr_weights(_ptr(mass), _ptr(pos), _ptr(protect), _ptr(seen), _ptr(logits),
                           int(mass.shape[-1]))


def fastocr_shared_attend(handle, q, kv: fastocr_kv, groups: fastocr_groups, out, ws, ws_bytes,
                          weights: fastocr_weights | None = None, stream=None) -> None:
    """Decode attention with a prefix shared by groups of sequences, read once a group."""
    w = ctypes.byref(weights) if weights is not None else None
    _check("fastocr_shared_attend",
           lib.fastocr_shared_attend(handle, _ptr(q), ctypes.byref(kv), ctypes.byref(groups), w,
                                     _ptr(out), _ptr(ws), int(ws_bytes), _stream(stream)))


def fastocr_weigh_attend(handle, q, kv: fastocr_kv, weights: fastocr_weights, out,
                         stream=None) -> None:
    """Full attention that adds every row's attention weight to its accumulator."""
    _check("fastocr_weigh_attend",
           lib.fastocr_weigh_attend(handle, _ptr(q), ctypes.byref(kv), ctypes.byref(weights),
                                    _ptr(out), _stream(stream)))


def fastocr_evict(handle, kv: fastocr_kv, weights: fastocr_weights, budget, recent, new_len=None,
                  stream=None) -> None:
    """Keep `budget` rows behind protect a KV head: recent ones, then the largest weights."""
    _check("fastocr_evict",
           lib.fastocr_evict(handle, ctypes.byref(kv), ctypes.byref(weights), int(budget),
                             int(recent), _ptr(new_len), _stream(stream)))


def fastocr_cross_attend(handle, q, kv: fastocr_kv, q_start, rows, out, ws, ws_bytes,
                         stream=None) -> None:
    """Packed, ragged queries against all states of their sequence."""
    _check("fastocr_cross_attend",
           lib.fastocr_cross_attend(handle, _ptr(q), ctypes.byref(kv), _ptr(q_start), int(rows),
                                    _ptr(out), _ptr(ws), int(ws_bytes), _stream(stream)))


def fastocr_write_rows(handle, kv: fastocr_kv, tokens: fastocr_tokens, rotary: fastocr_rotary | None = None,
                       stream=None) -> None:
    """Tokens to their rows of one layer's cache, with rotary positions for queries and keys."""
    r = ctypes.byref(rotary) if rotary is not None else None
    _check("fastocr_write_rows",
           lib.fastocr_write_rows(handle, ctypes.byref(kv), ctypes.byref(tokens), r, _stream(stream)))


def fastocr_read_rows(handle, kv: fastocr_kv, start, tokens, k_out, v_out, out_dtype, stream=None) -> None:
    """The last rows of every sequence, packed, as bf16 or fp32 values."""
    _check("fastocr_read_rows",
           lib.fastocr_read_rows(handle, ctypes.byref(kv), _ptr(start), int(tokens), _ptr(k_out),
                                 _ptr(v_out), int(out_dtype), _stream(stream)))


def fastocr_pool_workspace(handle, num_pages) -> int:
    n = lib.fastocr_pool_workspace(handle, int(num_pages))
    if n < 0:
        raise FastOCRError("fastocr_pool_workspace", int(n))
    return n


def fastocr_pool_reserve(handle, pool: fastocr_pool, rows, extra, missing=None, stream=None) -> None:
    """Pages for every sequence's next rows, shared ones copied before they are written."""
    _check("fastocr_pool_reserve",
           lib.fastocr_pool_reserve(handle, ctypes.byref(pool), _ptr(rows), int(extra), _ptr(missing),
                                    _stream(stream)))


def fastocr_pool_fork(handle, pool: fastocr_pool, src, dst, n, stream=None) -> None:
    """Sequences dst become copies of src that share their pages."""
    _check("fastocr_pool_fork",
           lib.fastocr_pool_fork(handle, ctypes.byref(pool), _ptr(src), _ptr(dst), int(n), _stream(stream)))


def fastocr_pool_release(handle, pool: fastocr_pool, seqs, n, stream=None) -> None:
    """Sequences give up their pages."""
    _check("fastocr_pool_release",
           lib.fastocr_pool_release(handle, ctypes.byref(pool), _ptr(seqs), int(n), _stream(stream)))


def fastocr_pool_trim(handle, pool: fastocr_pool, stream=None) -> None:
    """Every sequence gives up the pages behind its rows."""
    _check("fastocr_pool_trim", lib.fastocr_pool_trim(handle, ctypes.byref(pool), _stream(stream)))


def fastocr_pool_compact(handle, pool: fastocr_pool, used=None, stream=None) -> None:
    """The pages in use move together at the pool's start."""
    _check("fastocr_pool_compact",
           lib.fastocr_pool_compact(handle, ctypes.byref(pool), _ptr(used), _stream(stream)))


def fastocr_pool_copy(handle, pool: fastocr_pool, src, dst, n, stream=None) -> None:
    """Pages src to pages dst, in every layer."""
    _check("fastocr_pool_copy",
           lib.fastocr_pool_copy(handle, ctypes.byref(pool), _ptr(src), _ptr(dst), int(n), _stream(stream)))


def fastocr_profiler_reset(handle, stream=None) -> None:
    _check("fastocr_profiler_reset", lib.fastocr_profiler_reset(handle, _stream(stream)))


def fastocr_profiler_select(handle, n_focal, num_layers, stream=None):
    """Returns (focal layer ids ascending, image mass of every layer)."""
    layers = (ctypes.c_int32 * n_focal)()
    ratio = (ctypes.c_double * num_layers)()
    _check("fastocr_profiler_select",
           lib.fastocr_profiler_select(handle, int(n_focal), layers, ratio, _stream(stream)))
    return tuple(int(x) for x in layers), [float(x) for x in ratio]


def fastocr_profiler_read(handle, num_layers, stream=None) -> list:
    """The accumulated image mass of every layer (synchronises the stream)."""
    mass = (ctypes.c_double * num_layers)()
    _check("fastocr_profiler_read", lib.fastocr_profiler_read(handle, mass, _stream(stream)))
    return [float(x) for x in mass]


def fastocr_profiler_load(handle, mass, stream=None) -> None:
    """Load the accumulated image mass of every layer (len(mass) = num_layers)."""
    arr = (ctypes.c_double * len(mass))(*[float(x) for x in mass])
    _check("fastocr_profiler_load", lib.fastocr_profiler_load(handle, arr, _stream(stream)))


def fastocr_device_status(handle, stream=None) -> int:
    s = ctypes.c_int32()
    _check("fastocr_device_status",
           lib.fastocr_device_status(handle, ctypes.byref(s), _stream(stream)))
    return int(s.value)


def fastocr_set_length_hint(handle, n_t) -> None:
    _check("fastocr_set_length_hint", lib.fastocr_set_length_hint(handle, int(n_t)))


def fastocr_set_splits(handle, mode, splits) -> None:
    _check("fastocr_set_splits", lib.fastocr_set_splits(handle, int(mode), int(splits)))


VARIANT_AUTO, VARIANT_GENERAL, VARIANT_DEEP = 0, 1, 2


def fastocr_set_variant(handle, mode, variant) -> None:
    _check("fastocr_set_variant", lib.fastocr_set_variant(handle, int(mode), int(variant)))


NOALLOC_MAX_UNITS_IMG = 65536   # FASTOCR_NOALLOC_MAX_UNITS_IMG


def fastocr_focal_attend_noalloc(dims: fastocr_dims, q, kv: fastocr_kv, img_range, tau, out, idx,
                                 idx_stride, k_out, status, stream=None) -> None:
    """Focal layer without a handle, for callers that may not allocate GPU
    memory where they run; its scratch is a fixed array inside the library."""
    _check("fastocr_focal_attend_noalloc",
           lib.fastocr_focal_attend_noalloc(ctypes.byref(dims), _ptr(q), ctypes.byref(kv),
                                            _ptr(img_range), float(tau), _ptr(out), _ptr(idx),
                                            int(idx_stride), _ptr(k_out), _ptr(status),
                                            _stream(stream)))


def fastocr_copy(dst, src, nbytes, stream=None) -> None:
    """Copy nbytes from src to dst with the SMs (device or page-locked host memory)."""
    _check("fastocr_copy", lib.fastocr_copy(_ptr(dst), _ptr(src), int(nbytes), _stream(stream)))


def fastocr_read_probe(src, nbytes, sink, stream=None) -> None:
    """Read nbytes of device memory at src once (read-only bandwidth probe)."""
    _check("fastocr_read_probe",
           lib.fastocr_read_probe(_ptr(src), int(nbytes), _ptr(sink), _stream(stream)))
