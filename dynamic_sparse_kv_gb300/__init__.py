"""GB300-native decode attention of FastOCR (focal layers, top-tau image-token
selection, gather attention, Cross-Step Fixation Reuse) and R-SWA.

The compute path is libfastocr.so (CUDA, sm_103a) behind the C ABI of
include/fastocr.h; `_native` binds it with ctypes under the same names, and
`decoder.DecodeAttention` sequences the per-layer calls of a decode step.
Importing this package loads the library and fails if it is not built.
"""
from . import _native  # noqa: F401  (loads libfastocr.so or raises)
from ._native import (  # noqa: F401
    fastocr_abi_version, fastocr_create, fastocr_cross_attend, fastocr_destroy,
    fastocr_device_status, fastocr_evict, fastocr_focal_attend, fastocr_full_attend,
    fastocr_pool_compact, fastocr_pool_copy, fastocr_pool_fork, fastocr_pool_release,
    fastocr_pool_reserve, fastocr_pool_trim, fastocr_pool_workspace, fastocr_profiler_reset,
    fastocr_profiler_select, fastocr_read_rows, fastocr_rows_workspace, fastocr_rswa_attend,
    fastocr_set_length_hint, fastocr_set_splits, fastocr_shared_attend, fastocr_sparse_attend,
    fastocr_weigh_attend, fastocr_write_rows, make_groups, make_kv, make_weights)
from .cross import CrossAttention  # noqa: F401
from .decoder import (CapturedStep, DecodeAttention, ProfileSchedule, keep_capacity,  # noqa: F401
                      ring_block_table)
from .fp4 import Fp4Cache  # noqa: F401
from .pages import PagePool  # noqa: F401
from .rotary import Rotary  # noqa: F401
