// C ABI of the shared-prefix, weighing, eviction and cross-attention calls
// (declared in include/fastocr.h): argument checks, splits and launches.
#include <stdint.h>

#include "evict.cuh"
#include "handle.cuh"
#include "rows.cuh"
#include "rows_plan.cuh"

using namespace fastocr;

namespace {

fastocr_status check_device(const fastocr_handle* h) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FASTOCR_ERR_NO_DEVICE;
  return dev == h->device ? FASTOCR_OK : FASTOCR_ERR_INVALID;
}

fastocr_status check_weights(const fastocr_weights* w, bool attend) {
  if (!w || !w->mass || !w->pos || !w->protect || !w->seen || (attend && !w->logits))
    return FASTOCR_ERR_NULL;
  if (w->stride < 1) return FASTOCR_ERR_INVALID;
  if (attend && !aligned16(w->logits)) return FASTOCR_ERR_ALIGN;
  return FASTOCR_OK;
}

void set_weights(const fastocr_weights* w, Params& p) {
  p.mass = w->mass;
  p.row_pos = w->pos;
  p.protect = w->protect;
  p.seen = w->seen;
  p.w_logits = w->logits;
  p.w_stride = w->stride;
}

RowsParams rows_params(const fastocr_handle* h, const void* q, const fastocr_kv* kv) {
  RowsParams p;
  memset(&p, 0, sizeof(p));
  const fastocr_dims& d = h->dims;
  p.q = q;
  p.k = kv->k;
  p.v = kv->v;
  p.block_table = kv->block_table;
  p.seq_len = kv->seq_len;
  p.num_pages = kv->num_pages;
  p.max_pages = d.max_pages_per_seq;
  p.log2_page = h->log2_page;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.g = d.num_q_heads / d.num_kv_heads;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d.head_dim));
  p.status = h->status;
  return p;
}

// Lays the workspace out for `rows` query tokens from `base` on and returns its
// size: the slots, then what the readers of the parts need (see rows.cuh).
int64_t place_workspace(const fastocr_handle* h, int64_t rows, bool shared, char* base, RowsParams& p) {
  const int64_t d = h->dims.head_dim, Hq = h->dims.num_q_heads, Hkv = h->dims.num_kv_heads;
  const int64_t sr = slot_rows(h, rows), slots = 2 * (int64_t)h->num_sms * sr;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    char* x = base + at;
    at = align_up(at + (size_t)bytes, 256);
    return x;
  };
  p.slot_rows = (int)sr;
  p.slot_acc = reinterpret_cast<float*>(take(slots * d * 4));
  p.slot_ml = reinterpret_cast<float*>(take(slots * 8));
  if (shared) {
    p.token_part = reinterpret_cast<int4*>(take(rows * Hkv * 16));
    p.row_acc = reinterpret_cast<float*>(take(rows * Hq * d * 4));
    p.row_ml = reinterpret_cast<float*>(take(rows * Hq * 8));
  } else {
    p.item_part = reinterpret_cast<int4*>(take((int64_t)h->num_sms * 32));
  }
  return (int64_t)at;
}

fastocr_status launch_rows(const fastocr_handle* h, const RowsParams& p, cudaStream_t s) {
  const cudaError_t e = h->dims.dtype == FASTOCR_DTYPE_BF16 ? launch_rows_bf16(h->dims.head_dim, h->num_sms, p, s)
                                                            : launch_rows_f32(h->dims.head_dim, h->num_sms, p, s);
  return e == cudaSuccess ? FASTOCR_OK : FASTOCR_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t fastocr_rows_workspace(const fastocr_handle* h, int64_t rows) {
  if (!h) return FASTOCR_ERR_NULL;
  if (rows < 0 || rows * h->dims.num_q_heads >= (1LL << 31)) return FASTOCR_ERR_INVALID;
  RowsParams p;
  return place_workspace(h, rows > 0 ? rows : h->dims.batch, rows == 0, nullptr, p);
}

fastocr_status fastocr_shared_attend(fastocr_handle* h, const void* q, const fastocr_kv* kv,
                                     const fastocr_groups* groups, const fastocr_weights* weights,
                                     void* out, void* ws, int64_t ws_bytes, fastocr_stream stream) {
  if (!h || !q || !out || !groups || !groups->start || !groups->prefix_len || !ws)
    return FASTOCR_ERR_NULL;
  fastocr_status st = check_kv(h, kv);
  if (st != FASTOCR_OK) return st;
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return FASTOCR_ERR_ALIGN;
  const int64_t B = h->dims.batch;
  if (groups->n < 1 || groups->n > B || groups->max_prefix < 0) return FASTOCR_ERR_INVALID;
  if (weights && (st = check_weights(weights, true)) != FASTOCR_OK) return st;
  RowsParams r = rows_params(h, q, kv);
  if (ws_bytes < place_workspace(h, B, true, static_cast<char*>(ws), r)) return FASTOCR_ERR_INVALID;
  if (!units_fit(h, B, groups->n)) return FASTOCR_ERR_UNSUPPORTED;
  if ((st = check_device(h)) != FASTOCR_OK) return st;

  r.n_groups = groups->n;
  r.start = groups->start;
  r.prefix_len = groups->prefix_len;
  r.rows = (int)B;
  const long keys = groups->max_prefix > 0 ? groups->max_prefix : expected_tokens(h);
  r.tile_tokens = choose_tile_tokens(h, B, groups->n, keys);
  r.min_share = choose_share(h, B, keys);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = launch_rows(h, r, s)) != FASTOCR_OK) return st;

  const long all = expected_tokens(h);
  const long prefix = groups->max_prefix > 0 ? std::min<long>(groups->max_prefix, all) : 0;
  Params p = base_params(h, q, kv, out);
  p.first = groups->prefix_len;
  p.ext_part = r.token_part;
  p.ext_slot_acc = r.slot_acc;
  p.ext_slot_ml = r.slot_ml;
  p.ext_row_acc = r.row_acc;
  p.ext_row_ml = r.row_ml;
  p.ext_slot_rows = r.slot_rows;
  p.ext_ctas = h->num_sms;
  if (weights) set_weights(weights, p);
  return launch(h, weights ? kWeigh : kTail, std::max(1L, all - prefix), p, stream);
}

fastocr_status fastocr_weigh_attend(fastocr_handle* h, const void* q, const fastocr_kv* kv,
                                    const fastocr_weights* weights, void* out,
                                    fastocr_stream stream) {
  if (!h || !q || !out) return FASTOCR_ERR_NULL;
  fastocr_status st = check_kv(h, kv);
  if (st != FASTOCR_OK) return st;
  if (!aligned16(q) || !aligned16(out)) return FASTOCR_ERR_ALIGN;
  if ((st = check_weights(weights, true)) != FASTOCR_OK) return st;
  if ((st = check_device(h)) != FASTOCR_OK) return st;
  Params p = base_params(h, q, kv, out);
  set_weights(weights, p);
  return launch(h, kWeigh, expected_tokens(h), p, stream);
}

fastocr_status fastocr_evict(fastocr_handle* h, const fastocr_kv* kv, const fastocr_weights* weights,
                             int32_t budget, int32_t recent, int32_t* new_len,
                             fastocr_stream stream) {
  if (!h) return FASTOCR_ERR_NULL;
  fastocr_status st = check_kv(h, kv);
  if (st != FASTOCR_OK) return st;
  if ((st = check_weights(weights, false)) != FASTOCR_OK) return st;
  if (budget < 1 || recent < 0 || recent > budget) return FASTOCR_ERR_INVALID;
  if (new_len && new_len == kv->seq_len) return FASTOCR_ERR_INVALID;
  const int rows = (int)std::min<long>(weights->stride, max_tokens(h));
  if (rows > (long)kEvictSlice * kEvictCluster) return FASTOCR_ERR_UNSUPPORTED;
  if ((st = check_device(h)) != FASTOCR_OK) return st;
  EvictParams p;
  memset(&p, 0, sizeof(p));
  const fastocr_dims& d = h->dims;
  p.k = static_cast<char*>(const_cast<void*>(kv->k));
  p.v = static_cast<char*>(const_cast<void*>(kv->v));
  p.block_table = kv->block_table;
  p.seq_len = kv->seq_len;
  p.num_pages = kv->num_pages;
  p.max_pages = d.max_pages_per_seq;
  p.log2_page = h->log2_page;
  p.B = d.batch;
  p.Hkv = d.num_kv_heads;
  p.row_bytes = d.head_dim * (d.dtype == FASTOCR_DTYPE_BF16 ? 2 : 4);
  p.mass = weights->mass;
  p.pos = weights->pos;
  p.protect = weights->protect;
  p.seen = weights->seen;
  p.stride = weights->stride;
  p.budget = budget;
  p.recent = recent;
  p.new_len = new_len;
  p.status = h->status;
  // Two CTAs fit an SM. More CTAs a (sequence, KV head) shorten the selection, but
  // each of its rounds then crosses the cluster, and a second wave of CTAs costs more
  // than it brings. Measured, 1 / 2 / 4 / 8 CTAs: 128 units of 8192 rows 51 / 43 / 69 /
  // 145 us, 32 units 28 / 21 / 20 / 29, 4 units 26 / 19 / 17 / 19; 128 units of
  // 2048 rows 17 / 23 / 41 / 101.
  p.cluster = 1;
  while (p.cluster < kEvictCluster &&
         ((long)p.cluster * kEvictSlice < rows ||
          (2L * p.cluster * p.B * p.Hkv <= 2L * h->num_sms && rows / (2 * p.cluster) >= 2048)))
    p.cluster *= 2;
  p.slice = (rows + p.cluster - 1) / p.cluster;
  return launch_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FASTOCR_OK
                                                                           : FASTOCR_ERR_CUDA;
}

fastocr_status fastocr_cross_attend(fastocr_handle* h, const void* q, const fastocr_kv* kv,
                                    const int32_t* q_start, int64_t rows, void* out, void* ws,
                                    int64_t ws_bytes, fastocr_stream stream) {
  if (!h || !q || !out || !q_start || !ws) return FASTOCR_ERR_NULL;
  fastocr_status st = check_kv(h, kv);
  if (st != FASTOCR_OK) return st;
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return FASTOCR_ERR_ALIGN;
  if (rows < 0 || rows * h->dims.num_q_heads >= (1LL << 31)) return FASTOCR_ERR_INVALID;
  RowsParams p = rows_params(h, q, kv);
  if (rows > 0 && ws_bytes < place_workspace(h, rows, false, static_cast<char*>(ws), p))
    return FASTOCR_ERR_INVALID;
  if (!units_fit(h, rows, h->dims.batch)) return FASTOCR_ERR_UNSUPPORTED;
  if ((st = check_device(h)) != FASTOCR_OK) return st;
  if (rows == 0) return FASTOCR_OK;
  if (cross_by_token(h, rows)) {
    Params a = base_params(h, q, kv, out);
    a.q_start = q_start;
    a.q_rows = (int)rows;
    return launch(h, kCross, expected_tokens(h), a, stream);
  }
  p.out = out;
  p.n_groups = h->dims.batch;
  p.start = q_start;
  p.rows = (int)rows;
  p.tile_tokens = choose_tile_tokens(h, rows, p.n_groups, expected_tokens(h));
  p.min_share = choose_share(h, rows, expected_tokens(h));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = launch_rows(h, p, s)) != FASTOCR_OK) return st;
  return launch_rows_merge(h->dims.head_dim, h->dims.dtype == FASTOCR_DTYPE_BF16, h->num_sms, p, s) == cudaSuccess
             ? FASTOCR_OK
             : FASTOCR_ERR_CUDA;
}

}  // extern "C"
