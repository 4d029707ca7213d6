// The handle of libfastocr.so and the host helpers its entry points share:
// argument checks, split-K sizing and the launch of an attend kernel.
#pragma once

#include <math.h>
#include <string.h>

#include <algorithm>

#include "attend_kernels.cuh"
#include "fastocr.h"

namespace fastocr {
cudaError_t launch_bf16(int head_dim, int mode, const Params& p, cudaStream_t s);
cudaError_t launch_f32(int head_dim, int mode, const Params& p, cudaStream_t s);
cudaError_t launch_select(const Params& p, cudaStream_t s);
cudaError_t prepare_bf16();
cudaError_t prepare_f32();
int max_cluster_bf16(int head_dim, int variant);
int max_cluster_f32(int head_dim, int variant);
int active_clusters_bf16(int head_dim, int cluster);
int active_clusters_f32(int head_dim, int cluster);
}  // namespace fastocr

struct fastocr_handle {
  fastocr_dims dims;
  int device;
  int num_sms;
  int log2_page;
  int split_override[3];
  int variant_override[3];      // 0: automatic, else Variant + 1
  int max_splits;   // largest thread-block cluster the device co-schedules (<= 16)
  int max_splits_v[fastocr::kNumVariants];   // same per variant (0: the variant does not exist)
  int active[fastocr::kMaxSplits + 1];   // clusters of each size the device holds at once
  long len_hint;    // caller's N_t of the coming calls (0: unknown), split choice only
  void* ws;
  size_t ws_bytes;
  float* logits;
  float* sigma_part;
  double* profile;
  int32_t* status;
};

namespace fastocr {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int ilog2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return (1 << l) == x ? l : -1;
}

inline int slot_of(int mode) { return mode == kSparse ? 1 : (mode == kRswa ? 2 : 0); }

// Kernel variant and split count of a launch whose attend lists hold about
// `len` entries per (sequence, KV head) unit -- (query token, KV head) in cross
// mode, which has p.q_rows of them; caller overrides win.
inline void plan_launch(const fastocr_handle* h, int mode, long len, Params& p) {
  const int slot = slot_of(mode);
  const long units = (long)(mode == kCross ? p.q_rows : h->dims.batch) * h->dims.num_kv_heads;
  if (len < 1) len = 1;
  int v = h->variant_override[slot] - 1;   // -1: automatic
  int s = h->split_override[slot];         // 0: automatic
  if (s == 0) s = choose_splits(units, len, h->max_splits, h->active, h->num_sms);
  // grids that leave room for the next kernel's CTAs at one CTA per SM take
  // the deeper pipeline (more of each CTA's tiles staged before the wait)
  if (v < 0)
    v = (2L * s * units <= h->num_sms && s <= h->max_splits_v[kDeep]) ? kDeep : kGeneral;
  p.variant = v;
  p.splits = std::max(1, std::min(s, h->max_splits_v[v]));
  // small grids release the next kernel right away (its CTAs then prefetch
  // while this one runs); grids that need the whole GPU release it only
  // after their main loop, so its CTAs do not take slots from this grid
  p.pdl_early = (long)p.splits * units <= h->num_sms;
}

inline long max_tokens(const fastocr_handle* h) {
  return (long)h->dims.max_pages_per_seq << h->log2_page;
}

// cache length the split choice assumes: the caller's hint, else the capacity
inline long expected_tokens(const fastocr_handle* h) {
  return h->len_hint > 0 ? std::min(h->len_hint, max_tokens(h)) : max_tokens(h);
}

inline fastocr_status check_kv(const fastocr_handle* h, const fastocr_kv* kv) {
  if (!kv || !kv->k || !kv->v || !kv->block_table || !kv->seq_len) return FASTOCR_ERR_NULL;
  if (kv->num_pages < 1) return FASTOCR_ERR_INVALID;
  if (!aligned16(kv->k) || !aligned16(kv->v)) return FASTOCR_ERR_ALIGN;
  // cache rows are indexed with 32-bit integers inside the kernels
  if ((long long)kv->num_pages * h->dims.num_kv_heads * h->dims.page_size >= (1LL << 31))
    return FASTOCR_ERR_UNSUPPORTED;
  return FASTOCR_OK;
}

inline Params base_params(const fastocr_handle* h, const void* q, const fastocr_kv* kv, void* out) {
  Params p;
  memset(&p, 0, sizeof(p));
  const fastocr_dims& d = h->dims;
  p.q = q;
  p.out = out;
  p.k = kv->k;
  p.v = kv->v;
  p.block_table = kv->block_table;
  p.seq_len = kv->seq_len;
  p.num_pages = kv->num_pages;
  p.max_pages = d.max_pages_per_seq;
  p.log2_page = h->log2_page;
  p.B = d.batch;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.g = d.num_q_heads / d.num_kv_heads;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d.head_dim));
  p.logits = h->logits;
  p.sigma_part = h->sigma_part;
  p.sel_src = h->sigma_part;   // the selection sums the KV heads' score shares
  p.sel_heads = d.num_kv_heads;
  p.sel_head_stride = d.max_img_tokens;
  p.sel_batch_stride = (long)d.num_kv_heads * d.max_img_tokens;
  p.profile = h->profile;
  p.profile_layer = -1;
  p.status = h->status;
  p.max_img = d.max_img_tokens;
  return p;
}

inline fastocr_status launch(const fastocr_handle* h, int mode, long len, Params p,
                      fastocr_stream stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  plan_launch(h, mode, len, p);
  cudaError_t e = h->dims.dtype == FASTOCR_DTYPE_BF16 ? launch_bf16(h->dims.head_dim, mode, p, s)
                                                       : launch_f32(h->dims.head_dim, mode, p, s);
  return e == cudaSuccess ? FASTOCR_OK : FASTOCR_ERR_CUDA;
}

}  // namespace fastocr
