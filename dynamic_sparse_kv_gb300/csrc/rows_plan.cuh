// Plans of the row operators' calls: row tiles, shares and the form of a cross
// attention, from what the host knows (sizes and the expected length; offsets and
// lengths are on the device). Host code only.
#pragma once

#include "handle.cuh"
#include "rows.cuh"

namespace fastocr {

// Most rows of a row tile, in whole tokens.
inline int tile_rows(const fastocr_handle* h) {
  const int bm = h->dims.dtype == FASTOCR_DTYPE_BF16 ? kRowsBf16 : kRowsF32;
  const int g = h->dims.num_q_heads / h->dims.num_kv_heads;
  return bm / g * g;
}
inline int64_t slot_rows(const fastocr_handle* h, int64_t rows) {
  return std::min<int64_t>(tile_rows(h), rows * (h->dims.num_q_heads / h->dims.num_kv_heads));
}

// Tokens of a row tile. A bf16 tile of 256 rows reads each key once for all of
// them, one of 128 twice, but its parts are half as large: where the keys of
// few tiles are spread over all SMs, writing and joining the parts takes longer than
// reading the keys (4 key tiles an SM or fewer: 896 rows on 8320 keys 27 us with
// 256 rows, 22 us with 128). An fp32 tile of 64 rows reads shared memory less
// for a product; one of 16 is done sooner, where groups have few rows or all tiles
// of 16 still find an SM each (12 rows on 272 keys: 17.5 us and 13.6 us).
inline int choose_tile_tokens(const fastocr_handle* h, int64_t rows, int64_t groups, long keys) {
  const int64_t g = h->dims.num_q_heads / h->dims.num_kv_heads;
  auto units = [&](int bm) {   // about
    return std::max(groups, (rows * g + bm - 1) / bm) * h->dims.num_kv_heads * ((keys + kKeyTile - 1) / kKeyTile);
  };
  int bm;
  if (h->dims.dtype == FASTOCR_DTYPE_BF16)
    bm = units(kRowsBf16) <= 4 * h->num_sms ? kRowsBf16 / 2 : kRowsBf16;
  else
    bm = rows * g <= 16 * groups || units(16) <= h->num_sms ? 16 : kRowsF32;
  return bm / (int)g;
}

// Key tiles of a share, where few items are shared by all CTAs: a part of an item
// costs its rows' partials written and read (about 1 KB a row), a key tile of a
// share costs every CTA 1 to 2 us. The sum is least near sqrt(key tiles * rows /
// 1600): measured at 2, 6, 3 and 8 for 33 tiles and 224 rows (17.3 us), 65 and
// 896 (22.4 us), 16 and 896 (17.7 us), 65 and 1792 (30.3 us); within 1 us of
// the best share on nine shapes. fp32 tiles cost far more than their parts.
inline int choose_share(const fastocr_handle* h, int64_t rows, long keys) {
  if (h->dims.dtype != FASTOCR_DTYPE_BF16) return 1;
  const double tiles = (double)((keys + kKeyTile - 1) / kKeyTile);
  return (int)std::max(2.0, sqrt(tiles * (double)rows * h->dims.num_q_heads / 1600.0) + 0.5);
}

// The kernels count units of work in 32 bits.
inline bool units_fit(const fastocr_handle* h, int64_t rows, int64_t groups) {
  const int64_t g = h->dims.num_q_heads / h->dims.num_kv_heads;
  const int64_t least = (h->dims.dtype == FASTOCR_DTYPE_BF16 ? kRowsBf16 / 2 : 16) / g;   // tokens of a row tile
  const int64_t tiles = rows / least + std::min(rows, groups);
  return (double)tiles * h->dims.num_kv_heads * (max_tokens(h) / kKeyTile + 1) < 2147483647.0;
}

// Whether a cross attention goes to the split-K attend kernel, a query token a unit,
// instead of the row kernel: a decode step has one query token a sequence, or none,
// and the attend kernel's small tiles keep more of the states in flight (16 sequences,
// 10 heads, up to 2624 states: 32 us, row kernel and merge 46; two tokens in every
// other sequence 26 us and 32). Only the number of rows is known here, so all of them
// may be in one sequence, whose states a token a unit then reads again for each from
// L2 (14 TB/s), the row kernel once. So in bf16 the states of all tokens may come to
// 1 GB. Below it that worst case costs at most 75 us (128 tokens, 4 KV heads, 2624
// states: 54 us and 29; 64, 10, 2624: 71 and 16; 256, 10, 600: 95 and 23); above it
// the row kernel costs a decode step of as many sequences 4 to 20 % (64, 4, 8320
// states: 161 us and 178; 256, 4, 2624: 202 and 237; d = 64, 256, 2, 8320: 165 and
// 214), and one long prompt on a large handle gains (256, 4, 8320: 283 us and 45;
// 256, 10, 8320: 634 and 34). In fp32 the row kernel takes more than twice as long for
// a decode step (64, 4, 2624: 189 us and 395), so that always goes by token, although
// one prompt would gain where g is small (g = 1: 449 us and 82; g = 7: 183 and 198).
inline bool cross_by_token(const fastocr_handle* h, int64_t rows) {
  constexpr double kMost = 1e9;
  constexpr int64_t kGridZ = 65535;   // a token is a block in z
  if (rows > h->dims.batch || rows > kGridZ) return false;
  if (h->dims.dtype == FASTOCR_DTYPE_F32) return true;
  const double states = (double)expected_tokens(h) * h->dims.num_kv_heads * h->dims.head_dim * 2 * 2;   // K and V, bytes
  return (double)rows * states <= kMost;
}

}  // namespace fastocr
