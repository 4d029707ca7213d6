// Attention of many query rows to one list of keys: a prefix that a group of
// decode sequences shares, or an encoder's states under a sequence's packed
// queries. Row r of group i and KV head j is query token start[i] + r / g, head
// j*g + r % g; all rows of the group attend to keys [0, len_i) of one block
// table row, without a mask. The keys are cut into `splits` parts; every part
// leaves (max, sum, unnormalised output) of each row, in base 2, in the
// caller's workspace, or the output itself where one part has all keys.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attend_kernels.cuh"

namespace fastocr {

constexpr int kKeyTile = 128;   // keys a split's share is counted in

struct RowsParams {
  const void* q;              // [rows, H_q, d]
  void* out;                  // [rows, H_q, d]; NULL: partials only
  const void* k;
  const void* v;
  const int32_t* block_table;
  const int32_t* seq_len;     // [B]
  int num_pages, max_pages, log2_page;
  int Hq, Hkv, g;
  int n_groups;
  const int32_t* start;       // [n_groups + 1]
  const int32_t* prefix_len;  // shared prefix: [B]; NULL: group i reads all of sequence i
  long rows;                  // query tokens
  int splits;
  float* ml;                  // [splits, rows * H_q, 2]
  float* acc;                 // [splits, rows * H_q, d]
  float scale_log2;
  int32_t* status;
};

// One group as a CTA sees it.
struct RowGroup {
  int first;       // its first query token
  int n_rows;      // (tokens of the group) * g
  int table_row;   // sequence whose block table holds the keys
  int len;         // keys
  int tile;        // this CTA's row tile in the group; -1: no tile left
};

// Finds row tile `tile` (BM rows each, groups in order) by scanning the groups
// 32 at a time; called by one whole warp, every lane gets the result. Lengths
// and offsets out of range are clamped; faults are ORed into bad.
template <int BM>
__device__ __forceinline__ RowGroup find_tile(const RowsParams& p, int tile, int& bad) {
  const int lane = threadIdx.x & 31;
  RowGroup r;
  r.tile = -1;
  r.first = r.n_rows = r.table_row = r.len = 0;
  const int rows = (int)p.rows;
  int base = 0;   // tiles of the groups before this round's
  for (int i0 = 0; i0 < p.n_groups; i0 += 32) {
    const int i = i0 + lane;
    int s = 0, e = 0;
    if (i < p.n_groups) {
      s = __ldcg(p.start + i);
      e = __ldcg(p.start + i + 1);
      if (s < 0 || e < s || e > rows || (i == 0 && s != 0) ||
          (p.prefix_len && i == p.n_groups - 1 && e != rows))
        bad |= kDevBadGroup;
      s = min(max(s, 0), rows);
      e = min(max(e, s), rows);
    }
    const int tiles = ((e - s) * p.g + BM - 1) / BM;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > tile);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.tile = tile - base - __shfl_sync(0xffffffffu, incl - tiles, src);
      r.first = __shfl_sync(0xffffffffu, s, src);
      r.n_rows = (__shfl_sync(0xffffffffu, e, src) - r.first) * p.g;
      const int group = i0 + src;
      const int cap = p.max_pages << p.log2_page;
      r.table_row = p.prefix_len ? r.first : group;
      int len = __ldcg((p.prefix_len ? p.prefix_len : p.seq_len) + r.table_row);
      int most = cap;
      if (p.prefix_len) most = min(max(__ldcg(p.seq_len + r.table_row), 0), cap);
      if (len < 0 || len > most) {
        bad |= p.prefix_len ? kDevBadGroup : kDevBadSeqLen;
        len = len < 0 ? 0 : most;
      }
      r.len = len;
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// The sequences of a group must agree on their prefix; every thread of the CTA
// checks some.
__device__ __forceinline__ void check_group(const RowsParams& p, const RowGroup& r, int& bad) {
  if (!p.prefix_len) return;
  for (int i = threadIdx.x; i < r.n_rows / p.g; i += blockDim.x)
    if (__ldcg(p.prefix_len + r.first + i) != r.len) bad |= kDevBadGroup;
}

// Keys [lo, hi) of part `split`.
__device__ __forceinline__ void split_range(int len, int splits, int split, int& lo, int& hi) {
  const int tiles = (len + kKeyTile - 1) / kKeyTile;
  const int per = (tiles + splits - 1) / splits;
  lo = min(len, split * per * kKeyTile);
  hi = min(len, lo + per * kKeyTile);
}

// Cache row (page * H_kv + head) * page_size + slot of key `pos`, -1 where its
// page is out of range.
__device__ __forceinline__ int key_row(const RowsParams& p, const int32_t* table, int hkv, int pos,
                                       int& bad) {
  const int page = __ldcg(table + (pos >> p.log2_page));
  if (page < 0 || page >= p.num_pages) {
    bad |= kDevBadPage;
    return -1;
  }
  return ((page * p.Hkv + hkv) << p.log2_page) | (pos & ((1 << p.log2_page) - 1));
}

// Rows a CTA's tile holds, per dtype.
constexpr int kRowsF32 = 64;
constexpr int kRowsBf16 = 256;

cudaError_t launch_rows_f32(int head_dim, const RowsParams& p, cudaStream_t s);
cudaError_t launch_rows_bf16(int head_dim, const RowsParams& p, cudaStream_t s);
cudaError_t launch_rows_merge(int head_dim, bool bf16, const RowsParams& p, cudaStream_t s);
cudaError_t prepare_rows_f32();
cudaError_t prepare_rows_bf16();

// Row tiles a launch must cover, whatever the groups' sizes.
inline long max_row_tiles(const RowsParams& p, int bm) {
  return p.rows * p.g / bm + std::min<long>(p.n_groups, p.rows);
}

inline cudaError_t launch_pdl(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t s,
                              void** args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace fastocr
