// Attention of many query rows to one list of keys: a prefix that a group of
// decode sequences shares, or an encoder's states under a sequence's packed
// queries. All query tokens of group i attend to keys [0, len_i) of one block
// table row, without a mask.
//
// The work is a list of items -- (row tile, KV head) of every group, a row tile
// holding as many whole tokens (g rows each) as fit BM rows -- and an item's
// keys are a run of units. With many items a unit is a key tile, and the units of
// all items, in order, are dealt out in equal runs to one CTA per SM, whatever the
// groups' sizes: a CTA walks over segments of items, of which only the first and
// the last can be cut. With few items every CTA takes one unit, an equal share
// of one item: a second segment would cost it another start and
// output (5 us; 32 sequences on 8320 keys: 29 us dealt out, 22 us shared). A cut
// segment leaves (max, sum, unnormalised output) of its rows, in base 2, in one
// of the CTA's two slots of the workspace; who reads them (the tail's attend
// kernel, or merge_kernel) joins an item's parts in the order of their keys.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attend_kernels.cuh"

namespace fastocr {

constexpr int kKeyTile = 128;
constexpr int kRowsF32 = 64;     // BM per dtype
constexpr int kRowsBf16 = 256;   // or half of it, see tile_tokens

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
  int rows;                   // query tokens
  int tile_tokens;            // tokens of a row tile
  int min_share;              // least key tiles of a share, where CTAs take shares
  // workspace
  int slot_rows;              // rows a slot holds
  float* slot_acc;            // [CTAs, 2, slot_rows, d]
  float* slot_ml;             // [CTAs, 2, slot_rows, 2]: max, sum
  int4* token_part;           // shared: [rows, H_kv] where a token's parts are (see below)
  float* row_acc;             // shared: [rows, H_q, d], rows that one CTA has all keys of
  float* row_ml;              // shared: [rows, H_q, 2]
  int4* item_part;            // cross: [CTAs, 2] the cut item that starts in each CTA
  float scale_log2;
  int32_t* status;
};

// token_part: x = first CTA, y = parts, z = the first CTA's slot, w = row in the
// slot; with y == 1 the token's rows are in row_acc / row_ml.
// item_part: [0] x = first token, y = rows, z = KV head, w = parts (0: none);
// [1].x = the first CTA's slot.

// The keys of a group and where its tokens are.
struct RowGroup {
  int first, n_tok;   // query tokens
  int table_row;      // sequence whose block table holds the keys
  int len;            // keys
};

// Group i, offsets and lengths clamped into range; faults are ORed into bad, and
// `disordered` is set where the group ends before it starts.
__device__ __forceinline__ RowGroup load_group(const RowsParams& p, int i, int& bad, bool& disordered) {
  RowGroup r;
  int s = __ldcg(p.start + i), e = __ldcg(p.start + i + 1);
  disordered |= e < s;
  if (s < 0 || e < s || e > p.rows || (i == 0 && s != 0) ||
      (p.prefix_len && i == p.n_groups - 1 && e != p.rows))
    bad |= kDevBadGroup;
  s = min(max(s, 0), p.rows);
  e = min(max(e, s), p.rows);
  r.first = s;
  r.n_tok = e - s;
  r.table_row = p.prefix_len ? s : i;
  r.len = 0;
  if (r.n_tok > 0) {
    const int cap = p.max_pages << p.log2_page;
    int len = __ldcg((p.prefix_len ? p.prefix_len : p.seq_len) + r.table_row);
    int most = cap;
    if (p.prefix_len) most = min(max(__ldcg(p.seq_len + r.table_row), 0), cap);
    if (len < 0 || len > most) {
      bad |= p.prefix_len ? kDevBadGroup : kDevBadSeqLen;
      len = len < 0 ? 0 : most;
    }
    r.len = len;
  }
  return r;
}

// The sequences of a group must agree on their prefix; `n` threads, of which
// this is number `t`, check some each.
__device__ __forceinline__ void check_group(const RowsParams& p, const RowGroup& r, int t, int n, int& bad) {
  if (!p.prefix_len) return;
  for (int i = t; i < r.n_tok; i += n)
    if (__ldcg(p.prefix_len + r.first + i) != r.len) bad |= kDevBadGroup;
}

__device__ __forceinline__ int key_tiles(int len) { return (len + kKeyTile - 1) / kKeyTile; }

// Units of an item: its key tiles, or shares of about `share` of them (share > 0).
// An item without keys still has one unit, which writes its empty result.
__device__ __forceinline__ int units_of(int len, int share) {
  const int k = key_tiles(len);
  return max(1, share > 0 ? (k + share - 1) / share : k);
}

// A run of key tiles of one item.
struct Segment {
  RowGroup grp;
  int tok0, n_rows;     // the item's first token (of all) and rows
  int hkv;
  int k0, k1;           // key tiles
  bool whole;           // all of the item's keys
  bool starts;          // the item starts in this CTA
  int slot;             // where its part goes if it is cut
  int parts;            // starts: CTAs that share the item
};

// A CTA's walk over its segments. Units are counted in 32 bits: the host refuses
// a call whose groups could have 2^31 of them.
struct Walk {
  int unit, end;     // the CTA's units [unit, end)
  int begin, per;    // its first unit; units a CTA takes
  int group, off;    // group and unit within it
  int share;         // see units_of
  RowGroup grp;
};

// Row r of an item is token r / g, head r % g: the quotient for r < 256, g <= 8.
__device__ __forceinline__ int token_of_row(int r, int g_inv) { return (r * g_inv) >> 16; }
__device__ __forceinline__ int inverse_of(int g) { return (65535 + g) / g; }

// Items and units of a whole group.
__device__ __forceinline__ int group_items(const RowsParams& p, const RowGroup& r) {
  return (r.n_tok + p.tile_tokens - 1) / p.tile_tokens * p.Hkv;
}
__device__ __forceinline__ int group_units(const RowsParams& p, const RowGroup& r, int share) {
  return group_items(p, r) * units_of(r.len, share);
}

struct PlanSmem {
  int warp_sum[2][32], warp_items[32], warp_max[32];
  int group, off;
  RowGroup grp;
};

// Units a CTA takes and the share of an item, from the totals over all groups.
__device__ __forceinline__ void choose_share(const RowsParams& p, int all, int items, int most, Walk& w) {
  // an item's parts fit the merging kernels' lists
  const int C = gridDim.x, least = max(1, (most + kMaxExt - 3) / (kMaxExt - 2));
  w.share = 0;
  if (2 * items <= C) {   // the shares are at most all / share + items <= C
    w.share = max(max(p.min_share, least), (all + C - items - 1) / (C - items));
    w.per = 1;
  } else {
    w.per = max(least, (all + C - 1) / C);
  }
}

// The CTA's run of `all` units; false: it has none.
__device__ __forceinline__ bool take_units(int all, Walk& w) {
  const long long first = (long long)blockIdx.x * w.per;
  w.begin = w.unit = (int)min((long long)all, first);
  w.end = (int)min((long long)all, first + w.per);
  return first < all;
}

// Where this CTA's units are; called by all THREADS threads. False: it has none.
// Offsets out of order leave all CTAs without work: groups would share rows, and
// their units could be more than 32 bits count.
// faulty: the offsets or lengths are, so some tokens may be in no group.
// Up to 32 groups every warp works it out for itself, without a barrier (every
// call starts with this: 2 us through barriers, about 1 us without).
template <int THREADS>
__device__ __forceinline__ bool plan_walk(const RowsParams& p, PlanSmem& s, Walk& w, bool& faulty, int& bad) {
  constexpr int NW = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto warp_prefix = [&](int x) {
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    return incl;
  };
  RowGroup grp = {0, 0, 0, 0};
  bool disordered = false;
  faulty = false;
  if (p.n_groups <= 32) {
    int sum = 0, items = 0, most = 0;
    if (lane < p.n_groups) {
      grp = load_group(p, lane, bad, disordered);
      sum = group_units(p, grp, 0);
      items = group_items(p, grp);
      most = grp.n_tok > 0 ? key_tiles(grp.len) : 0;
    }
    faulty = __any_sync(0xffffffffu, bad & kDevBadGroup);
    if (faulty && __any_sync(0xffffffffu, disordered)) return false;
    choose_share(p, __reduce_add_sync(0xffffffffu, sum), __reduce_add_sync(0xffffffffu, items),
                 __reduce_max_sync(0xffffffffu, most), w);
    if (w.share > 0) sum = group_units(p, grp, w.share);   // 0 for a lane without a group
    const int incl = warp_prefix(sum);
    if (!take_units(__shfl_sync(0xffffffffu, incl, 31), w)) return false;
    const int src = __ffs(__ballot_sync(0xffffffffu, incl > w.unit)) - 1;
    w.group = src;
    w.off = w.unit - __shfl_sync(0xffffffffu, incl - sum, src);
    w.grp.first = __shfl_sync(0xffffffffu, grp.first, src);
    w.grp.n_tok = __shfl_sync(0xffffffffu, grp.n_tok, src);
    w.grp.table_row = __shfl_sync(0xffffffffu, grp.table_row, src);
    w.grp.len = __shfl_sync(0xffffffffu, grp.len, src);
    return true;
  }
  const int chunk = (p.n_groups + THREADS - 1) / THREADS;   // consecutive groups a thread sums
  const int i0 = min(p.n_groups, tid * chunk), i1 = min(p.n_groups, i0 + chunk);
  int sum = 0, items = 0, most = 0;
  for (int i = i0; i < i1; ++i) {
    grp = load_group(p, i, bad, disordered);
    sum += group_units(p, grp, 0);
    items += group_items(p, grp);
    most = max(most, grp.n_tok > 0 ? key_tiles(grp.len) : 0);
  }
  faulty = __syncthreads_or(bad & kDevBadGroup);
  if (faulty && __syncthreads_or(disordered)) return false;
  // units before this thread, and of all
  int mine, all;
  auto scan = [&](int x, int* warp_sum) {
    const int incl = warp_prefix(x);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const int c = warp_sum[v];
      if (v < warp) before += c;
      all += c;
    }
    mine = before + incl - x;
  };
  items = __reduce_add_sync(0xffffffffu, items);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    s.warp_items[warp] = items;
    s.warp_max[warp] = most;
  }
  scan(sum, s.warp_sum[0]);
  items = 0;
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    items += s.warp_items[v];
    most = max(most, s.warp_max[v]);
  }
  choose_share(p, all, items, most, w);
  if (w.share > 0) {
    sum = 0;
    for (int i = i0; i < i1; ++i) {
      if (chunk > 1) grp = load_group(p, i, bad, disordered);
      sum += group_units(p, grp, w.share);
    }
    scan(sum, s.warp_sum[1]);
  }
  if (!take_units(all, w)) return false;
  if (mine <= w.unit && w.unit < mine + sum) {
    int at = mine, i = i0;
    if (chunk > 1) {   // which of this thread's groups
      for (;; ++i) {
        grp = load_group(p, i, bad, disordered);
        const int u = group_units(p, grp, w.share);
        if (w.unit < at + u) break;
        at += u;
      }
    }
    s.group = i;
    s.off = w.unit - at;
    s.grp = grp;
  }
  __syncthreads();
  w.group = s.group;
  w.off = s.off;
  w.grp = s.grp;
  return true;
}

// The next segment; false at the end. Warp-uniform.
__device__ __forceinline__ bool next_segment(const RowsParams& p, Walk& w, Segment& s) {
  if (w.unit >= w.end) return false;
  const int tpt = p.tile_tokens;
  while (w.off >= group_units(p, w.grp, w.share)) {   // another group with rows exists: w.unit < w.end
    int none = 0;                                // reported by plan_walk
    bool disordered = false;
    w.grp = load_group(p, ++w.group, none, disordered);
    w.off = 0;
  }
  const int u = units_of(w.grp.len, w.share), n_tiles = key_tiles(w.grp.len);
  const int item = w.off / u, k = w.off - item * u;   // item in the group, unit in the item
  const int tile = item / p.Hkv;
  const int n = min(u - k, w.end - w.unit);
  s.hkv = item - tile * p.Hkv;
  s.grp = w.grp;
  s.tok0 = w.grp.first + tile * tpt;
  s.n_rows = min(tpt, w.grp.n_tok - tile * tpt) * p.g;
  s.k0 = (int)((long long)k * n_tiles / u);
  s.k1 = (int)((long long)(k + n) * n_tiles / u);
  s.whole = n == u;
  s.starts = k == 0;
  s.slot = w.unit == w.begin ? 0 : 1;
  s.parts = (w.unit + u - 1) / w.per - (int)blockIdx.x + 1;   // of an item that starts here
  w.unit += n;
  w.off += n;
  return true;
}

// Tells the tail's attend kernel where the parts of a shared prefix's item that
// starts here are; `n` threads, of which this is number `t`.
__device__ __forceinline__ void publish_parts(const RowsParams& p, const Segment& s, int t, int n) {
  if (!p.token_part || !s.starts) return;
  for (int i = t; i < s.n_rows / p.g; i += n)
    p.token_part[(size_t)(s.tok0 + i) * p.Hkv + s.hkv] = make_int4(blockIdx.x, s.parts, s.slot, i * p.g);
}

// A token that no group has gets no parts, so that the tail's attend kernel does not
// join what an earlier call left there. For `n` threads of CTA 0, of which this is
// number `t`, after its wait: the kernel before may read the workspace. Without any
// work in CTA 0 (no_work) no token is in a group, else those from the first offset to
// the last are.
__device__ __forceinline__ void publish_none(const RowsParams& p, bool no_work, int t, int n) {
  if (!p.token_part || blockIdx.x != 0) return;
  int s = p.rows, e = p.rows;
  if (!no_work) {
    s = min(max(__ldcg(p.start), 0), p.rows);
    e = min(max(__ldcg(p.start + p.n_groups), s), p.rows);
  }
  s *= p.Hkv;
  e *= p.Hkv;
  for (int i = t; i < s + p.rows * p.Hkv - e; i += n) p.token_part[i < s ? i : i - s + e] = make_int4(0, 0, 0, 0);
}

// Tells merge_kernel the cut item that starts in this CTA (cross attention):
// only its last segment can be one.
__device__ __forceinline__ void publish_cut(const RowsParams& p, const Segment& s) {
  p.item_part[2 * blockIdx.x] = make_int4(s.tok0, s.n_rows, s.hkv, s.parts);
  p.item_part[2 * blockIdx.x + 1] = make_int4(s.slot, 0, 0, 0);
}
__device__ __forceinline__ void publish_no_cut(const RowsParams& p) {
  p.item_part[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
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

// One CTA an SM.
cudaError_t launch_rows_f32(int head_dim, int ctas, const RowsParams& p, cudaStream_t s);
cudaError_t launch_rows_bf16(int head_dim, int ctas, const RowsParams& p, cudaStream_t s);
cudaError_t launch_rows_merge(int head_dim, bool bf16, int ctas, const RowsParams& p, cudaStream_t s);
cudaError_t prepare_rows_f32();
cudaError_t prepare_rows_bf16();

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
