// Eviction by accumulated attention weight.
//
// Of the n = N_t - protect rows of a sequence and KV head, `keep` = min(n,
// budget) stay: the recent ones (position >= seen - recent), then those of
// largest weight, ties to the lower row. Attention does not depend on the
// order of its rows, so the kept rows at or behind `keep` (survivors) move
// into the rows before it that go (holes), i-th to i-th: every moved row is
// read and written once and no kept row before `keep` moves at all.
//
// One cluster of CTAs has a (sequence, KV head). A CTA keeps the 32-bit sort
// keys of its slice of rows in shared memory; a radix select by 11, 11 and 10 bits
// finds the keep-th largest key (weights share few exponents), the CTAs
// joining their histograms through distributed shared memory; each CTA then lists
// its holes and survivors, and the moves are dealt out evenly over the cluster
// by rank, whoever listed them.
//
// Measured: 128 units of 8192 rows cut to 1024 (58 MB read and 58 MB written in rows
// of 256 bytes) 41 us, of which the moves take 21 us at 5.3 TB/s and the selection
// about 10; one row of 513 in 32 units 7 us, the latency of its rounds.
#include "evict.cuh"

#include "attend_kernels.cuh"

namespace fastocr {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 2;        // histogram copies, against equal digits of neighbouring warps
constexpr int kBins = 2048;    // four a thread
static_assert(kBins == 4 * kThreads, "a thread's bins");
constexpr int kMoveBatch = 4;  // row copies a warp has in flight

struct EvictSmem {
  int hist[kSub][kBins];    // a pass's digits of this CTA's rows, bins in descending order
  int total[2][kBins];      // their sums, read by the cluster; passes take turns
  int counts[4];            // equal keys, holes, survivors of this CTA, read by the cluster
  int warp_sum[kWarps];
  int pick[4];              // digit, rows above it, rows in it
  int hole_base[kEvictCluster + 1], stay_base[kEvictCluster + 1];
};

__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int ld_peer(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int4 ld_peer4(uint32_t a) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ int ld_peer_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared::cluster.u16 %0, [%1];\n" : "=h"(v) : "r"(a) : "memory");
  return v;
}

// Unsigned order = order of the weights; a NaN goes first.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Counts digit d (of a warp's active lanes; -1: none). Equal digits of a whole warp,
// e.g. of rows that have no weight yet, count as one.
__device__ __forceinline__ void count_digit(int* hist, int d) {
  const int first = __shfl_sync(0xffffffffu, d, 0);
  if (__all_sync(0xffffffffu, d == first)) {
    if ((threadIdx.x & 31) == 0 && d >= 0) atomicAdd(hist + (kBins - 1 - d), 32);
  } else if (d >= 0) {
    atomicAdd(hist + (kBins - 1 - d), 1);
  }
}

// Exclusive prefix of x over the block's threads, and the block's sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // warp_sum of the scan before is read to the end
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int c = warp_sum[w];
    if (w < warp) before += c;
    all += c;
  }
  sum = all;
  return before + incl - x;
}

__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ EvictSmem s;
  uint32_t* keys = reinterpret_cast<uint32_t*>(dyn);                        // [slice]
  uint16_t* list = reinterpret_cast<uint16_t*>(dyn + (size_t)p.slice * 4);  // [slice]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.cluster, rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const size_t unit = (size_t)b * p.Hkv + h;
  auto cluster_barrier = [&]() {
    if (S > 1) cluster_sync();
    else __syncthreads();
  };

  // lengths are final before the kernel preceding this one; weights are not
  int bad = 0;
  const int cap = p.max_pages << p.log2_page;
  int n_t = __ldcg(p.seq_len + b), protect = __ldcg(p.protect + b);
  const int edge = __ldcg(p.seen + b) - p.recent;
  if (n_t < 0 || n_t > cap) {
    bad |= kDevBadSeqLen;
    n_t = n_t < 0 ? 0 : cap;
  }
  if (protect < 0) {
    bad |= kDevBadWeights;
    protect = 0;
  }
  const int n = max(0, n_t - protect);
  int keep = min(n, p.budget);
  if (n > p.stride) {   // rows without weights: leave the sequence as it is
    bad |= kDevBadWeights;
    keep = n;
  }
  for (int i = tid; i < kSub * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;

  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (rank == 0 && h == 0 && tid == 0 && p.new_len) p.new_len[b] = min(n_t, protect) + keep;
  if (bad && tid == 0) atomicOr(p.status, bad);
  if (n <= keep) return;   // the same for the whole cluster

  const int per = (n + S - 1) / S;   // <= slice, from the host
  const int lo = min(n, rank * per), mine = min(n, lo + per) - lo;
  const float* mass = p.mass + unit * p.stride;
  const int32_t* pos = p.pos + unit * p.stride;
  __syncthreads();
  constexpr int kKeyBatch = 8;   // rows a thread has in flight (one after the other: 1 us each)
  int* my_hist = s.hist[warp % kSub];
  for (int i0 = tid; i0 - lane < mine; i0 += kKeyBatch * kThreads) {
    int at[kKeyBatch];
    float w[kKeyBatch];
#pragma unroll
    for (int u = 0; u < kKeyBatch; ++u) {
      const int i = i0 + u * kThreads;
      at[u] = i < mine ? __ldcg(pos + lo + i) : 0;
      w[u] = i < mine ? __ldcg(mass + lo + i) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kKeyBatch; ++u) {
      const int i = i0 + u * kThreads;
      const uint32_t key = at[u] >= edge ? 0xffffffffu : weight_key(w[u]);
      if (i < mine) keys[i] = key;
      if (i - lane < mine) count_digit(my_hist, i < mine ? (int)(key >> 21) : -1);
    }
  }
  // --- the keep-th largest key
  uint32_t prefix = 0, mask = 0;
  int krem = keep;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 0x3ffu : 0x7ffu;
    if (pass > 0) {
      for (int i = tid; i - lane < mine; i += kThreads) {
        const uint32_t key = i < mine ? keys[i] : 0u;
        const bool in = i < mine && (key & mask) == prefix;
        if (__any_sync(0xffffffffu, in)) count_digit(my_hist, in ? (int)((key >> shift) & digits) : -1);
      }
    }
    __syncthreads();
    int4 c = *reinterpret_cast<const int4*>(&s.hist[0][4 * tid]);
#pragma unroll
    for (int q = 1; q < kSub; ++q) {
      const int4 x = *reinterpret_cast<const int4*>(&s.hist[q][4 * tid]);
      c = make_int4(c.x + x.x, c.y + x.y, c.z + x.z, c.w + x.w);
    }
#pragma unroll
    for (int q = 0; q < kSub; ++q) *reinterpret_cast<int4*>(&s.hist[q][4 * tid]) = make_int4(0, 0, 0, 0);
    if (S > 1) {
      *reinterpret_cast<int4*>(&s.total[pass & 1][4 * tid]) = c;
      cluster_sync();
      int4 v[kEvictCluster];
#pragma unroll
      for (int r = 0; r < kEvictCluster; ++r)
        v[r] = r < S ? ld_peer4(peer(&s.total[pass & 1][4 * tid], r)) : make_int4(0, 0, 0, 0);
      c = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kEvictCluster; ++r)
        c = make_int4(c.x + v[r].x, c.y + v[r].y, c.z + v[r].z, c.w + v[r].w);
    }
    int all;
    const int above = block_scan(c.x + c.y + c.z + c.w, s.warp_sum, all);   // bins in descending order
    const int bin[4] = {c.x, c.y, c.z, c.w};
    int run = above;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (run < krem && krem <= run + bin[j]) {
        s.pick[0] = kBins - 1 - (4 * tid + j);
        s.pick[1] = run;
        s.pick[2] = bin[j];
      }
      run += bin[j];
    }
    __syncthreads();
    prefix |= (uint32_t)s.pick[0] << shift;
    mask |= digits << shift;
    krem -= s.pick[1];
    if (krem == s.pick[2]) break;   // every key with this prefix stays: the same in every CTA
    __syncthreads();
  }

  // --- who stays: a key above the prefix, or one of the first krem equal ones
  const int chunk = (mine + kThreads - 1) / kThreads | 1;   // a thread's consecutive rows; odd: no bank conflicts
  const int c0 = min(mine, tid * chunk), c1 = min(mine, c0 + chunk);
  int eq_run = 0;   // equal keys of the rows before this thread's; not needed where all of them stay
  if (krem != s.pick[2]) {
    int eq = 0, eq_all;
    for (int i = c0; i < c1; ++i) eq += (keys[i] & mask) == prefix;
    eq_run = block_scan(eq, s.warp_sum, eq_all);
    if (S > 1) {
      if (tid == 0) s.counts[0] = eq_all;
      cluster_sync();
      int v[kEvictCluster];
#pragma unroll
      for (int r = 0; r < kEvictCluster; ++r) v[r] = r < rank ? ld_peer(peer(&s.counts[0], r)) : 0;
#pragma unroll
      for (int r = 0; r < kEvictCluster; ++r) eq_run += v[r];
    }
  } else {
    krem = 0x7fffffff;
  }
  const int cut = min(max(keep - lo, 0), mine);   // rows of the slice before `keep`
  int holes = 0, stays = 0, e = eq_run;
  for (int i = c0; i < c1; ++i) {
    const uint32_t key = keys[i] & mask;
    const bool stay = key > prefix || (key == prefix && e++ < krem);
    holes += !stay && i < cut;
    stays += stay && i >= cut;
  }
  // both in one scan: a slice has at most 2^15 of either
  int both_all;
  const uint32_t before = (uint32_t)block_scan((int)((uint32_t)holes << 16 | (uint32_t)stays), s.warp_sum, both_all);
  const int holes_all = (int)((uint32_t)both_all >> 16), stays_all = both_all & 0xffff;
  int hole_at = (int)(before >> 16), stay_at = (int)(before & 0xffffu);
  e = eq_run;
  for (int i = c0; i < c1; ++i) {   // holes fill the list from its start, survivors behind them
    const uint32_t key = keys[i] & mask;
    const bool stay = key > prefix || (key == prefix && e++ < krem);
    if (!stay && i < cut) list[hole_at++] = (uint16_t)i;
    if (stay && i >= cut) list[holes_all + stay_at++] = (uint16_t)i;
  }
  if (tid == 0) {
    s.counts[1] = holes_all;
    s.counts[2] = stays_all;
  }
  cluster_barrier();
  if (warp == 0) {   // lane r: the lists of CTA r
    int x = 0, y = 0;
    if (lane < S) {
      x = S > 1 ? ld_peer(peer(&s.counts[1], lane)) : holes_all;
      y = S > 1 ? ld_peer(peer(&s.counts[2], lane)) : stays_all;
    }
    int xs = x, ys = y;
#pragma unroll
    for (int o = 1; o < kEvictCluster; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, xs, o), b2 = __shfl_up_sync(0xffffffffu, ys, o);
      if (lane >= o) {
        xs += a;
        ys += b2;
      }
    }
    if (lane < S) {
      s.hole_base[lane + 1] = xs;
      s.stay_base[lane + 1] = ys;
    }
    if (lane == 0) s.hole_base[0] = s.stay_base[0] = 0;
  }
  __syncthreads();
  const int moves = min(s.hole_base[S], s.stay_base[S]);   // equal
  const int m0 = (int)((long)moves * rank / S), m1 = (int)((long)moves * (rank + 1) / S);
  const int32_t* table = p.block_table + (size_t)b * p.max_pages;
  // row (from `protect`) of entry `at` of the concatenated lists
  auto listed = [&](const int* base, int at, bool survivor) -> int {
    int r = 0;
    while (r + 1 < S && at >= base[r + 1]) ++r;
    int off = at - base[r];
    if (survivor) off += s.hole_base[r + 1] - s.hole_base[r];
    const int i = S > 1 ? ld_peer_u16(peer(list + off, r)) : list[off];
    return r * per + i;
  };
  // 32 moves a warp at a time: each lane looks one up and moves its weight and
  // position; then the warp copies the rows, 16 bytes a lane, K and V together
  const int lanes_row = p.row_bytes / 16;           // 8 .. 32 lanes a row
  const int lane_row = lane / lanes_row, lane_col = (lane % lanes_row) * 16;
  const int at_once = 32 / lanes_row;               // rows one instruction covers
  for (int r0 = m0 + warp * 32; r0 < m1; r0 += kWarps * 32) {
    const int cnt = min(32, m1 - r0);
    long src = -1, dst = -1;
    if (lane < cnt) {
      const int from = listed(s.stay_base, r0 + lane, true), to = listed(s.hole_base, r0 + lane, false);
      const int rf = protect + from, rt = protect + to;
      const int pf = __ldcg(table + (rf >> p.log2_page)), pt = __ldcg(table + (rt >> p.log2_page));
      const int sm = (1 << p.log2_page) - 1;
      if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) {
        bad |= kDevBadPage;
      } else {
        src = ((((long)pf * p.Hkv + h) << p.log2_page) | (rf & sm)) * p.row_bytes;
        dst = ((((long)pt * p.Hkv + h) << p.log2_page) | (rt & sm)) * p.row_bytes;
      }
      p.mass[unit * p.stride + to] = __ldcg(mass + from);
      p.pos[unit * p.stride + to] = __ldcg(pos + from);
    }
    for (int i0 = 0; i0 < cnt; i0 += kMoveBatch * at_once) {
      uint4 kx[kMoveBatch], vx[kMoveBatch];
      long to[kMoveBatch];
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u) {
        const int i = i0 + u * at_once + lane_row;
        const long from = __shfl_sync(0xffffffffu, src, i & 31);
        to[u] = __shfl_sync(0xffffffffu, dst, i & 31);
        if (i >= cnt) to[u] = -1;
        if (to[u] >= 0) {
          kx[u] = __ldcg(reinterpret_cast<const uint4*>(p.k + from + lane_col));
          vx[u] = __ldcg(reinterpret_cast<const uint4*>(p.v + from + lane_col));
        }
      }
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u) {
        if (to[u] >= 0) {
          *reinterpret_cast<uint4*>(p.k + to[u] + lane_col) = kx[u];
          *reinterpret_cast<uint4*>(p.v + to[u] + lane_col) = vx[u];
        }
      }
    }
  }
  if (bad & kDevBadPage) atomicOr(p.status, kDevBadPage);
  if (S > 1) cluster_sync();   // the lists are read by the whole cluster
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(p.cluster, p.Hkv, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.slice * 6;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel, p);
}

cudaError_t prepare_evict() {
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kEvictSlice * 6);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

}  // namespace fastocr
