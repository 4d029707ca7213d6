// Row attention on the CUDA cores (fp32, no TF32), and the kernel that joins
// the parts of cut items.
//
// A CTA of 256 threads holds 16 R query rows and streams its keys in tiles of
// 64 through shared memory, the next tile's rows in registers meanwhile: thread
// (ty, tx) computes rows R ty.. and keys tx + 16j of the scores, and output dims
// of the same rows; softmax is online, in base 2, with the row statistics of
// 16 neighbouring lanes joined by shuffles. R = 4 reads a shared-memory value for
// eight products; R = 1 for few rows, where a tile's latency counts.
#include <algorithm>

#include <math_constants.h>

#include "rows.cuh"

namespace fastocr {

namespace {

constexpr int kThreads = 256;
constexpr int BN = 64;

template <int D, int R>
struct SmemF32 {
  static constexpr int BM = 16 * R;
  static constexpr int LD = D + 4;      // K rows: 16 keys apart in a warp, no bank conflicts
  static constexpr int kQ = 0;          // [BM][D]
  static constexpr int kK = kQ + BM * D;
  static constexpr int kV = kK + BN * LD;
  static constexpr int kP = kV + BN * D;     // [BM][BN]
  static constexpr int kRow = kP + BM * BN;  // int [2][BN]: cache rows of a tile's keys, -1: none
  static constexpr int kBytes = (kRow + 2 * BN) * 4;
};

__device__ __forceinline__ float4 load4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const RowsParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ PlanSmem plan;
  using S = SmemF32<D, R>;
  constexpr int LD = S::LD, DT = D / 64;   // DT: float4 columns of the output a thread holds
  constexpr int kLoads = BN * (D / 4) / kThreads;      // float4 of K and of V a thread loads a tile
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float* qs = sm + S::kQ;
  float* ks = sm + S::kK;
  float* vs = sm + S::kV;
  float* ps = sm + S::kP;
  int* rows = reinterpret_cast<int*>(sm + S::kRow);
  int bad = 0;
  Walk walk;
  bool faulty;
  const bool work = plan_walk<kThreads>(p, plan, walk, faulty, bad);
  // the kernel before may still write q or read the workspace; the next one
  // reads this one's output after its own wait
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (faulty || !work) publish_none(p, !work, tid, kThreads);
  bool cut = false;
  Segment seg;
  while (work && next_segment(p, walk, seg)) {
    if (seg.starts && seg.hkv == 0 && seg.tok0 == seg.grp.first) check_group(p, seg.grp, tid, kThreads, bad);
    publish_parts(p, seg, tid, kThreads);
    if (p.item_part && seg.starts && !seg.whole) {
      cut = true;
      if (tid == 0) publish_cut(p, seg);
    }
    const int lo = seg.k0 * kKeyTile, hi = min(seg.grp.len, seg.k1 * kKeyTile), hkv = seg.hkv;
    const int n_rows = seg.n_rows;
    const int32_t* table = p.block_table + (size_t)seg.grp.table_row * p.max_pages;
    // q and out index (in heads) of row r
    auto head_of = [&](int r) -> size_t {
      return (size_t)(seg.tok0 + r / p.g) * p.Hq + hkv * p.g + r % p.g;
    };
    auto resolve = [&](int key) -> int { return key < hi ? key_row(p, table, hkv, key, bad) : -1; };
    float4 kx[kLoads], vx[kLoads];
    auto fetch = [&](const int* row) {   // rows without a key as zeros
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int e = tid + u * kThreads, j = e / (D / 4), c = e % (D / 4);
        const int r = row[j];
        const size_t off = (size_t)max(r, 0) * D + 4 * c;
        kx[u] = vx[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r >= 0) {
          kx[u] = load4(static_cast<const float*>(p.k) + off);
          vx[u] = load4(static_cast<const float*>(p.v) + off);
        }
      }
    };
    __syncthreads();   // the segment before is read to the end
    if (tid < BN) rows[tid] = resolve(lo + tid);
    {
      float4 v[R * DT];
#pragma unroll
      for (int u = 0; u < R * DT; ++u) {
        const int e = tid + u * kThreads, r = e / (D / 4), c = e % (D / 4);
        v[u] = r < n_rows ? load4(static_cast<const float*>(p.q) + head_of(r) * D + 4 * c)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < R * DT; ++u) *reinterpret_cast<float4*>(qs + 4 * (tid + u * kThreads)) = v[u];
    }
    __syncthreads();
    fetch(rows);
    int row_next = tid < BN ? resolve(lo + BN + tid) : -1;
    float m[R], l[R];
    float4 o[R][DT];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[i][t] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int it = 0;
    for (int k0 = lo; k0 < hi; k0 += BN, ++it) {
      __syncthreads();   // the tile before is read to the end
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int e = tid + u * kThreads, j = e / (D / 4), c = e % (D / 4);
        *reinterpret_cast<float4*>(ks + j * LD + 4 * c) = kx[u];
        *reinterpret_cast<float4*>(vs + j * D + 4 * c) = vx[u];
      }
      const int* live = rows + (it & 1) * BN;
      int* next = rows + ((it + 1) & 1) * BN;
      if (tid < BN) next[tid] = row_next;
      __syncthreads();
      if (k0 + BN < hi) {
        fetch(next);
        if (tid < BN) row_next = resolve(k0 + 2 * BN + tid);
      }
      float s[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 4; ++c) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(qs + (R * ty + i) * D + 4 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * LD + 4 * c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
            s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
            s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
            s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = live[tx + 16 * j] >= 0 ? s[i][j] * p.scale_log2 : -CUDART_INF_F;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int q = 8; q > 0; q >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
        const float base = mx == -CUDART_INF_F ? 0.f : mx;
        const float al = fast_exp2(m[i] - base);
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = fast_exp2(s[i][j] - base);
          sum += e;
          ps[(R * ty + i) * BN + tx + 16 * j] = e;
        }
        l[i] = fmaf(l[i], al, sum);   // this lane's keys; the 16 lanes join at the end
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          o[i][t].x *= al;
          o[i][t].y *= al;
          o[i][t].z *= al;
          o[i][t].w *= al;
        }
      }
      __syncwarp();   // rows R ty.. of ps are written and read by the same half warp
#pragma unroll 4
      for (int j = 0; j < BN; j += 4) {
        float4 pr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) pr[i] = *reinterpret_cast<const float4*>(ps + (R * ty + i) * BN + j);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            const float4 v = *reinterpret_cast<const float4*>(vs + (j + u) * D + 64 * t + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float w = u == 0 ? pr[i].x : u == 1 ? pr[i].y : u == 2 ? pr[i].z : pr[i].w;
              o[i][t].x = fmaf(w, v.x, o[i][t].x);
              o[i][t].y = fmaf(w, v.y, o[i][t].y);
              o[i][t].z = fmaf(w, v.z, o[i][t].z);
              o[i][t].w = fmaf(w, v.w, o[i][t].w);
            }
          }
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int q = 8; q > 0; q >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], q);
      const int r = R * ty + i;
      if (r >= n_rows) continue;
      const size_t head = head_of(r);
      if (p.out && seg.whole) {
        const float inv = l[i] > 0.f ? __frcp_rn(l[i]) : (l[i] == 0.f ? 0.f : l[i]);
#pragma unroll
        for (int t = 0; t < DT; ++t)
          store4(static_cast<float*>(p.out) + head * D + 64 * t + 4 * tx,
                 make_float4(o[i][t].x * inv, o[i][t].y * inv, o[i][t].z * inv, o[i][t].w * inv));
      } else {
        const size_t at = seg.whole ? head : (size_t)(2 * blockIdx.x + seg.slot) * p.slot_rows + r;
        float* ml = seg.whole ? p.row_ml : p.slot_ml;
        float* acc = seg.whole ? p.row_acc : p.slot_acc;
        if (tx == 0) *reinterpret_cast<float2*>(ml + 2 * at) = make_float2(m[i], l[i]);
        if (lo < hi) {
#pragma unroll
          for (int t = 0; t < DT; ++t) *reinterpret_cast<float4*>(acc + at * D + 64 * t + 4 * tx) = o[i][t];
        }
      }
    }
  }
  if (p.item_part && !cut && tid == 0) publish_no_cut(p);
  if (bad) atomicOr(p.status, bad);
}

// Joins the parts of the cut items of a cross attention: block (c, y) has rows
// 8y.. of the item that starts in CTA c of the row kernel, a warp each row.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const RowsParams p) {
  const int lane = threadIdx.x & 31, r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int4 item = __ldcg(p.item_part + 2 * blockIdx.x);
  const int slot = __ldcg(p.item_part + 2 * blockIdx.x + 1).x;
  if (r >= item.y) return;
  const int n_parts = item.w;   // <= kMaxExt; 0 without a cut item, which has no rows either
  auto row_at = [&](int s) -> size_t {   // of part s in the slots
    return (size_t)(2 * (blockIdx.x + s) + (s == 0 ? slot : 0)) * p.slot_rows + r;
  };
  float ms[2], ls[2];   // parts lane and lane + 32
  float M = -CUDART_INF_F;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int s = lane + 32 * u;
    const float2 x = s < n_parts ? __ldcg(reinterpret_cast<const float2*>(p.slot_ml) + row_at(s))
                                 : make_float2(-CUDART_INF_F, 0.f);
    ms[u] = x.x;
    ls[u] = x.y;
    M = fmaxf(M, x.x);
  }
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, q));
  const float base = M == -CUDART_INF_F ? 0.f : M;
  float sc[2], L = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    sc[u] = fast_exp2(ms[u] - base);
    L = fmaf(ls[u], sc[u], L);
  }
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) L += __shfl_xor_sync(0xffffffffu, L, q);
  float a[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < n_parts; ++s) {
    const float w = __shfl_sync(0xffffffffu, s < 32 ? sc[0] : sc[1], s & 31);
    if (__shfl_sync(0xffffffffu, s < 32 ? ls[0] : ls[1], s & 31) == 0.f) continue;   // no rows there
    const float* src = p.slot_acc + row_at(s) * D + lane * (D / 32);
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      a[0] = fmaf(v.x, w, a[0]);
      a[1] = fmaf(v.y, w, a[1]);
      a[2] = fmaf(v.z, w, a[2]);
      a[3] = fmaf(v.w, w, a[3]);
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      a[0] = fmaf(v.x, w, a[0]);
      a[1] = fmaf(v.y, w, a[1]);
    }
  }
  const float inv = L > 0.f ? __frcp_rn(L) : (L == 0.f ? 0.f : L);
  const size_t head = (size_t)(item.x + r / p.g) * p.Hq + item.z * p.g + r % p.g;
  T* dst = static_cast<T*>(p.out) + head * D + lane * (D / 32);
  if constexpr (D == 128) {
    store4(dst, make_float4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv));
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float2*>(dst) = make_float2(a[0] * inv, a[1] * inv);
  } else {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(a[0] * inv, a[1] * inv);
  }
}

template <int D, int R>
cudaError_t launch_rows_t(int ctas, const RowsParams& p, cudaStream_t s) {
  RowsParams a = p;
  void* args[] = {&a};
  return launch_pdl(reinterpret_cast<const void*>(rows_kernel<D, R>), dim3(ctas), kThreads,
                    SmemF32<D, R>::kBytes, s, args);
}

template <typename T, int D>
cudaError_t launch_merge_t(int ctas, const RowsParams& p, cudaStream_t s) {
  RowsParams a = p;
  void* args[] = {&a};
  return launch_pdl(reinterpret_cast<const void*>(merge_kernel<T, D>),
                    dim3(ctas, (p.slot_rows + kMergeWarps - 1) / kMergeWarps), 32 * kMergeWarps, 0, s, args);
}

template <int D, int R>
cudaError_t prepare_t() {
  return cudaFuncSetAttribute(rows_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SmemF32<D, R>::kBytes);
}

}  // namespace

cudaError_t launch_rows_f32(int head_dim, int ctas, const RowsParams& p, cudaStream_t s) {
  if (p.tile_tokens * p.g <= 16)
    return head_dim == 64 ? launch_rows_t<64, 1>(ctas, p, s) : launch_rows_t<128, 1>(ctas, p, s);
  return head_dim == 64 ? launch_rows_t<64, 4>(ctas, p, s) : launch_rows_t<128, 4>(ctas, p, s);
}

cudaError_t launch_rows_merge(int head_dim, bool bf16, int ctas, const RowsParams& p, cudaStream_t s) {
  if (bf16)
    return head_dim == 64 ? launch_merge_t<__nv_bfloat16, 64>(ctas, p, s)
                          : launch_merge_t<__nv_bfloat16, 128>(ctas, p, s);
  return head_dim == 64 ? launch_merge_t<float, 64>(ctas, p, s) : launch_merge_t<float, 128>(ctas, p, s);
}

cudaError_t prepare_rows_f32() {
  cudaError_t e;
  if ((e = prepare_t<64, 1>())) return e;
  if ((e = prepare_t<128, 1>())) return e;
  if ((e = prepare_t<64, 4>())) return e;
  return prepare_t<128, 4>();
}

}  // namespace fastocr
