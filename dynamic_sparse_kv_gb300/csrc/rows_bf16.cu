// Row attention on the tensor cores (bf16).
//
// A CTA holds up to 256 query rows of one (group, KV head) as two row tiles of
// 128 and streams its share of the keys in tiles of 128:
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S in TMEM (fp32)
//   P           softmax warps: one thread a row reads S, exponentiates in base 2
//               against a lazily moved running max and writes P (bf16) over S
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory, O in TMEM (fp32)
// The two row tiles take turns, so that one's softmax runs under the other's
// products. With at most 128 rows both turns work on the same rows and
// alternate key tiles; their O, max and sum are joined at the end.
//
// Roles: warps 0-3 and 4-7 the softmax of turn 0 and 1 (warp w owns TMEM lanes
// 32 (w % 4)..), warps 8-11 copy K and V rows, gathered from pages of any size,
// into 128-byte-swizzled tiles with 16-byte cp.async, warp 12 issues the MMAs
// (warps 13-15 only make its register share a whole warpgroup's).
#include <math_constants.h>

#include "rows.cuh"

namespace fastocr {

namespace {

constexpr int kThreads = 16 * 32;
// Registers a thread of each role, 128 on average as launched: a softmax thread
// holds a whole row of 128 scores.
constexpr int kRegsSoftmax = 184, kRegsLoad = 88, kRegsMma = 56;
static_assert(2 * kRegsSoftmax + kRegsLoad + kRegsMma == 4 * 128, "the launch's registers");
constexpr int kLoadThreads = 128;
constexpr int kTileRows = 128;
constexpr int kMaskRing = 8;

template <int D>
struct SmemBf16 {
  static constexpr int kTileBytes = 128 * D * 2;     // a row or key tile: blocks of 64 columns
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kQ = 0;                       // two row tiles
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kRow = kRing + kStages * kTileBytes;   // int [2][128]: cache rows of a key tile
  static constexpr int kMask = kRow + 2 * 128 * 4;            // u32 [kMaskRing][4]: keys that exist
  static constexpr int kMl = kRing;   // float2 [2][128]: the turns' max and sum, once the ring is read
  static constexpr int kBar = kMask + kMaskRing * 16;
  static constexpr int kNumBars = 2 * kStages + 1 + 5 * 2;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kDead = kTmem + 4;
  static constexpr int kBytes = kDead + 4 + 1024;    // room to align the base to 1024
};
static_assert(SmemBf16<128>::kBytes <= 227 * 1024, "shared memory of one CTA");

// ---------------------------------------------------------------- PTX helpers

__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for a phase, at most about two seconds: then (a library bug) `dead` is
// set, every later wait gives up at once, and the kernel ends with an error
// status instead of hanging.
__device__ __forceinline__ void mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* dead) {
  const long long t0 = clock64();
  while (!*dead) {
    if (mbar_try(bar, parity)) return;
    if (clock64() - t0 > 4000000000LL) *dead = 1;
  }
}
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
  if (!mbar_try(bar, parity)) mbar_wait_slow(bar, parity, dead);
}

// The issuing warp stays converged, so that operands are computed in uniform
// registers (a divergent single thread took 60-120 cycles an instruction); the
// instructions themselves are predicated to its one elected lane.
__device__ __forceinline__ void tc_commit(uint32_t bar, int elected) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

#define FOCR_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define FOCR_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : FOCR_R8(r, 0), FOCR_R8(r, 8), FOCR_R8(r, 16), FOCR_R8(r, 24)
      : "r"(addr));
}
// Completes this thread's TMEM loads. Nothing but these operands tells the
// compiler that the loaded registers are not valid before the wait, so every
// block of 32 that a load filled is passed through here before it is used.
#define FOCR_T8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
__device__ __forceinline__ void tc_loaded(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : FOCR_T8(r, 0), FOCR_T8(r, 8), FOCR_T8(r, 16), FOCR_T8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::FOCR_I8(r, 0),
      FOCR_I8(r, 8), FOCR_I8(r, 16), FOCR_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::FOCR_I8(r, 0),
      FOCR_I8(r, 8), "r"(addr)
      : "memory");
}

// Shared-memory operand of 128-byte-swizzled rows: `lead` and `stride` are the
// leading and stride byte offsets (fields in units of 16 bytes), bit 46 is the
// descriptor version of this architecture, 2 << 61 the 128-byte swizzle.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, bf16 operands, M = 128, N columns;
// `trans_b`: B's rows are the reduced dimension (V as it lies in the cache).
__host__ __device__ constexpr uint32_t instruction(int n, bool trans_b) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (trans_b ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc,
                                       int elected) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int acc,
                                       int elected) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(elected)
      : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---------------------------------------------------------------- the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const RowsParams p) {
  extern __shared__ unsigned char smem_raw[];
  using S = SmemBf16<D>;
  constexpr int kSt = S::kStages;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.z, hkv = blockIdx.y;
  volatile int* dead = reinterpret_cast<volatile int*>(smem + S::kDead);
  int bad = 0;
  const RowGroup grp = find_tile<2 * kTileRows>(p, blockIdx.x, bad);
  if (grp.tile < 0) {   // the same in every thread
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (bad && tid == 0) atomicOr(p.status, bad);
    return;
  }
  if (split == 0 && hkv == 0 && grp.tile == 0) check_group(p, grp, bad);
  int lo, hi;
  split_range(grp.len, p.splits, split, lo, hi);
  const int row0 = grp.tile * 2 * kTileRows;
  const int n_rows = min(2 * kTileRows, grp.n_rows - row0);
  const bool pair = n_rows > kTileRows;    // two row tiles; else one, its keys in two turns
  const int n_tiles = (hi - lo + kKeyTile - 1) / kKeyTile;
  const int32_t* table = p.block_table + (size_t)grp.table_row * p.max_pages;

  // barriers: ring full / empty, Q, then per turn: S full, P ready, PV done, O done
  auto full = [&](int st) { return sbase + S::kBar + 8 * st; };
  auto empty = [&](int st) { return sbase + S::kBar + 8 * (kSt + st); };
  const uint32_t q_full = sbase + S::kBar + 8 * (2 * kSt);
  auto turn_bar = [&](int kind, int t) { return q_full + 8 + 8 * (2 * kind + t); };
  enum { kSFull = 0, kPReady = 1, kPReady2 = 2, kPvDone = 3, kODone = 4 };
  // warps of a turn that hold rows
  auto warps_of = [&](int t) {
    const int r = pair ? min(kTileRows, n_rows - t * kTileRows) : n_rows;
    return (r + 31) / 32;
  };
  if (tid == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(full(s), kLoadThreads);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 8);
    for (int t = 0; t < 2; ++t) {
      mbar_init(turn_bar(kSFull, t), 2);
      mbar_init(turn_bar(kPReady, t), warps_of(t));
      mbar_init(turn_bar(kPReady2, t), warps_of(t));
      mbar_init(turn_bar(kPvDone, t), 1);
      mbar_init(turn_bar(kODone, t), 1);
    }
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(sbase + S::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kTmem);
  auto s_col = [&](int t) { return tmem + 128 * t; };
  auto o_col = [&](int t) { return tmem + 256 + D * t; };
  // turn t's i-th key tile, and how many it has
  auto tile_of = [&](int t, int i) { return pair ? i : 2 * i + t; };
  auto count_of = [&](int t) { return pair ? n_tiles : (n_tiles + 1 - t) / 2; };

  if (warp < 8) {
    // ---------------- softmax of turn t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, w = warp & 3;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    // Q rows into the swizzled tiles, all warps together
    if (n_tiles > 0) {
      const int c = tid & (D / 8 - 1);
      constexpr int kStep = 256 / (D / 8), kBatch = 8;
      const int total = pair ? 2 * kTileRows : kTileRows;
      for (int r0 = tid / (D / 8); r0 < total; r0 += kBatch * kStep) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kStep;
          v[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < n_rows) {
            const int x = row0 + r;
            const size_t head = (size_t)(grp.first + x / p.g) * p.Hq + hkv * p.g + x % p.g;
            v[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + head * D) + c);
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kStep;
          if (r < total)
            *reinterpret_cast<uint4*>(smem + S::kQ + (r >> 7) * S::kTileBytes + (c >> 3) * 16384 +
                                      (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[u];
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int n = count_of(t);
    const uint32_t lane_base = (uint32_t)(32 * w) << 16;
    float m = -CUDART_INF_F, l = 0.f;
    if (w < warps_of(t)) {
      const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + S::kMask);
      for (int i = 0; i < n; ++i) {
        mbar_wait(turn_bar(kSFull, t), i & 1, dead);
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(x + 32 * c, s_col(t) + lane_base + 32 * c);
        const uint4 mk = *reinterpret_cast<const uint4*>(masks + 4 * (tile_of(t, i) % kMaskRing));
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_loaded(x + 32 * c);
        if ((mk.x & mk.y & mk.z & mk.w) != 0xffffffffu) {
          const uint32_t mw[4] = {mk.x, mk.y, mk.z, mk.w};
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!((mw[c >> 5] >> (c & 31)) & 1u)) x[c] = 0xff800000u;
        }
        float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int c = 0; c < 128; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
        const bool move = top > m + kLazyMax;
        if (__any_sync(0xffffffffu, move)) {
          const float al = move ? fast_exp2(m - top) : 1.f;
          if (move) m = top;
          l *= al;
          if (i > 0) {   // the products before this S are complete
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc_ld32(o, o_col(t) + lane_base + c);
              tc_loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc_st32(o_col(t) + lane_base + c, o);
            }
          }
        }
        const float base = m == -CUDART_INF_F ? 0.f : m;
        const uint64_t scale2 = pack2(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
        const uint64_t base2 = pack2(__float_as_uint(-base), __float_as_uint(-base));
        uint64_t sum[2] = {0ull, 0ull};
        // P in two halves: the product over the first runs under the second
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b;
            unpack2(fma2(pack2(x[32 * c + 2 * e], x[32 * c + 2 * e + 1]), scale2, base2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[e & 1] = add2(sum[e & 1], pack2(__float_as_uint(a), __float_as_uint(b)));
            pk[e] = pack_bf16(a, b);
          }
          tc_st16(s_col(t) + lane_base + 16 * c, pk);
          if (c & 1) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(turn_bar(c == 1 ? kPReady : kPReady2, t));
          }
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      // ---------------- output
      const int r = 32 * w + lane;   // row in the tile
      float* ml = reinterpret_cast<float*>(smem + S::kMl);
      float wt[2];                   // weights of the turns' O
      bool have[2];
      if (pair) {
        if (n > 0) mbar_wait(turn_bar(kODone, t), 0, dead);
        have[0] = have[1] = n > 0;
        wt[0] = wt[1] = 1.f;
      } else {
        for (int u = 0; u < 2; ++u)
          if (count_of(u) > 0) mbar_wait(turn_bar(kODone, u), 0, dead);
        reinterpret_cast<float2*>(ml)[t * 128 + r] = make_float2(m, l);
        asm volatile("bar.sync 1, %0;\n" ::"r"(64 * warps_of(0)) : "memory");
        const float2 o0 = reinterpret_cast<float2*>(ml)[r], o1 = reinterpret_cast<float2*>(ml)[128 + r];
        m = fmaxf(o0.x, o1.x);
        const float base = m == -CUDART_INF_F ? 0.f : m;
        wt[0] = fast_exp2(o0.x - base);
        wt[1] = fast_exp2(o1.x - base);
        l = o0.y * wt[0] + o1.y * wt[1];
        have[0] = count_of(0) > 0;
        have[1] = count_of(1) > 0;
      }
      tc_fence_after();
      const bool direct = p.out && p.splits == 1;
      const float inv = direct ? (l > 0.f ? __frcp_rn(l) : (l == 0.f ? 0.f : l)) : 1.f;
      const int rr = pair ? t * kTileRows + r : r;
      const bool mine = rr < n_rows;
      const int xr = row0 + (mine ? rr : 0);
      const int head = (grp.first + xr / p.g) * p.Hq + hkv * p.g + xr % p.g;   // < 2^31, from the host
      const size_t part = (size_t)split * p.rows * p.Hq;
      if (!direct && mine && (pair || t == 0))
        *reinterpret_cast<float2*>(p.ml + 2 * (part + head)) = make_float2(m, l);
      if (direct || n_tiles > 0) {
        // Half the columns at a time go through this warp's share of its turn's
        // Q tile (read to the end by now), so that rows leave as whole
        // segments: a thread's own 16-byte stores touch 32 rows at once. A pair's
        // turn writes whole rows, otherwise each turn half of them.
        constexpr int kCw = D / 2;                  // columns a round
        unsigned char* stage = smem + S::kQ + t * S::kTileBytes + w * (S::kTileBytes / 4);
        const int valid = min(32, (pair ? n_rows - t * kTileRows : n_rows) - 32 * w);
#pragma unroll 1
        for (int round = 0; round < (pair ? 2 : 1); ++round) {
          const int c0 = pair ? round * kCw : t * kCw;
#pragma unroll 1
          for (int c = 0; c < kCw; c += 32) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
            for (int u = pair ? t : 0; u < (pair ? t + 1 : 2); ++u) {
              if (!have[u]) continue;
              uint32_t y[32];
              tc_ld32(y, o_col(u) + lane_base + c0 + c);
              tc_loaded(y);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(y[e]), wt[u], o[e]);
            }
            if (direct) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                *reinterpret_cast<uint4*>(stage + lane * (kCw * 2) + ((((c + e) >> 3) ^ (lane & (kCw / 8 - 1))) << 4)) =
                    make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                               pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(stage + lane * (kCw * 4) + ((((c + e) >> 2) ^ (lane & 7)) << 4)) =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          __syncwarp();
          const int per_row = direct ? kCw / 8 : kCw / 4;   // 16-byte chunks of a row
          const int swz = direct ? kCw / 8 - 1 : 7;
          for (int e = lane; e < 32 * per_row; e += 32) {
            const int q = e / per_row, ch = e % per_row;
            const int hq = __shfl_sync(0xffffffffu, head, q);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + q * per_row * 16 + ((ch ^ (q & swz)) << 4));
            if (q < valid) {
              if (direct)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)hq * D + c0 + 8 * ch) = v;
              else
                *reinterpret_cast<uint4*>(p.acc + (part + hq) * D + c0 + 4 * ch) = v;
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (warp < 12) {
    // ---------------- K and V rows into the ring: K_0, V_0, K_1, V_1, ...
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsLoad));
    const int lt = tid - 256;
    if (!p.prefix_len) asm volatile("griddepcontrol.wait;\n" ::: "memory");
    int* rows = reinterpret_cast<int*>(smem + S::kRow);
    uint32_t* masks = reinterpret_cast<uint32_t*>(smem + S::kMask);
    constexpr int kChunks = D / 8;                    // 16-byte chunks of a row
    constexpr int kRowsAtOnce = kLoadThreads / kChunks;
    const int c = lt % kChunks, r_lane = lt / kChunks;
    constexpr int kLag = 2;                           // copies in flight behind the newest
    const uint64_t pol = l2_policy_evict_first();
    auto resolve = [&](int j) -> int {
      const int pos = lo + j * kKeyTile + lt;
      return pos < hi ? key_row(p, table, hkv, pos, bad) : -1;
    };
    int next = n_tiles > 0 ? resolve(0) : -1;
    for (int j = 0; j < n_tiles; ++j) {
      rows[(j & 1) * 128 + lt] = next;
      const uint32_t live = __ballot_sync(0xffffffffu, next >= 0);
      if (lane == 0) masks[4 * (j % kMaskRing) + (warp - 8)] = live;
      if (j + 1 < n_tiles) next = resolve(j + 1);
      asm volatile("bar.sync 2, 128;\n" ::: "memory");
      // this thread's cache rows, read together: a load between two copies
      // would make each wait for the last (1050 instead of ... cycles a tile)
      int row[128 / kRowsAtOnce];
#pragma unroll
      for (int i = 0; i < 128 / kRowsAtOnce; ++i) row[i] = rows[(j & 1) * 128 + i * kRowsAtOnce + r_lane];
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int idx = 2 * j + kv, st = idx % kSt;
        if (idx >= kSt) mbar_wait(empty(st), (idx / kSt - 1) & 1, dead);
        const char* src = static_cast<const char*>(kv ? p.v : p.k) + c * 16;
        const uint32_t dst0 = sbase + S::kRing + st * S::kTileBytes + (c >> 3) * 16384;
#pragma unroll
        for (int i = 0; i < 128 / kRowsAtOnce; ++i) {
          const int r = i * kRowsAtOnce + r_lane;
          cp_async16(dst0 + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (size_t)max(row[i], 0) * (D * 2),
                     row[i] >= 0 ? 16 : 0, pol);
        }
        cp_async_commit();
        if (idx >= kLag) {
          cp_async_wait<kLag>();
          fence_async_shared();
          mbar_arrive(full((idx - kLag) % kSt));
        }
      }
    }
    cp_async_wait<0>();
    fence_async_shared();
    for (int idx = max(0, 2 * n_tiles - kLag); idx < 2 * n_tiles; ++idx) mbar_arrive(full(idx % kSt));
  } else {
    // ---------------- MMA: warp 12 issues for the CTA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsMma));
    if (warp == 12 && n_tiles > 0) {
      uint32_t elected;
      asm volatile(
          "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n"
          : "=r"(elected));
      constexpr uint32_t kIdQk = instruction(128, false), kIdPv = instruction(D, true);
      constexpr uint64_t kKMajor = 1ull << 16, kVMajor = (uint64_t)(16384 >> 4) << 16;   // leading offsets
      const uint64_t q_op = operand(sbase + S::kQ, 0, 1024), ring_op = operand(sbase + S::kRing, 0, 1024);
      auto wait_ring = [&](int idx) { mbar_wait(full(idx % kSt), (idx / kSt) & 1, dead); };
      auto qk = [&](int t, int j) {
        const int st = (2 * j) % kSt;
        const uint64_t a = q_op + ((pair ? t : 0) * S::kTileBytes >> 4) + kKMajor;
        const uint64_t b = ring_op + (st * S::kTileBytes >> 4) + kKMajor;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          mma_ss(s_col(t), a + off, b + off, kIdQk, k > 0, elected);
        }
        tc_commit(turn_bar(kSFull, t), elected);
        if (elected) mbar_arrive(turn_bar(kSFull, t));   // orders the key mask before the softmax's reading
        __syncwarp();
        if (!pair || t == 1) tc_commit(empty(st), elected);
      };
      auto pv = [&](int t, int i, int j, bool first, bool last) {
        const int st = (2 * j + 1) % kSt;
        const uint64_t b = ring_op + (st * S::kTileBytes >> 4) + kVMajor;
        mbar_wait(turn_bar(kPReady, t), i & 1, dead);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(o_col(t), s_col(t) + 8 * k, b + (2048 * k >> 4), kIdPv, !first || k > 0, elected);
        mbar_wait(turn_bar(kPReady2, t), i & 1, dead);
        tc_fence_after();
#pragma unroll
        for (int k = 4; k < 8; ++k)
          mma_ts(o_col(t), s_col(t) + 8 * k, b + (2048 * k >> 4), kIdPv, 1, elected);
        tc_commit(turn_bar(last ? kODone : kPvDone, t), elected);
        if (!pair || t == 1) tc_commit(empty(st), elected);
      };
      mbar_wait(q_full, 0, dead);
      tc_fence_after();
      for (int t = 0; t < 2; ++t)
        if (count_of(t) > 0) {
          if (t == 0 || !pair) wait_ring(2 * tile_of(t, 0));
          tc_fence_after();
          qk(t, tile_of(t, 0));
        }
      for (int i = 0; i < count_of(0); ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = count_of(t);
          if (i >= n) continue;
          const bool last = i + 1 == n;
          wait_ring(2 * tile_of(t, i) + 1);
          pv(t, i, tile_of(t, i), i == 0, last);
          if (!last) {
            wait_ring(2 * tile_of(t, i + 1));
            mbar_wait(turn_bar(kPvDone, t), i & 1, dead);   // S overwrites the P that PV reads
            tc_fence_after();
            qk(t, tile_of(t, i + 1));
          }
        }
      for (int t = 0; t < 2; ++t)
        if (count_of(t) > 0) mbar_wait(turn_bar(kODone, t), 0, dead);
    }
    __syncwarp();
  }
  if (bad) atomicOr(p.status, bad);
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *dead) atomicOr(p.status, kDevInternal);
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

template <int D>
cudaError_t launch_t(const RowsParams& p, cudaStream_t s) {
  RowsParams a = p;
  void* args[] = {&a};
  return launch_pdl(reinterpret_cast<const void*>(rows_kernel<D>),
                    dim3((unsigned)max_row_tiles(p, kRowsBf16), p.Hkv, p.splits), kThreads,
                    SmemBf16<D>::kBytes, s, args);
}

template <int D>
cudaError_t prepare_t() {
  cudaError_t e = cudaFuncSetAttribute(rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       SmemBf16<D>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(rows_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

}  // namespace

cudaError_t launch_rows_bf16(int head_dim, const RowsParams& p, cudaStream_t s) {
  return head_dim == 64 ? launch_t<64>(p, s) : launch_t<128>(p, s);
}

cudaError_t prepare_rows_bf16() {
  const cudaError_t e = prepare_t<64>();
  return e != cudaSuccess ? e : prepare_t<128>();
}

}  // namespace fastocr
