// Row attention on the tensor cores (bf16).
//
// A CTA holds up to 256 query rows of one (group, KV head) as two row tiles of
// 128 and streams its share of the keys in tiles of 128:
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S in TMEM (fp32)
//   P           softmax warps: one thread a row reads S, exponentiates in base 2
//               against the row's base and writes P (bf16) over S
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory, O in TMEM (fp32)
// The two row tiles take turns, so that one's softmax runs under the other's
// products. With at most 128 rows both turns work on the same rows and
// alternate key tiles; their O, max and sum are joined at the end.
//
// Roles: warps 0-3 and 4-7 the softmax of turn 0 and 1 (warp w owns TMEM lanes
// 32 (w % 4)..), warps 8-11 copy K and V rows, gathered from pages of any size,
// into 128-byte-swizzled tiles with 16-byte cp.async, warp 12 issues the MMAs
// (warps 13-15 only make its register share a whole warpgroup's). TMA in the
// copies' place was slower here: a page of 16 keys makes boxes of 2 KB, 23
// bytes a cycle and SM (4 x 1024 queries on 8320 states 437 us), and four
// gathered rows an instruction 7 (1190 us); K by TMA next to V by cp.async 380 us;
// cp.async alone 370 us, all before the work was dealt out evenly.
//
// Many rows (4 x 1024 queries, 28 heads, up to 8320 states): 275 us back to back (1.18
// PFLOP/s), 290 to 299 us as a call among others (1.09 to 1.12). The products of a key
// tile of two row tiles take 2048 cycles, alone and at full rate as measured, a tile
// here 3200. What bounds it is a turn's chain: S = QK^T, 1400 cycles of softmax
// behind TMEM loads, PV, and about 250 cycles each time a commit or a P has to be seen
// through a barrier. The turn's next S is issued behind its PV, which reads P from
// columns 0-63 of S's 128; the other 64 are free once the scores are in registers, and
// with D = 64 another 128 of TMEM's 512 are, so half an S could start earlier (not
// tried). A sixth of a CTA's cycles are the starts and ends of its three or four
// segments. The compiler spills 168 bytes of stores and 228 of loads at D = 128 (148
// and 208 at 64). It is not the copies: without any, 284 us became 273. Against those
// 284 us, sixteen softmax warps with half a row each took 283 (the issuing warp is the
// slowest link then), an issuing warp a turn 309 (the turns' products interleave and
// both end late), a warp apart for the block table 283, and S loaded in blocks of 32
// columns under the exponentials 351 (far more spills). D = 64: 213 us.
// Few rows: the chain of a start, one or two tiles and the output, 9 us in all (8
// sequences on 4160 keys), and the parts' way through the L2.
#include <math_constants.h>

#include <type_traits>

#include "rows.cuh"

namespace fastocr {

namespace {

constexpr int kThreads = 16 * 32;
// Registers a thread of each role, 128 on average as launched: a softmax thread
// holds a whole row of 128 scores.
constexpr int kRegsSoftmax = 184, kRegsLoad = 80, kRegsMma = 64;
static_assert(2 * kRegsSoftmax + kRegsLoad + kRegsMma == 4 * 128, "the launch's registers");
constexpr int kLoadThreads = 128;
constexpr int kTileRows = 128;
constexpr int kMaskRing = 8;
// A probability may grow to 2^kRange before its row's base moves: sums of 2^30
// of them times values up to 2^30 stay inside fp32 and bf16.
constexpr float kRange = 60.f;

template <int D>
struct SmemBf16 {
  static constexpr int kTileBytes = 128 * D * 2;     // a row or key tile: blocks of 64 columns
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kQ = 0;                       // two row tiles
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kMask = kRing + kStages * kTileBytes;  // u32 [kMaskRing][4]: keys that exist
  static constexpr int kWalk = kMask + kMaskRing * 16;        // Walk [13]: each warp's, kept out of its registers
  static constexpr int kSeg = kWalk + 13 * (int)sizeof(Walk); // Segment [13]: likewise
  static constexpr int kBar = (kSeg + 13 * (int)sizeof(Segment) + 7) / 8 * 8;
  static constexpr int kNumBars = 2 * kStages + 2 + 5 * 2;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kDead = kTmem + 4;
  static constexpr int kFaulty = kDead + 4;          // see plan_walk
  static constexpr int kBytes = kFaulty + 4;
};
static_assert(SmemBf16<128>::kBytes <= 227 * 1024, "shared memory of one CTA");

// ---------------------------------------------------------------- PTX helpers

__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Arrives once every cp.async this thread has issued so far has landed.
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
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
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
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

// next_segment with the walk in shared memory: it is needed between segments only.
__device__ __forceinline__ bool next_from(const RowsParams& p, Walk* walk, Segment* seg) {
  Walk w = *walk;
  Segment s;
  __syncwarp();
  const bool more = next_segment(p, w, s);
  if ((threadIdx.x & 31) == 0) {
    *walk = w;
    if (more) *seg = s;
  }
  __syncwarp();
  return more;
}

// ---------------------------------------------------------------- the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const RowsParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = SmemBf16<D>;
  constexpr int kSt = S::kStages;
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* dead = reinterpret_cast<volatile int*>(smem + S::kDead);
  int bad = 0;
  Walk* walk = reinterpret_cast<Walk*>(smem + S::kWalk) + min(warp, 12);
  {
    Walk w;
    bool faulty;
    if (!plan_walk<kThreads>(p, *reinterpret_cast<PlanSmem*>(smem), w, faulty, bad)) {
      asm volatile("griddepcontrol.wait;\n" ::: "memory");
      publish_none(p, true, tid, kThreads);
      if (p.item_part && tid == 0) publish_no_cut(p);
      if (bad) atomicOr(p.status, bad);
      return;
    }
    if (lane == 0 && warp < 13) *walk = w;
    if (tid == 0) *reinterpret_cast<int*>(smem + S::kFaulty) = faulty;
  }

  // barriers: ring full / empty, Q, O read, then per turn: S full, P ready (two
  // halves), PV done, O done
  auto full = [&](int st) { return sbase + S::kBar + 8 * st; };
  auto empty = [&](int st) { return sbase + S::kBar + 8 * (kSt + st); };
  const uint32_t q_full = sbase + S::kBar + 8 * (2 * kSt), o_free = q_full + 8;
  auto turn_bar = [&](int kind, int t) { return q_full + 16 + 8 * (2 * kind + t); };
  enum { kSFull = 0, kPReady = 1, kPReady2 = 2, kPvDone = 3, kODone = 4 };
  if (tid == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(full(s), kLoadThreads + kLoadThreads / 32);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 8);
    mbar_init(o_free, 8);
    for (int t = 0; t < 2; ++t) {
      mbar_init(turn_bar(kSFull, t), 2);
      mbar_init(turn_bar(kPReady, t), 4);
      mbar_init(turn_bar(kPReady2, t), 4);
      mbar_init(turn_bar(kPvDone, t), 1);
      mbar_init(turn_bar(kODone, t), 1);
    }
    *dead = (sbase & 1023u) != 0;   // the swizzled tiles need that alignment
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
  // A segment with more than 128 rows has a row tile for each turn (a pair),
  // otherwise its key tiles alternate: turn t's i-th tile, and how many it has.
  auto tile_of = [](bool pair, int t, int i) { return pair ? i : 2 * i + t; };
  auto count_of = [](bool pair, int n, int t) { return pair ? n : (n + 1 - t) / 2; };
  Segment* seg_p = reinterpret_cast<Segment*>(smem + S::kSeg) + min(warp, 12);

  if (warp < 8) {
    // ---------------- softmax of turn t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, w = warp & 3;
    bool more = next_from(p, walk, seg_p);   // there is a first segment; found while the kernel before ends
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const uint32_t lane_base = (uint32_t)(32 * w) << 16;
    const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + S::kMask);
    const int g_inv = inverse_of(p.g);
    int s_count = 0;      // S tiles this turn has seen
    int k_count = 0;      // key tiles of the segments before
    bool cut = false;
    // index (in heads of q and out) of row r of an item
    auto head_of = [&](int tok0, int hkv, int r) -> int {   // < 2^31, from the host
      const int tok = token_of_row(r, g_inv);
      return (tok0 + tok) * p.Hq + hkv * p.g + r - tok * p.g;
    };
    for (int n_seg = 0; more; ++n_seg) {
      const int n_tiles = seg_p->k1 - seg_p->k0;
      const bool pair = seg_p->n_rows > kTileRows;
      const int n = count_of(pair, n_tiles, t);
      {
      const Segment seg = *seg_p;
      if (seg.starts && seg.hkv == 0 && seg.tok0 == seg.grp.first) check_group(p, seg.grp, tid, 256, bad);
      publish_parts(p, seg, tid, 256);
      if (p.item_part && seg.starts && !seg.whole) {
        cut = true;
        if (tid == 0) publish_cut(p, seg);
      }
      // Q rows into the swizzled tiles, all warps together
      if (n_seg > 0) asm volatile("bar.sync 1, 256;\n" ::: "memory");   // the output before is staged there
      if (n_tiles > 0) {
        const int c = tid & (D / 8 - 1);
        constexpr int kStep = 256 / (D / 8), kBatch = 2 * kTileRows / kStep;   // loads in flight
        const int total = pair ? 2 * kTileRows : kTileRows;
        {
          const int r0 = tid / (D / 8);
          uint4 v[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int r = r0 + u * kStep;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < seg.n_rows)
              v[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                           (size_t)head_of(seg.tok0, seg.hkv, r) * D) + c);
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
      }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      // this warp's rows of its turn's tile
      const int valid = min(32, seg_p->n_rows - (pair ? t * kTileRows : 0) - 32 * w);
      float m = -CUDART_INF_F, l = 0.f;
      for (int i = 0; i < n; ++i, ++s_count) {
        mbar_wait(turn_bar(kSFull, t), s_count & 1, dead);
        tc_fence_after();
        if (valid <= 0) {   // no rows: P is never read back
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(turn_bar(kPReady, t));
            mbar_arrive(turn_bar(kPReady2, t));
          }
          continue;
        }
        // scores in base-2 units times 1 / scale_log2; keys that do not exist at -inf
        uint32_t x[128];
        auto load_scores = [&]() {
#pragma unroll
          for (int c = 0; c < 4; ++c) tc_ld32(x + 32 * c, s_col(t) + lane_base + 32 * c);
          const uint4 mk = *reinterpret_cast<const uint4*>(masks + 4 * ((k_count + tile_of(pair, t, i)) % kMaskRing));
#pragma unroll
          for (int c = 0; c < 4; ++c) tc_loaded(x + 32 * c);
          if ((mk.x & mk.y & mk.z & mk.w) != 0xffffffffu) {
            const uint32_t mw[4] = {mk.x, mk.y, mk.z, mk.w};
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!((mw[c >> 5] >> (c & 31)) & 1u)) x[c] = 0xff800000u;
          }
        };
        auto max_of = [&](int c0, int c1, float mx[4]) {
#pragma unroll
          for (int c = c0; c < c1; c += 2)
            mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        };
        load_scores();
        if (i == 0) {
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
          max_of(0, 128, mx);
          m = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
        }
        // P in two halves: the product over the first runs under the second. The
        // base is the max of the first tile; a tile's own max is taken under
        // its exponentials and only checked, since what a probability may not do
        // is leave fp32's range: all values of P, l and O keep their relative
        // precision however far they are above 1.
        uint32_t pk[32];
        uint64_t sum[2] = {0ull, 0ull};
        const uint64_t scale2 = pack2(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
        uint64_t base2;
        auto exp_half = [&](int half, float mx[4]) {
          sum[0] = half ? sum[0] : 0ull;
          sum[1] = half ? sum[1] : 0ull;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a, b;
            unpack2(fma2(pack2(x[64 * half + 2 * e], x[64 * half + 2 * e + 1]), scale2, base2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            // P is rounded to bf16, each value by 2^-8 at most, which the products take;
            // l adds the values themselves, since a weighed step makes the rows' weights
            // of it. Relative error against 64 bits 0.0019 to 0.0025, with fp32
            // probabilities 0.0017. Adding the rounded values, so that a row's weights sum
            // to 1, leaves 0.0019 to 0.0022 for 3 % more time (8 % with few rows); a second
            // bf16 part (as in the attend kernel's weigh mode) would make the products of a
            // tile half as long again.
            sum[e & 1] = add2(sum[e & 1], pack2(__float_as_uint(a), __float_as_uint(b)));
            pk[e] = pack_bf16(a, b);
            if (!half) max_of(4 * e, 4 * e + 4, mx);
          }
        };
        auto set_base = [&]() {
          const float base = m == -CUDART_INF_F ? 0.f : m;
          base2 = pack2(__float_as_uint(-base), __float_as_uint(-base));
        };
        set_base();
        while (true) {
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
          exp_half(0, mx);
          const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
          const bool move = top > m + kRange;
          if (!__any_sync(0xffffffffu, move)) break;
          // a new base: what the tiles before left moves to it, and this half is
          // made again (at most once a tile: the base is then its max)
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
          load_scores();
          set_base();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half) exp_half(1, nullptr);
          tc_st32(s_col(t) + lane_base + 32 * half, pk);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(turn_bar(half ? kPReady2 : kPReady, t));
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      k_count += n_tiles;

      // ---------------- output; the next segment is found, and its Q fetched
      // into L2, under the last products
      const int r = 32 * w + lane;   // row in the turn's tile
      const int rr = (pair ? t * kTileRows : 0) + (lane < valid ? r : 0);
      const bool whole = seg_p->whole, direct = p.out && whole;
      // where this row goes: the output, a slot, or a shared prefix's whole rows
      const int at = whole ? head_of(seg_p->tok0, seg_p->hkv, rr)
                           : (2 * (int)blockIdx.x + seg_p->slot) * p.slot_rows + rr;
      more = next_from(p, walk, seg_p);
      if (more && tid < seg_p->n_rows) {
        const char* row = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                        (size_t)head_of(seg_p->tok0, seg_p->hkv, tid) * D);
#pragma unroll
        for (int e = 0; e < D * 2; e += 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(row + e));
      }
      float wt[2] = {1.f, 1.f};      // weights of the turns' O
      bool have[2] = {n > 0, n > 0};
      mbar_wait(turn_bar(kODone, t), n_seg & 1, dead);
      if (!pair) {
        // the turns' max and sum meet in the Q tile that one row tile leaves free
        mbar_wait(turn_bar(kODone, 1 - t), n_seg & 1, dead);
        float2* ml = reinterpret_cast<float2*>(smem + S::kQ + S::kTileBytes);
        ml[t * 128 + r] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;\n" ::: "memory");
        const float2 o0 = ml[r], o1 = ml[128 + r];
        asm volatile("bar.sync 1, 256;\n" ::: "memory");
        m = fmaxf(o0.x, o1.x);
        const float base = m == -CUDART_INF_F ? 0.f : m;
        wt[0] = fast_exp2(o0.x - base);
        wt[1] = fast_exp2(o1.x - base);
        l = o0.y * wt[0] + o1.y * wt[1];
        have[0] = count_of(pair, n_tiles, 0) > 0;
        have[1] = count_of(pair, n_tiles, 1) > 0;
      }
      tc_fence_after();
      if (valid > 0) {
        const float inv = direct ? (l > 0.f ? __frcp_rn(l) : (l == 0.f ? 0.f : l)) : 1.f;
        float* ml_dst = whole ? p.row_ml : p.slot_ml;
        float* acc_dst = whole ? p.row_acc : p.slot_acc;
        if (!direct && lane < valid && (pair || t == 0))
          *reinterpret_cast<float2*>(ml_dst + 2 * (size_t)at) = make_float2(m, l);
        if (direct || n_tiles > 0) {
          // Half the columns at a time go through this warp's share of its turn's
          // Q tile (read to the end by now), so that rows leave as whole
          // segments: a thread's own 16-byte stores touch 32 rows at once. A pair's
          // turn writes whole rows, otherwise each turn half of them.
          constexpr int kCw = D / 2;                  // columns a round
          unsigned char* stage = smem + S::kQ + t * S::kTileBytes + w * (S::kTileBytes / 4);
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
            // rows out: kRow lanes a row, 16 bytes each
            auto rows_out = [&](auto direct_c) {
              constexpr bool kDirect = decltype(direct_c)::value;
              constexpr int kRow = kDirect ? kCw / 8 : kCw / 4, kSwz = kDirect ? kCw / 8 - 1 : 7;
              constexpr int kAtOnce = kRow < 8 ? kRow : 8;
              const int ch = lane % kRow;
              char* dst = kDirect ? static_cast<char*>(p.out) + c0 * 2 + ch * 16
                                  : reinterpret_cast<char*>(acc_dst) + c0 * 4 + ch * 16;
#pragma unroll
              for (int e0 = 0; e0 < kRow; e0 += kAtOnce) {
                uint4 v[kAtOnce];
                int to[kAtOnce];
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e) {
                  const int q = (e0 + e) * (32 / kRow) + lane / kRow;
                  to[e] = __shfl_sync(0xffffffffu, at, q);
                  if (q >= valid) to[e] = -1;
                  v[e] = *reinterpret_cast<const uint4*>(stage + q * kRow * 16 + ((ch ^ (q & kSwz)) << 4));
                }
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                  if (to[e] >= 0) *reinterpret_cast<uint4*>(dst + (size_t)to[e] * (D * (kDirect ? 2 : 4))) = v[e];
              }
            };
            if (direct)
              rows_out(std::true_type());
            else
              rows_out(std::false_type());
            __syncwarp();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
    if (p.item_part && !cut && tid == 0) publish_no_cut(p);
  } else if (warp < 12) {
    // ---------------- K and V rows into the ring: K_0, V_0, K_1, V_1, ...
    // Warp w copies keys 32w .. of a tile: lane l looks key 32w + l up, and every
    // copy gets its row by a shuffle, so that the warps need not meet.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsLoad));
    const int w = warp - 8;
    uint32_t* masks = reinterpret_cast<uint32_t*>(smem + S::kMask);
    constexpr int kChunks = D / 8;                    // 16-byte chunks of a row
    constexpr int kRowsAtOnce = 32 / kChunks;         // rows an instruction covers
    constexpr int kCopies = 32 / kRowsAtOnce;
    const int c = lane % kChunks, r_lane = lane / kChunks;
    // this lane's place in row r_lane of the warp's rows; rows 8 apart have the same
    // swizzle, so copy i adds a constant to that of copy i % kSwz
    constexpr int kSwz = 8 / kRowsAtOnce;
    uint32_t place[kSwz];
#pragma unroll
    for (int i = 0; i < kSwz; ++i) {
      const int r = i * kRowsAtOnce + r_lane;
      place[i] = sbase + S::kRing + (c >> 3) * 16384 + (32 * w + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
    // for keys that one or two row tiles read (64 sequences in 4 groups 89 us, 97
    // with evict_normal); 29 row tiles of a group would be 2% faster with that, which
    // a choice between the two costs again in registers
    const uint64_t pol = l2_policy_evict_first();
    int idx = 0;                                      // tiles copied into the ring so far
    int k_count = 0;
    while (next_from(p, walk, seg_p)) {
      const int32_t* table = p.block_table + (size_t)seg_p->grp.table_row * p.max_pages;
      const int lo = seg_p->k0 * kKeyTile, hi = min(seg_p->grp.len, seg_p->k1 * kKeyTile);
      const int n_tiles = seg_p->k1 - seg_p->k0, hkv = seg_p->hkv;
      // the segment's part of the block table into L2, a 32-byte sector a lookup
      for (int e = (lo >> p.log2_page) + 8 * (tid - 256); e < (hi + (1 << p.log2_page) - 1) >> p.log2_page;
           e += 8 * kLoadThreads)
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(table + e));
      // this lane's key of tile j: its page number, loaded two tiles ahead and not
      // looked at before its turn (the load returns behind the copies in flight)
      auto page_of = [&](int j) -> int {
        const int pos = lo + j * kKeyTile + 32 * w + lane;
        return j < n_tiles && pos < hi ? __ldcg(table + (pos >> p.log2_page)) : -1;
      };
      int page = page_of(0), page_next = page_of(1);
      for (int j = 0; j < n_tiles; ++j, ++k_count) {
        const int pos = lo + j * kKeyTile + 32 * w + lane;
        int key = -1;
        if (pos < hi) {
          if (page < 0 || page >= p.num_pages)
            bad |= kDevBadPage;
          else
            key = ((page * p.Hkv + hkv) << p.log2_page) | (pos & ((1 << p.log2_page) - 1));
        }
        const uint32_t live = __ballot_sync(0xffffffffu, key >= 0);
        if (lane == 0) masks[4 * (k_count % kMaskRing) + w] = live;
        page = page_next;
        page_next = page_of(j + 2);
        int row[kCopies];
#pragma unroll
        for (int i = 0; i < kCopies; ++i) row[i] = __shfl_sync(0xffffffffu, key, i * kRowsAtOnce + r_lane);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++idx) {
          const int st = idx % kSt;
          if (idx >= kSt) mbar_wait(empty(st), (idx / kSt - 1) & 1, dead);
          const char* src = static_cast<const char*>(kv ? p.v : p.k) + c * 16;
          const uint32_t off = st * S::kTileBytes;
#pragma unroll
          for (int i = 0; i < kCopies; ++i)
            cp_async16(place[i % kSwz] + off + i / kSwz * 1024, src + (size_t)max(row[i], 0) * (D * 2),
                       row[i] >= 0 ? 16 : 0, pol);
          // The arrival is left to the copies' completion and the fence to the
          // MMA's side: fence.proxy.async here would wait for every copy in
          // flight, so that one tile at a time was loaded.
          mbar_arrive_copies(full(st));
          // The copies' arrival does not order this warp's key mask before the softmax's
          // reading, which follows from this barrier by way of the MMA; a plain one does.
          if (lane == 0) mbar_arrive(full(st));
        }
      }
    }
    cp_async_wait_all();
  } else {
    // ---------------- MMA: warp 12 issues for the CTA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsMma));
    if (warp == 12) {
      uint32_t elected;
      asm volatile(
          "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n"
          : "=r"(elected));
      constexpr uint32_t kIdQk = instruction(128, false), kIdPv = instruction(D, true);
      constexpr uint64_t kKMajor = 1ull << 16, kVMajor = (uint64_t)(16384 >> 4) << 16;   // leading offsets
      const uint64_t q_op = operand(sbase + S::kQ, 0, 1024), ring_op = operand(sbase + S::kRing, 0, 1024);
      int idx0 = 0;              // ring index of the segment's first tile
      int n_seg = 0;
      int s_count[2] = {0, 0};   // per turn: S tiles made, PV commits before the last of a segment
      int pv_count[2] = {0, 0};
      for (; next_from(p, walk, seg_p); ++n_seg) {
        const int n_tiles = seg_p->k1 - seg_p->k0;
        const bool pair = seg_p->n_rows > kTileRows;
        const int count[2] = {count_of(pair, n_tiles, 0), count_of(pair, n_tiles, 1)};
        auto wait_ring = [&](int i) {
          mbar_wait(full((idx0 + i) % kSt), ((idx0 + i) / kSt) & 1, dead);
          fence_async_shared();   // the copies are generic writes, the MMA reads by the async proxy
        };
        auto qk = [&](int t, int j) {
          const int st = (idx0 + 2 * j) % kSt;
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
        auto pv = [&](int t, int j, bool first, bool last) {
          const int st = (idx0 + 2 * j + 1) % kSt;
          const uint64_t b = ring_op + (st * S::kTileBytes >> 4) + kVMajor;
          mbar_wait(turn_bar(kPReady, t), s_count[t] & 1, dead);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(o_col(t), s_col(t) + 8 * k, b + (2048 * k >> 4), kIdPv, !first || k > 0, elected);
          mbar_wait(turn_bar(kPReady2, t), s_count[t] & 1, dead);
          tc_fence_after();
#pragma unroll
          for (int k = 4; k < 8; ++k)
            mma_ts(o_col(t), s_col(t) + 8 * k, b + (2048 * k >> 4), kIdPv, 1, elected);
          tc_commit(turn_bar(last ? kODone : kPvDone, t), elected);
          if (!pair || t == 1) tc_commit(empty(st), elected);
          ++s_count[t];
        };
        mbar_wait(q_full, n_seg & 1, dead);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (count[t] > 0) {
            if (t == 0 || !pair) wait_ring(2 * tile_of(pair, t, 0));
            tc_fence_after();
            qk(t, tile_of(pair, t, 0));
          }
        // the output before must have been read out of O
        if (n_seg > 0) mbar_wait(o_free, (n_seg - 1) & 1, dead);
        tc_fence_after();
        for (int i = 0; i < count[0]; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int n = count[t];
            if (i >= n) continue;
            const bool last = i + 1 == n;
            if (t == 0 || !pair) wait_ring(2 * tile_of(pair, t, i) + 1);   // else the other turn waited
            pv(t, tile_of(pair, t, i), i == 0, last);
            if (!last) {
              if (t == 0 || !pair) wait_ring(2 * tile_of(pair, t, i + 1));
              mbar_wait(turn_bar(kPvDone, t), pv_count[t] & 1, dead);   // S overwrites the P that PV reads
              ++pv_count[t];
              tc_fence_after();
              qk(t, tile_of(pair, t, i + 1));
            }
          }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (count[t] == 0) tc_commit(turn_bar(kODone, t), elected);   // every segment has this phase
          mbar_wait(turn_bar(kODone, t), n_seg & 1, dead);
        }
        tc_fence_after();
        idx0 += 2 * n_tiles;
      }
    }
    __syncwarp();
  }
  if (bad) atomicOr(p.status, bad);
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *dead) atomicOr(p.status, kDevInternal);
  if (*reinterpret_cast<const int*>(smem + S::kFaulty)) publish_none(p, false, tid, kThreads);
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

template <int D>
cudaError_t launch_t(int ctas, const RowsParams& p, cudaStream_t s) {
  RowsParams a = p;
  void* args[] = {&a};
  return launch_pdl(reinterpret_cast<const void*>(rows_kernel<D>), dim3(ctas), kThreads,
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

cudaError_t launch_rows_bf16(int head_dim, int ctas, const RowsParams& p, cudaStream_t s) {
  return head_dim == 64 ? launch_t<64>(ctas, p, s) : launch_t<128>(ctas, p, s);
}

cudaError_t prepare_rows_bf16() {
  const cudaError_t e = prepare_t<64>();
  return e != cudaSuccess ? e : prepare_t<128>();
}

}  // namespace fastocr
