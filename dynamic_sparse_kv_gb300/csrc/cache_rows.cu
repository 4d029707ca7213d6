// Rows of a paged cache: rotary positions and the write of new tokens, and the way back.
//
// Write. Pair i of a rotary head dimension turns by the angle of its axis' position:
// (x0, x1) -> (x0 c - x1 s, x1 c + x0 s), c and s from a table in 32 bits made of angles in
// 64 bits (a position of 32768 loses 11 of a float's 24 bits to its whole turns). The
// products are rounded one by one, not fused, so the codes of a cache in 4 bits do not
// depend on how a compiler contracts them. The work is a copy: D / 16 neighbouring threads
// take a token's head, 8 dims of either half each (16-byte accesses; in rotate-halves
// layout every pair is then inside a thread, and a group of 16 inside two), and go through
// heads slot, slot + slots, ... of the token with its cosines in registers. `slots` spreads
// the heads of few tokens over the SMs (one token of 36 heads: 36 slots) and is 1 where
// the tokens alone fill them.
//
// Read. A thread takes 16 dims (one group) of one row.
#include <cuda_bf16.h>
#include <float.h>
#include <math_constants.h>

#include "attend_kernels.cuh"
#include "cache_rows.cuh"
#include "fastocr.h"
#include "fp4.cuh"

namespace fastocr {
namespace {

constexpr int kThreads = 256;

// Sequence of a packed token (the last that starts at or before it), or -1: none has it.
__device__ __forceinline__ int sequence_of(const CacheRows& c, int token, int& first, int& end) {
  if (!c.start) {
    first = token;
    end = token + 1;
    return token < c.B ? token : -1;
  }
  int lo = 0, hi = c.B;   // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(c.start + mid) <= token)
      lo = mid;
    else
      hi = mid;
  }
  first = __ldcg(c.start + lo);
  end = __ldcg(c.start + lo + 1);
  return token >= first && token < end ? lo : -1;
}

// Page slot of a token's row, as rows of one KV head are counted ((page * H_kv) << log2_page,
// plus the slot), or -1 for none; the token is the last but (end - 1 - token) of sequence b.
__device__ __forceinline__ long row_of(const CacheRows& c, int b, int token, int first, int end, int& bad) {
  int n = __ldcg(c.seq_len + b);
  if (n < 0 || n > (c.max_pages << c.log2_page)) {
    bad |= kDevBadSeqLen;
    return -1;
  }
  const long r = (long)n - (end - token);
  if (first < 0 || end > c.tokens || r < 0) {
    bad |= kDevBadGroup;
    return -1;
  }
  const int page = __ldcg(c.block_table + (size_t)b * c.max_pages + (r >> c.log2_page));
  if (page < 0 || page >= c.num_pages) {
    bad |= kDevBadPage;
    return -1;
  }
  return (((long)page * c.Hkv) << c.log2_page) + (r & ((1 << c.log2_page) - 1));
}

__device__ __forceinline__ void load8(const char* at, float x[8], const __nv_bfloat16*) {
  const uint4 w = __ldcg(reinterpret_cast<const uint4*>(at));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const char* at, float x[8], const float*) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(at)), b = __ldcg(reinterpret_cast<const float4*>(at) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(char* at, const float x[8], const __nv_bfloat16*) {
  *reinterpret_cast<uint4*>(at) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(char* at, const float x[8], const float*) {
  reinterpret_cast<float4*>(at)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(at)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// 8 dims of a group of 16 whose other 8 the neighbouring lane holds, as codes; *scale is
// the group's. Every lane of the warp takes part.
__device__ __forceinline__ uint32_t pack_codes(const float x[8], float gain, uint32_t* scale) {
  float y[8], top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = __fdiv_rn(x[i], gain);
    top = fmaxf(top, fabsf(y[i]));
    finite &= fabsf(y[i]) <= FLT_MAX;   // false for NaN
  }
  top = finite ? top : CUDART_INF_F;
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  uint32_t s;
  asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, 0f00000000, %1;\n cvt.u32.u16 %0, t;\n}\n"
      : "=r"(s)
      : "f"(__fdiv_rn(top, 6.f)));
  const uint32_t pair = e4m3_pair(s);
  const float sf = unpack_f16(pair).x;
  const bool live = top <= FLT_MAX && sf > 0.f;
  *scale = top <= FLT_MAX ? s : 0x7fu;   // a NaN or an infinity makes the group NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = live ? __fdiv_rn(y[i], sf) : 0.f;
  uint32_t code;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(code)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return code;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) write_kernel(const WriteParams p) {
  using Q = typename Held<T>::Q;
  constexpr int L = D / 16;   // threads a head
  constexpr int E = sizeof(Q);
  const CacheRows& c = p.c;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  // One token a sequence: only row N_b - 1 is written, which an attention call reads
  // after its own wait, so it may start now. (A grid that writes older rows is launched
  // without this, and followed by launch_fence.)
  if (p.single) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  const long f = (long)blockIdx.x * kThreads + threadIdx.x;
  const int j = (int)(f % L);
  const int slot = (int)(f / L % p.slots);
  const int token = (int)min(f / L / p.slots, (long)c.tokens);
  int first = 0, end = 0, bad = 0;
  const int b = token < c.tokens ? sequence_of(c, token, first, end) : -1;
  const long row = b >= 0 ? row_of(c, b, token, first, end, bad) : -1;

  // this thread's dims: 8 from `lo`, 8 from `hi`
  const int turning = p.rotary / 16;   // threads whose dims turn
  const bool turns = j < turning;
  const int rest = D - p.rotary;
  const int lo = turns ? 8 * j : p.rotary + 8 * (j - turning);
  const int hi = lo + (turns ? p.rotary / 2 : rest / 2);
  // their 8 pairs: rotate-halves takes dim lo + i with hi + i (pair lo + i), the adjacent
  // layout neighbouring dims (pairs lo / 2 .. and hi / 2 ..)
  float co[8], si[8];
  if (turns && b >= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = p.adjacent ? (i < 4 ? lo / 2 + i : hi / 2 + i - 4) : lo + i;
      const int a = min(max((int)__ldg(p.axis + pair), 0), p.axes - 1);
      int at = __ldcg(p.pos + (size_t)a * c.tokens + token);
      if (at < 0 || at >= p.positions) {
        bad |= kDevBadPosition;
        at = at < 0 ? 0 : p.positions - 1;
      }
      const float2 cs = __ldg(reinterpret_cast<const float2*>(p.cos_sin) + (size_t)at * (p.rotary / 2) + pair);
      co[i] = cs.x;
      si[i] = cs.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = 1.f, si[i] = 0.f;
  }

  const int Hq = p.q ? p.Hq : 0, heads = Hq + 2 * c.Hkv;
  const int page = 1 << c.log2_page;
#pragma unroll 2
  for (int h0 = 0; h0 < heads; h0 += p.slots) {   // the same number of turns for every thread
    const int h = h0 + slot;
    const bool is_q = h < Hq, is_v = h >= Hq + c.Hkv;
    const int hk = h - Hq - (is_v ? c.Hkv : 0);
    const bool on = b >= 0 && h < heads && (is_q || row >= 0);
    float x[8], y[8];
    if (on) {
      const char* src = (is_q   ? p.q + token * p.q_stride + (long)h * (D * E)
                         : is_v ? p.v + token * p.v_stride + (long)hk * (D * E)
                                : p.k + token * p.k_stride + (long)hk * (D * E));
      load8(src + lo * E, x, static_cast<const Q*>(nullptr));
      load8(src + hi * E, y, static_cast<const Q*>(nullptr));
      if (turns && !is_v) {
        if (p.adjacent) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = x[2 * i], a1 = x[2 * i + 1], b0 = y[2 * i], b1 = y[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a0, co[i]), __fmul_rn(a1, si[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(a1, co[i]), __fmul_rn(a0, si[i]));
            y[2 * i] = __fsub_rn(__fmul_rn(b0, co[4 + i]), __fmul_rn(b1, si[4 + i]));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(b1, co[4 + i]), __fmul_rn(b0, si[4 + i]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = x[i], e = y[i];
            x[i] = __fsub_rn(__fmul_rn(a, co[i]), __fmul_rn(e, si[i]));
            y[i] = __fadd_rn(__fmul_rn(e, co[i]), __fmul_rn(a, si[i]));
          }
        }
      }
      if (is_q) {
        char* dst = p.q_out + ((long)token * p.Hq + h) * (D * E);
        store8(dst + lo * E, x, static_cast<const Q*>(nullptr));
        store8(dst + hi * E, y, static_cast<const Q*>(nullptr));
      } else if constexpr (!Held<T>::kFp4) {
        char* dst = (is_v ? c.v : c.k) + (row + (long)hk * page) * (D * E);
        store8(dst + lo * E, x, static_cast<const Q*>(nullptr));
        store8(dst + hi * E, y, static_cast<const Q*>(nullptr));
      }
    }
    if constexpr (Held<T>::kFp4) {
      const bool mine = on && !is_q;
      if (__any_sync(0xffffffffu, mine)) {   // the lanes of a group agree; the shuffles need all
        if (!mine) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
        }
        const float gain = mine ? __ldcg((is_v ? c.v_gain : c.k_gain) + hk) : 1.f;
        uint32_t sx, sy;
        const uint32_t cx = pack_codes(x, gain, &sx), cy = pack_codes(y, gain, &sy);
        if (mine) {
          const long at = row + (long)hk * page;
          char* codes = (is_v ? c.v : c.k) + at * (D / 2);
          uint8_t* scales = (is_v ? c.v_scale : c.k_scale) + at * (D / 16);
          *reinterpret_cast<uint32_t*>(codes + lo / 2) = cx;
          *reinterpret_cast<uint32_t*>(codes + hi / 2) = cy;
          if ((lo & 15) == 0) {
            scales[lo / 16] = (uint8_t)sx;
            scales[hi / 16] = (uint8_t)sy;
          }
        }
      }
    }
  }
  if (bad) atomicOr(c.status, bad);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  constexpr int L = D / 16;
  const CacheRows& c = p.c;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const long f = (long)blockIdx.x * kThreads + threadIdx.x;
  const int j = (int)(f % L);
  const int h = (int)(f / L % c.Hkv);
  const long token_l = f / L / c.Hkv;
  if (token_l >= c.tokens) return;
  const int token = (int)token_l;
  int first = 0, end = 0, bad = 0;
  const int b = sequence_of(c, token, first, end);
  if (b < 0) return;   // behind the last sequence
  const long row = row_of(c, b, token, first, end, bad);
  const long at = row + ((long)h << c.log2_page);
  const long out = ((long)token * c.Hkv + h) * D + 16 * j;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (row >= 0) {
      if constexpr (Held<T>::kFp4) {
        const uint2 w = __ldcg(reinterpret_cast<const uint2*>((which ? c.v : c.k) + at * (D / 2)) + j);
        const float s = unpack_f16(e4m3_pair(__ldcg((which ? c.v_scale : c.k_scale) + at * (D / 16) + j))).x;
        const float gain = __ldcg((which ? c.v_gain : c.k_gain) + h);
        uint32_t v[8];
        fp4_decode8(w.x, v);
        fp4_decode8(w.y, v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = unpack_f16(v[i]);
          x[2 * i] = __fmul_rn(__fmul_rn(e.x, s), gain);
          x[2 * i + 1] = __fmul_rn(__fmul_rn(e.y, s), gain);
        }
      } else {
        const char* src = (which ? c.v : c.k) + (at * D + 16 * j) * (long)sizeof(T);
        load8(src, x, static_cast<const T*>(nullptr));
        load8(src + 8 * sizeof(T), x + 8, static_cast<const T*>(nullptr));
      }
    }
    char* dst = which ? p.v_out : p.k_out;
    if (p.out_f32) {
      store8(dst + out * 4, x, static_cast<const float*>(nullptr));
      store8(dst + out * 4 + 32, x + 8, static_cast<const float*>(nullptr));
    } else {
      store8(dst + out * 2, x, static_cast<const __nv_bfloat16*>(nullptr));
      store8(dst + out * 2 + 16, x + 8, static_cast<const __nv_bfloat16*>(nullptr));
    }
  }
  if (bad) atomicOr(c.status, bad);
}

__global__ void fence_kernel() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// With programmatic dependent launch: every kernel here begins with its wait.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), long threads, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(threads < kThreads ? 32 * (unsigned)((threads + 31) / 32) : kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D>
cudaError_t write_rows(const WriteParams& p, cudaStream_t s) {
  const cudaError_t e = launch_early(write_kernel<T, D>, (long)p.c.tokens * p.slots * (D / 16), s, p);
  return e != cudaSuccess || p.single ? e : launch_fence(s);
}

template <typename T, int D>
cudaError_t read_rows(const ReadParams& p, cudaStream_t s) {
  return launch_early(read_kernel<T, D>, (long)p.c.tokens * p.c.Hkv * (D / 16), s, p);
}

}  // namespace

cudaError_t launch_fence(cudaStream_t s) {
  return launch_early(fence_kernel, 1, s);
}

cudaError_t launch_write_rows(int dtype, int head_dim, int num_sms, WriteParams p, cudaStream_t s) {
  // as many threads as the SMs hold at a quarter of their registers, and no more slots than heads
  const long groups = (long)num_sms * 1024 / (head_dim / 16);
  const int heads = (p.q ? p.Hq : 0) + 2 * p.c.Hkv;
  long slots = (groups + p.c.tokens - 1) / p.c.tokens;
  p.slots = (int)(slots < 1 ? 1 : slots > heads ? heads : slots);
  switch (dtype) {
    case FASTOCR_DTYPE_BF16:
      return head_dim == 64 ? write_rows<__nv_bfloat16, 64>(p, s) : write_rows<__nv_bfloat16, 128>(p, s);
    case FASTOCR_DTYPE_F32: return head_dim == 64 ? write_rows<float, 64>(p, s) : write_rows<float, 128>(p, s);
  }
  return head_dim == 64 ? write_rows<Fp4, 64>(p, s) : write_rows<Fp4, 128>(p, s);
}

cudaError_t launch_read_rows(int dtype, int head_dim, const ReadParams& p, cudaStream_t s) {
  switch (dtype) {
    case FASTOCR_DTYPE_BF16:
      return head_dim == 64 ? read_rows<__nv_bfloat16, 64>(p, s) : read_rows<__nv_bfloat16, 128>(p, s);
    case FASTOCR_DTYPE_F32: return head_dim == 64 ? read_rows<float, 64>(p, s) : read_rows<float, 128>(p, s);
  }
  return head_dim == 64 ? read_rows<Fp4, 64>(p, s) : read_rows<Fp4, 128>(p, s);
}

}  // namespace fastocr
