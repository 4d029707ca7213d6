// Parameters of the eviction kernel (evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fastocr {

// Rows of one (sequence, KV head) that a CTA of a cluster may own: their sort
// keys (32 bits) and their places in the hole / survivor list (16 bits) stay in
// its shared memory.
constexpr int kEvictSlice = 32768;
constexpr int kEvictCluster = 8;   // the portable cluster size

struct EvictParams {
  char* k;                     // [num_pages, H_kv, page_size, d]
  char* v;
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* seq_len;      // [B]
  int num_pages, max_pages, log2_page;
  int B, Hkv;
  int row_bytes;               // d * element size
  float* mass;                 // [B, H_kv, stride]
  int32_t* pos;                // [B, H_kv, stride]
  const int32_t* protect;      // [B]
  const int32_t* seen;         // [B]
  int stride;
  int budget, recent;
  int32_t* new_len;            // [B] or NULL
  int cluster;                 // CTAs of one (sequence, KV head)
  int slice;                   // rows a CTA's shared memory holds
  int32_t* status;
};

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s);
cudaError_t prepare_evict();

}  // namespace fastocr
