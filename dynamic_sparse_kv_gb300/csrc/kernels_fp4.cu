// Instances of the decode-attention kernel for a cache held in 4 bits (bf16 q and out).
#include "attend_impl.cuh"

namespace fastocr {

cudaError_t launch_fp4(int head_dim, int mode, const Params& p, cudaStream_t s) {
  switch (head_dim) {
    case 64: return dispatch_mode<Fp4, 64>(mode, p, s);
    case 128: return dispatch_mode<Fp4, 128>(mode, p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t prepare_fp4() {
  cudaError_t e = prepare_all_modes<Fp4, 64>();
  return e != cudaSuccess ? e : prepare_all_modes<Fp4, 128>();
}

int max_cluster_fp4(int head_dim, int variant) {
  return head_dim == 64 ? max_cluster_of<Fp4, 64>(variant) : max_cluster_of<Fp4, 128>(variant);
}

int active_clusters_fp4(int head_dim, int cluster) {
  return head_dim == 64 ? active_clusters<Fp4, 64>(cluster) : active_clusters<Fp4, 128>(cluster);
}

// the same with shared memory for one CTA an SM
int spread_clusters_fp4(int head_dim, int cluster) {
  constexpr int kMost = 227 * 1024;
  return head_dim == 64 ? active_clusters<Fp4, 64>(cluster, kMost) : active_clusters<Fp4, 128>(cluster, kMost);
}

}  // namespace fastocr
