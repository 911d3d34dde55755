// Launches of the paged extend kernel (extend_kernel.cuh) over half tiles
// (requests of few rows), split over a cluster or not: calls with a window,
// block scales or both.
#include "extend_split.cuh"

namespace pkv {

cudaError_t launch_extend_half(const CUtensorMap& kmap, const CUtensorMap& vmap,
               const CUtensorMap& qmap, const CUtensorMap& omap, const ExtendParams& p,
               int head_dim, int cache_dt, int act_dt, cudaStream_t stream) {
  return launch_split<true>(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
}

}  // namespace pkv
