// Launches of the paged extend kernel (extend_kernel.cuh) with each item's key
// tiles split over a cluster: calls with a window,
// block scales or both.
#include "extend_split.cuh"

namespace pkv {

cudaError_t launch_extend_split(const CUtensorMap& kmap, const CUtensorMap& vmap,
               const CUtensorMap& qmap, const CUtensorMap& omap, const ExtendParams& p,
               int head_dim, int cache_dt, int act_dt, cudaStream_t stream) {
  return launch_split<false>(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
}

}  // namespace pkv
