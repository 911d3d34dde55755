// Launches of the paged extend kernel (extend_kernel.cuh) under a window with
// sink tokens.
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_window(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const CUtensorMap& qmap, const CUtensorMap& omap,
                                 const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                                 cudaStream_t stream) {
#define PKV_EXT(HD, CT, AT)                             \
  if (head_dim == HD && cache_dt == CT && act_dt == AT) \
    return launch_extend_view_t<HD, CT, AT, true, false>(kmap, vmap, qmap, omap, p, stream);
  PKV_EXT(128, DT_BF16_V16, DT_BF16)
  PKV_EXT(64, DT_BF16_V16, DT_BF16)
  PKV_EXT(128, DT_F16, DT_F16)
  PKV_EXT(128, DT_BF16, DT_BF16)
  PKV_EXT(128, DT_E4M3, DT_F16)
  PKV_EXT(128, DT_E4M3, DT_BF16)
  PKV_EXT(64, DT_F16, DT_F16)
  PKV_EXT(64, DT_BF16, DT_BF16)
  PKV_EXT(64, DT_E4M3, DT_F16)
  PKV_EXT(64, DT_E4M3, DT_BF16)
#undef PKV_EXT
  return cudaErrorInvalidValue;
}

}  // namespace pkv
