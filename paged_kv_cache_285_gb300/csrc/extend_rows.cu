// Launches of the paged extend kernel (extend_kernel.cuh) for calls with a window
// and / or block scales whose blocks are counted by rows.
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_by_rows(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const CUtensorMap& qmap, const CUtensorMap& omap,
                                  const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                                  cudaStream_t stream) {
  const ExtendPartialParams pp{};
  const bool win = p.window > 0, scaled = p.k_scales != nullptr;
#define PKV_EXT(HD, CT, AT, WIN, BSC)                                                  \
  if (head_dim == HD && cache_dt == CT && act_dt == AT && win == WIN && scaled == BSC) \
    return launch_extend_t<HD, CT, AT, false, false, WIN, BSC, 2>(kmap, vmap, qmap, omap, p, pp, stream);
#define PKV_EXT_BOTH(CT, AT, WIN, BSC) \
  PKV_EXT(64, CT, AT, WIN, BSC)        \
  PKV_EXT(128, CT, AT, WIN, BSC)
  PKV_EXT_BOTH(DT_F16, DT_F16, true, false)
  PKV_EXT_BOTH(DT_BF16, DT_BF16, true, false)
  PKV_EXT_BOTH(DT_E4M3, DT_F16, true, false)
  PKV_EXT_BOTH(DT_E4M3, DT_BF16, true, false)
  PKV_EXT_BOTH(DT_BF16_V16, DT_BF16, true, false)
  PKV_EXT_BOTH(DT_F16, DT_F16, false, false)
  PKV_EXT_BOTH(DT_BF16_V16, DT_BF16, false, false)
  PKV_EXT_BOTH(DT_E4M3, DT_F16, true, true)
  PKV_EXT_BOTH(DT_E4M3, DT_BF16, true, true)
  PKV_EXT_BOTH(DT_E4M3, DT_F16, false, true)
  PKV_EXT_BOTH(DT_E4M3, DT_BF16, false, true)
#undef PKV_EXT_BOTH
#undef PKV_EXT
  return cudaErrorInvalidValue;
}

}  // namespace pkv
