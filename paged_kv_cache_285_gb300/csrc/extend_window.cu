// Launches of the paged extend kernel (extend_kernel.cuh) under a window with
// sink tokens.
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_window(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const CUtensorMap& qmap, const CUtensorMap& omap,
                                 const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                                 cudaStream_t stream) {
  const int checked_dt = cache_dt == DT_BF16_V16 ? DT_BF16 : cache_dt;
  if (!extend_supported(head_dim, checked_dt, act_dt, p.group)) return cudaErrorInvalidValue;
  if (p.num_items <= 0 || p.num_ctas <= 0 || p.tok != BM / p.group || p.window <= 0 ||
      p.sink_tokens < 0)
    return cudaErrorInvalidValue;
  const ExtendPartialParams pp{};
#define PKV_EXT(HD, CT, AT)                             \
  if (head_dim == HD && cache_dt == CT && act_dt == AT) \
    return launch_extend_t<HD, CT, AT, false, false, true>(kmap, vmap, qmap, omap, p, pp, stream);
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
