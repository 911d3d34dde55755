// Launches of the extend kernels over e2m1 codes that take their items by rows (a
// translation unit of their own).
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_mx4_by_rows(const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const CUtensorMap& qmap, const CUtensorMap& omap,
                                      const ExtendParams& p, int head_dim, int act_dt, cudaStream_t stream) {
  const ExtendPartialParams pp{};
#define PKV_EXT(HD, AT, WIN)                                   \
  if (head_dim == HD && act_dt == AT && (p.window > 0) == WIN) \
    return launch_extend_t<HD, DT_E2M1, AT, false, false, WIN, false, 2>(kmap, vmap, qmap, omap, p, pp, stream);
  PKV_EXT(64, DT_F16, false)
  PKV_EXT(64, DT_F16, true)
  PKV_EXT(64, DT_BF16, false)
  PKV_EXT(64, DT_BF16, true)
  PKV_EXT(128, DT_F16, false)
  PKV_EXT(128, DT_F16, true)
  PKV_EXT(128, DT_BF16, false)
  PKV_EXT(128, DT_BF16, true)
#undef PKV_EXT
  return cudaErrorInvalidValue;
}

}  // namespace pkv
