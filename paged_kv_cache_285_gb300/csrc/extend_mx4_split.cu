// Launches of the extend kernels over e2m1 codes whose key tiles are
// split over clusters, in whole tiles (a translation unit of their own).
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_mx4_split(const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const CUtensorMap& qmap, const CUtensorMap& omap,
                                    const ExtendParams& p, int head_dim, int act_dt, cudaStream_t stream) {
  if (!(p.splits == 1 || p.splits == 2 || p.splits == 4 || p.splits == 8) ||
      (int64_t)p.num_items * p.splits > INT32_MAX)
    return cudaErrorInvalidValue;
#define PKV_EXT(HD, AT, WIN)                                   \
  if (head_dim == HD && act_dt == AT && (p.window > 0) == WIN) \
    return launch_extend_split_t<HD, DT_E2M1, AT, WIN, false, false>(kmap, vmap, qmap, omap, p, stream);
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
