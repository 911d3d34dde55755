// The launch switch of the split extend kernels, for whole (HALF false) and half
// tiles: one translation unit each.
#pragma once
#include "extend_kernel.cuh"

namespace pkv {

template <bool HALF>
cudaError_t launch_split(const CUtensorMap& kmap, const CUtensorMap& vmap,
                           const CUtensorMap& qmap, const CUtensorMap& omap,
                           const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                           cudaStream_t stream) {
  if (!(p.splits == 1 || p.splits == 2 || p.splits == 4 || p.splits == 8) ||
      (int64_t)p.num_items * p.splits > INT32_MAX)
    return cudaErrorInvalidValue;
  const bool scaled = p.k_scales != nullptr, win = p.window > 0;
#define PKV_EXT(HD, CT, AT, WIN, BSC)                                                 \
  if (head_dim == HD && cache_dt == CT && act_dt == AT && win == WIN && scaled == BSC) \
    return launch_extend_split_t<HD, CT, AT, WIN, BSC, HALF>(kmap, vmap, qmap, omap, p, stream);
  PKV_EXT(128, DT_F16, DT_F16, true, false)
  PKV_EXT(128, DT_BF16, DT_BF16, true, false)
  PKV_EXT(128, DT_E4M3, DT_F16, true, false)
  PKV_EXT(128, DT_E4M3, DT_BF16, true, false)
  PKV_EXT(64, DT_F16, DT_F16, true, false)
  PKV_EXT(64, DT_BF16, DT_BF16, true, false)
  PKV_EXT(64, DT_E4M3, DT_F16, true, false)
  PKV_EXT(64, DT_E4M3, DT_BF16, true, false)
  PKV_EXT(128, DT_E4M3, DT_F16, true, true)
  PKV_EXT(128, DT_E4M3, DT_BF16, true, true)
  PKV_EXT(64, DT_E4M3, DT_F16, true, true)
  PKV_EXT(64, DT_E4M3, DT_BF16, true, true)
  PKV_EXT(128, DT_E4M3, DT_F16, false, true)
  PKV_EXT(128, DT_E4M3, DT_BF16, false, true)
  PKV_EXT(64, DT_E4M3, DT_F16, false, true)
  PKV_EXT(64, DT_E4M3, DT_BF16, false, true)
#undef PKV_EXT
  return cudaErrorInvalidValue;
}

}  // namespace pkv
