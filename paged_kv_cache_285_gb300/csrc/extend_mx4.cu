// Launches of the paged extend kernel (extend_kernel.cuh) over e2m1 codes with
// microscales, and the choice among its instances.
#include "extend_kernel.cuh"

namespace pkv {

cudaError_t launch_extend_mx4(const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const CUtensorMap& qmap, const CUtensorMap& omap, const ExtendParams& p,
                              int head_dim, int act_dt, cudaStream_t stream) {
  if (!extend_supported(head_dim, act_dt, act_dt, p.group)) return cudaErrorInvalidValue;
  if (p.num_items <= 0 || p.num_ctas <= 0 || p.tok != BM / p.group || p.window < 0 || p.sink_tokens < 0 ||
      !p.k_mx || !p.v_mx || p.k_scales)
    return cudaErrorInvalidValue;
  if (p.runs > 0) return launch_extend_mx4_runs(kmap, vmap, qmap, omap, p, head_dim, act_dt, stream);
  if (p.half) return launch_extend_mx4_half(kmap, vmap, qmap, omap, p, head_dim, act_dt, stream);
  if (p.splits > 1) return launch_extend_mx4_split(kmap, vmap, qmap, omap, p, head_dim, act_dt, stream);
  if (p.by_rows) return launch_extend_mx4_by_rows(kmap, vmap, qmap, omap, p, head_dim, act_dt, stream);
#define PKV_EXT(HD, AT, WIN)                                          \
  if (head_dim == HD && act_dt == AT && (p.window > 0) == WIN)        \
    return launch_extend_view_t<HD, DT_E2M1, AT, WIN, false>(kmap, vmap, qmap, omap, p, stream);
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
