// Launches of the paged extend kernel (extend_kernel.cuh) over fp8 codes with
// scales per block and kv head, and the choice among its instances for a call
// with a window, scales or both.
#include "extend_kernel.cuh"

namespace pkv {

namespace {

template <int HD, int AT>
cudaError_t launch_scaled_t(const CUtensorMap& kmap, const CUtensorMap& vmap,
                            const CUtensorMap& qmap, const CUtensorMap& omap,
                            const ExtendParams& p, cudaStream_t stream) {
  return p.window > 0 ? launch_extend_view_t<HD, DT_E4M3, AT, true, true>(kmap, vmap, qmap, omap, p, stream)
                      : launch_extend_view_t<HD, DT_E4M3, AT, false, true>(kmap, vmap, qmap, omap, p, stream);
}

// Pages widened beforehand, every key seen: K in the queries' type, V as f16.
template <int HD>
cudaError_t launch_widened_t(const CUtensorMap& kmap, const CUtensorMap& vmap,
                             const CUtensorMap& qmap, const CUtensorMap& omap,
                             const ExtendParams& p, int act_dt, cudaStream_t stream) {
  return act_dt == DT_BF16
             ? launch_extend_view_t<HD, DT_BF16_V16, DT_BF16, false, false>(kmap, vmap, qmap, omap, p, stream)
             : launch_extend_view_t<HD, DT_F16, DT_F16, false, false>(kmap, vmap, qmap, omap, p, stream);
}

}  // namespace

cudaError_t launch_extend_view(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const CUtensorMap& qmap, const CUtensorMap& omap,
                               const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                               cudaStream_t stream) {
  const int checked_dt = cache_dt == DT_BF16_V16 ? DT_BF16 : cache_dt;
  if (!extend_supported(head_dim, checked_dt, act_dt, p.group)) return cudaErrorInvalidValue;
  if (p.num_items <= 0 || p.num_ctas <= 0 || p.tok != BM / p.group || p.window < 0 ||
      p.sink_tokens < 0)
    return cudaErrorInvalidValue;
  if (p.k_scales && (!p.v_scales || cache_dt != DT_E4M3)) return cudaErrorInvalidValue;
  if (p.half) return launch_extend_half(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
  if (p.splits > 1)
    return launch_extend_split(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
  if (p.by_rows)
    return launch_extend_by_rows(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
  if (!p.k_scales) {
    if (p.window <= 0) {
      if (cache_dt != DT_BF16_V16 && cache_dt != DT_F16) return cudaErrorInvalidValue;
      return head_dim == 128 ? launch_widened_t<128>(kmap, vmap, qmap, omap, p, act_dt, stream)
                             : launch_widened_t<64>(kmap, vmap, qmap, omap, p, act_dt, stream);
    }
    return launch_extend_window(kmap, vmap, qmap, omap, p, head_dim, cache_dt, act_dt, stream);
  }
  if (head_dim == 128)
    return act_dt == DT_BF16 ? launch_scaled_t<128, DT_BF16>(kmap, vmap, qmap, omap, p, stream)
                             : launch_scaled_t<128, DT_F16>(kmap, vmap, qmap, omap, p, stream);
  return act_dt == DT_BF16 ? launch_scaled_t<64, DT_BF16>(kmap, vmap, qmap, omap, p, stream)
                           : launch_scaled_t<64, DT_F16>(kmap, vmap, qmap, omap, p, stream);
}

}  // namespace pkv
