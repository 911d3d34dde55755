// Launches of the paged decode kernel (decode_kernel.cuh) under a window with
// sink tokens, and over fp8 codes with scales per block and kv head.
#include "decode_kernel.cuh"

namespace pkv {

namespace {

template <int HD, int CT, int AT, bool WIN, bool BSC>
cudaError_t launch_view(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                        const DecodeExtraParams& ap, cudaStream_t stream) {
  if (ap.join_cluster)
    return launch_decode_t<HD, CT, AT, false, 0, kNW, WIN, BSC, true>(kmap, vmap, p, ap, stream);
  if (ap.two_warps)
    return launch_decode_t<HD, CT, AT, false, 0, 2, WIN, BSC>(kmap, vmap, p, ap, stream);
  return launch_decode_t<HD, CT, AT, false, 0, kNW, WIN, BSC>(kmap, vmap, p, ap, stream);
}

}  // namespace

cudaError_t launch_decode_window(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const DecodeParams& p, const DecodeExtraParams& ap, int head_dim,
                                 int cache_dt, int act_dt, cudaStream_t stream) {
  const bool scaled = ap.k_scales != nullptr;
  if (scaled && (!ap.v_scales || cache_dt != DT_E4M3)) return cudaErrorInvalidValue;
  if (!scaled && ap.window <= 0) return cudaErrorInvalidValue;
  if (ap.join_cluster && p.num_splits != 2 && p.num_splits != 4 && p.num_splits != 8)
    return cudaErrorInvalidValue;
#define PKV_WIN(HD, CT, AT)                                                              \
  if (head_dim == HD && cache_dt == CT && act_dt == AT && !scaled)                       \
    return launch_view<HD, CT, AT, true, false>(kmap, vmap, p, ap, stream);
#define PKV_BSC(HD, AT)                                                                  \
  if (head_dim == HD && act_dt == AT && scaled)                                          \
    return ap.window > 0                                                                 \
               ? launch_view<HD, DT_E4M3, AT, true, true>(kmap, vmap, p, ap, stream)     \
               : launch_view<HD, DT_E4M3, AT, false, true>(kmap, vmap, p, ap, stream);
  PKV_WIN(64, DT_F16, DT_F16)
  PKV_WIN(64, DT_BF16, DT_BF16)
  PKV_WIN(64, DT_E4M3, DT_F16)
  PKV_WIN(64, DT_E4M3, DT_BF16)
  PKV_WIN(128, DT_F16, DT_F16)
  PKV_WIN(128, DT_BF16, DT_BF16)
  PKV_WIN(128, DT_E4M3, DT_F16)
  PKV_WIN(128, DT_E4M3, DT_BF16)
  PKV_BSC(64, DT_F16)
  PKV_BSC(64, DT_BF16)
  PKV_BSC(128, DT_F16)
  PKV_BSC(128, DT_BF16)
#undef PKV_WIN
#undef PKV_BSC
  return cudaErrorInvalidValue;
}

}  // namespace pkv
