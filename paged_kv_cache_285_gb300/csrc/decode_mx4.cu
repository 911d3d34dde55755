// Launches of the paged decode kernel (decode_kernel.cuh) over e2m1 codes with
// microscales, with and without a window.
#include "decode_kernel.cuh"

namespace pkv {

namespace {

template <int HD, int AT, bool WIN>
cudaError_t launch_mx4_t(const DecodeParams& p, const DecodeExtraParams& ap, cudaStream_t stream) {
  const CUtensorMap none{};  // (copied by each thread, without TMA)
  if (ap.join_cluster)
    return launch_decode_t<HD, DT_E2M1, AT, false, 0, kNW, WIN, false, true>(none, none, p, ap, stream);
  if (ap.two_warps)
    return launch_decode_t<HD, DT_E2M1, AT, false, 0, 2, WIN, false>(none, none, p, ap, stream);
  return launch_decode_t<HD, DT_E2M1, AT, false, 0, kNW, WIN, false>(none, none, p, ap, stream);
}

}  // namespace

cudaError_t launch_decode_mx4(const DecodeParams& p, const DecodeExtraParams& ap, int head_dim,
                              int act_dt, cudaStream_t stream) {
  if (ap.join_cluster && p.num_splits != 2 && p.num_splits != 4 && p.num_splits != 8)
    return cudaErrorInvalidValue;
#define PKV_MX4(HD, AT)                                                \
  if (head_dim == HD && act_dt == AT)                                  \
    return ap.window > 0 ? launch_mx4_t<HD, AT, true>(p, ap, stream)   \
                         : launch_mx4_t<HD, AT, false>(p, ap, stream);
  PKV_MX4(64, DT_F16)
  PKV_MX4(64, DT_BF16)
  PKV_MX4(128, DT_F16)
  PKV_MX4(128, DT_BF16)
#undef PKV_MX4
  return cudaErrorInvalidValue;
}

}  // namespace pkv
