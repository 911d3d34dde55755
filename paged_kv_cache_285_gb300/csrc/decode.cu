// Launches of the paged decode kernel (decode_kernel.cuh): plain decode and the
// own-token part of the shared-prefix decode.
#include "decode_kernel.cuh"

namespace pkv {

size_t decode_smem_bytes(int head_dim, int cache_dt) {
  switch (head_dim * 4 + cache_dt) {
    case 64 * 4 + DT_F16: return DecodeCfg<64, DT_F16, kNW, stages_for<64, DT_F16>()>::SMEM;
    case 64 * 4 + DT_BF16: return DecodeCfg<64, DT_BF16, kNW, stages_for<64, DT_BF16>()>::SMEM;
    case 64 * 4 + DT_E4M3: return DecodeCfg<64, DT_E4M3, kNW, stages_for<64, DT_E4M3>()>::SMEM;
    case 128 * 4 + DT_F16: return DecodeCfg<128, DT_F16, kNW, stages_for<128, DT_F16>()>::SMEM;
    case 128 * 4 + DT_BF16: return DecodeCfg<128, DT_BF16, kNW, stages_for<128, DT_BF16>()>::SMEM;
    case 128 * 4 + DT_E4M3: return DecodeCfg<128, DT_E4M3, kNW, stages_for<128, DT_E4M3>()>::SMEM;
    default: return 0;
  }
}

cudaError_t launch_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                          const DecodeExtraParams& ap, int head_dim, int cache_dt, int act_dt,
                          cudaStream_t stream) {
#define PKV_DEC(HD, CT, AT)                                              \
  if (head_dim == HD && cache_dt == CT && act_dt == AT)                  \
    return launch_decode_t<HD, CT, AT, false>(kmap, vmap, p, ap, stream);
  PKV_DEC(64, DT_F16, DT_F16)
  PKV_DEC(64, DT_BF16, DT_BF16)
  PKV_DEC(64, DT_E4M3, DT_F16)
  PKV_DEC(64, DT_E4M3, DT_BF16)
  PKV_DEC(128, DT_F16, DT_F16)
  PKV_DEC(128, DT_BF16, DT_BF16)
  PKV_DEC(128, DT_E4M3, DT_F16)
  PKV_DEC(128, DT_E4M3, DT_BF16)
#undef PKV_DEC
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_cascade(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const DecodeParams& p, const DecodeExtraParams& ap, int head_dim,
                                  int cache_dt, int act_dt, cudaStream_t stream,
                                  cudaEvent_t merge_after) {
  if (!ap.group_indptr || !ap.group_prefix_lens || ap.num_groups <= 0 || !p.ws_o)
    return cudaErrorInvalidValue;
  // Short runs per CTA (the members' own tokens are typically a few hundred):
  // small CTAs of two warps with two stages each (~33 KB at bf16 d128), so
  // that many fit on an SM and their fixed costs (setup, first copy,
  // epilogue) overlap.  Shared-prompt layer, 320 tokens per CTA: 50.5 us,
  // against 51.5 (2 warps, 1 stage), 53.1 (4 warps, 1 stage), 59.6 (4 warps,
  // 3 stages) and 65.5 (8 warps, 1 stage).  Long runs keep the plain decode's
  // configuration.
  const bool short_runs = p.chunk <= 512;
#define PKV_CASC(HD, CT, AT)                                                                   \
  if (head_dim == HD && cache_dt == CT && act_dt == AT)                                        \
    return short_runs                                                                          \
               ? launch_decode_t<HD, CT, AT, true, 2, 2>(kmap, vmap, p, ap, stream, merge_after) \
               : launch_decode_t<HD, CT, AT, true>(kmap, vmap, p, ap, stream, merge_after);
  PKV_CASC(64, DT_F16, DT_F16)
  PKV_CASC(64, DT_BF16, DT_BF16)
  PKV_CASC(64, DT_E4M3, DT_F16)
  PKV_CASC(64, DT_E4M3, DT_BF16)
  PKV_CASC(128, DT_F16, DT_F16)
  PKV_CASC(128, DT_BF16, DT_BF16)
  PKV_CASC(128, DT_E4M3, DT_F16)
  PKV_CASC(128, DT_E4M3, DT_BF16)
#undef PKV_CASC
  return cudaErrorInvalidValue;
}

}  // namespace pkv
