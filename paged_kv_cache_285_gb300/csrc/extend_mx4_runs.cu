// Launches of the extend kernels over e2m1 codes in runs of key tiles, one per CTA,
// and the sum of the parts of items that more than one CTA took (a translation unit
// of their own).
#include "extend_kernel.cuh"

namespace pkv {

namespace {

constexpr int kMergeThreads = 256, kMergeCtas = 4;

// CTA c of the launch before took part k of an item with n parts: here it sums up rows
// k, k + n, .. of the item's 256 (over kMergeCtas CTAs), a thread 8 values of a row,
// O = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c.
template <int HD, int AT>
__global__ void __launch_bounds__(kMergeThreads) merge_runs_kernel(const ExtendParams p) {
  grid_dependency_wait();
  const int cta = blockIdx.x / kMergeCtas, quarter = blockIdx.x % kMergeCtas;
  const int4 of = *(p.run_of + 2 * cta), rows = *(p.run_of + 2 * cta + 1);
  const int parts = of.x, part = of.y, g = of.z;
  if (parts < 2) return;
  constexpr int UPR = HD / 8;
  const int u = threadIdx.x % UPR;
  // the slots of the item's parts: CTAs a head's width apart
  const int64_t slot0 = (int64_t)cta - (int64_t)part * p.num_kv_heads, width = p.num_kv_heads;
  constexpr int STEP = kMergeThreads / UPR;  // rows at a time
  for (int R = part + (quarter * STEP + (int)(threadIdx.x / UPR)) * parts; R < 2 * BM;
       R += kMergeCtas * STEP * parts) {
    const int x = R / BM, r = R % BM, rtok = r / p.group;
    if (rtok >= (x ? rows.z : rows.y)) continue;
    float m = -INFINITY, l = 0.f;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < parts; c0 += 2) {
      // two parts at a time, all loads before their use (the values of a part without a
      // key for the row are not used: its weights' sum is 0)
      float2 s[2];
      uint32_t v[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s[c] = make_float2(-INFINITY, 0.f);
        if (c0 + c < parts) {
          const int64_t at = (slot0 + (c0 + c) * width) * (2 * BM) + R;
          s[c] = p.run_ml[at];
          ld_global_v8(p.run_o + at * HD + 8 * u, v[c]);
        }
      }
      float top = m;
#pragma unroll
      for (int c = 0; c < 2; ++c) top = fmaxf(top, s[c].x);
      if (top > m) {  // (the first parts: sums are 0)
        const float f = m == -INFINITY ? 0.f : fast_exp2(m - top);
        if (l != 0.f) {
          l *= f;
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] *= f;
        }
        m = top;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!has_keys(s[c])) continue;
        const float w = fast_exp2(s[c].x - m);
        l += w * s[c].y;
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += w * __uint_as_float(v[c][q]);
      }
    }
    const int64_t row = (int64_t)(rows.x + x * p.tok + rtok) * p.num_q_heads + g * p.group + (r - rtok * p.group);
    const float f = p.out_scale / l;
    uint4 w4;
    w4.x = pack2<AT == DT_BF16>(o[0] * f, o[1] * f);
    w4.y = pack2<AT == DT_BF16>(o[2] * f, o[3] * f);
    w4.z = pack2<AT == DT_BF16>(o[4] * f, o[5] * f);
    w4.w = pack2<AT == DT_BF16>(o[6] * f, o[7] * f);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + row * HD + u * 8) = w4;
    if (p.lse_out && u == 0) p.lse_out[row] = (m + log2f(l)) * kLn2f;
  }
}

template <int HD, int AT, bool WIN>
cudaError_t launch_runs_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                          const CUtensorMap& omap, const ExtendParams& p, cudaStream_t stream) {
  auto k = extend_kernel<HD, DT_E2M1, AT, false, false, WIN, false, false, 3, false>;
  constexpr int smem = ExtCfg<HD, DT_E2M1, AT>::SMEM_RUN;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  const dim3 grid((unsigned)(p.runs * p.num_kv_heads));
  cudaLaunchConfig_t cfg = dependent_launch(grid, smem, stream, at, 1);
  const ExtendPartialParams pp{};
  if ((e = cudaLaunchKernelEx(&cfg, k, kmap, vmap, qmap, omap, p, pp)) != cudaSuccess) return e;
  cfg = dependent_launch(dim3(grid.x * kMergeCtas), 0, stream, at, 1);
  cfg.blockDim = dim3(kMergeThreads);
  return cudaLaunchKernelEx(&cfg, merge_runs_kernel<HD, AT>, p);
}

}  // namespace

cudaError_t launch_extend_mx4_runs(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   const CUtensorMap& qmap, const CUtensorMap& omap,
                                   const ExtendParams& p, int head_dim, int act_dt, cudaStream_t stream) {
  if (p.runs * p.num_kv_heads > kMaxRuns || p.num_items > p.runs * p.num_kv_heads || !p.run_o || !p.run_ml || !p.run_of)
    return cudaErrorInvalidValue;
#define PKV_EXT(HD, AT, WIN)                                   \
  if (head_dim == HD && act_dt == AT && (p.window > 0) == WIN) \
    return launch_runs_t<HD, AT, WIN>(kmap, vmap, qmap, omap, p, stream);
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
