// Launches of the paged extend kernel (extend_kernel.cuh): plain extend, the
// shared-prefix extend, the prefix pass of the shared-prefix decode, and the
// passes that widen a cache's pages into 16-bit pools.
#include <algorithm>

#include "extend_kernel.cuh"

namespace pkv {

bool extend_supported(int head_dim, int cache_dt, int act_dt, int group) {
  if (head_dim != 64 && head_dim != 128) return false;
  if (!(act_dt == DT_F16 || act_dt == DT_BF16)) return false;
  if (!(cache_dt == act_dt || cache_dt == DT_E4M3)) return false;
  return group >= 1 && group <= BM;
}

namespace {

template <bool PP, bool SX>
cudaError_t launch_extend_any(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                              const CUtensorMap& omap, const ExtendParams& p,
                              const ExtendPartialParams& pp, int head_dim, int cache_dt, int act_dt,
                              cudaStream_t stream) {
  // K bf16 with V widened to f16 beforehand is checked as a bf16 cache
  const int checked_dt = cache_dt == DT_BF16_V16 ? DT_BF16 : cache_dt;
  if (!extend_supported(head_dim, checked_dt, act_dt, p.group)) return cudaErrorInvalidValue;
  if (p.num_items <= 0 || p.num_ctas <= 0 || p.tok != BM / p.group) return cudaErrorInvalidValue;
#define PKV_EXT(HD, CT, AT)                                    \
  if (head_dim == HD && cache_dt == CT && act_dt == AT)        \
    return launch_extend_t<HD, CT, AT, PP, SX>(kmap, vmap, qmap, omap, p, pp, stream);
  if constexpr (!PP) {
    PKV_EXT(128, DT_BF16_V16, DT_BF16)
    PKV_EXT(64, DT_BF16_V16, DT_BF16)
  }
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

// Pages of a shared-prefix extend widened into 16-bit shadow pools with the
// cache's block ids, so that the extend kernel reads them without converting
// and its converter warps only zero the keys past a segment's end: a bf16
// cache's V pages to f16 (SRC = DT_BF16), or an fp8 cache's K pages to KOUT
// (the queries' type, so that S = Q K^T needs no query conversion) and V
// pages to f16 (SRC = DT_E4M3; every e4m3 value is exact in both).
// Request r (the k-th member of its group of n) widens its own blocks, from
// the group's shared prefix to its last key, and every n-th of the group's
// shared blocks from the k-th on (read through the group's first member's
// table), so a long shared prefix is spread over the members.  CTA (x, r)
// takes every gridDim.x-th block of r's list from the x-th.  bf16 -> f16
// rounds to nearest (+-inf beyond the f16 range) as the converter warps do.
template <int SRC, int OUT>
__device__ __forceinline__ void widen_block(const uint4* __restrict__ src, uint4* __restrict__ dst,
                                            int in_vec) {
  // in_vec 16-byte input vectors: bf16 -> one f16 vector each, e4m3 -> two
  for (int u0 = threadIdx.x; u0 < in_vec; u0 += 8 * 256) {
    uint4 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (u0 + e * 256 < in_vec) x[e] = __ldg(src + u0 + e * 256);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int u = u0 + e * 256;
      if (u < in_vec) {
        if constexpr (SRC == DT_BF16) {
          x[e].x = to_f16x2<true>(x[e].x);
          x[e].y = to_f16x2<true>(x[e].y);
          x[e].z = to_f16x2<true>(x[e].z);
          x[e].w = to_f16x2<true>(x[e].w);
          dst[u] = x[e];
        } else {
          uint4 lo, hi;
          widen16<OUT>(x[e], lo, hi);
          dst[2 * u] = lo;
          dst[2 * u + 1] = hi;
        }
      }
    }
  }
}

template <int SRC, int KOUT>
__global__ void __launch_bounds__(256) widen_kernel(const uint4* __restrict__ k,
                                                    const uint4* __restrict__ v,
                                                    uint4* __restrict__ k16, uint4* __restrict__ v16,
                                                    const ExtendParams p, int num_groups,
                                                    int in_vec) {
  const int r = blockIdx.y;
  if (r < __ldg(p.group_indptr) || r >= __ldg(p.group_indptr + num_groups)) return;
  int lo = 0, hi = num_groups;  // r's group: the last g with group_indptr[g] <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.group_indptr + mid) <= r) lo = mid;
    else hi = mid;
  }
  const int first = __ldg(p.group_indptr + lo);
  const int members = __ldg(p.group_indptr + lo + 1) - first, kk = r - first;
  const int total = __ldg(p.prefix_lens + r) + (__ldg(p.q_indptr + r + 1) - __ldg(p.q_indptr + r));
  const int nb = min(p.max_blocks, (max(total, 0) + (1 << p.bs_shift) - 1) >> p.bs_shift);
  const int ws = min(max(__ldg(p.group_shared + lo), 0) >> p.bs_shift, p.max_blocks);
  const int n_own = max(nb - ws, 0);
  const int n_shared = ws > kk ? (ws - kk + members - 1) / members : 0;
  const int out_vec = SRC == DT_BF16 ? in_vec : 2 * in_vec;
  for (int t = blockIdx.x; t < n_own + n_shared; t += gridDim.x) {
    const int row = t < n_own ? r : first;
    const int i = t < n_own ? ws + t : kk + (t - n_own) * members;
    const int blk = __ldg(p.block_tables + (int64_t)row * p.max_blocks + i);
    if (blk < 0 || blk >= p.num_blocks) continue;
    if constexpr (SRC == DT_E4M3)
      widen_block<SRC, KOUT>(k + (int64_t)blk * in_vec, k16 + (int64_t)blk * out_vec, in_vec);
    widen_block<SRC, DT_F16>(v + (int64_t)blk * in_vec, v16 + (int64_t)blk * out_vec, in_vec);
  }
}

// Plain extend: the pages each request reads (blocks 0 .. ceil((P + S) /
// block_size) - 1 of its table), widened once per block although requests
// may share blocks.  claims = [count][flag per block][list]: the claim pass
// gives thread (x, r, t) blocks 256 x + t, 256 (x + gridDim.x) + t, ... of
// request r; the first request to set a block's flag (zeroed before the pass)
// appends it to the list.  The widening pass then spreads the list over a
// grid of persistent CTAs, so that the blocks of a shared prefix, which the
// requests that start first win, do not queue up in those requests' CTAs.
__global__ void __launch_bounds__(256) claim_kernel(int* claims, const ExtendParams p) {
  const int r = blockIdx.y;
  const int total = __ldg(p.prefix_lens + r) + (__ldg(p.q_indptr + r + 1) - __ldg(p.q_indptr + r));
  const int nb = min(p.max_blocks, (max(total, 0) + (1 << p.bs_shift) - 1) >> p.bs_shift);
  const int w0 = p.window > 0 ? max(__ldg(p.prefix_lens + r), 0) - p.window + 1 : 0;
  // the grid is sized from the call's length hint; a request past it loops
  for (int base = blockIdx.x * 256; base < nb; base += gridDim.x * 256) {
    const int i = base + threadIdx.x;
    int blk = -1;
    // a block that a window hides from every row is not read
    const bool unseen = p.window > 0 && (i << p.bs_shift) >= p.sink_tokens &&
                        ((i + 1) << p.bs_shift) <= w0;
    if (i < nb && !unseen) blk = __ldg(p.block_tables + (int64_t)r * p.max_blocks + i);
    const bool won = blk >= 0 && blk < p.num_blocks && atomicCAS(claims + 1 + blk, 0, 1) == 0;
    // one list slot reservation per warp
    const unsigned m = __ballot_sync(0xffffffffu, won);
    if (m != 0) {
      const int lane = threadIdx.x & 31, leader = __ffs(m) - 1;
      int slot = 0;
      if (lane == leader) slot = atomicAdd(claims, __popc(m));
      slot = __shfl_sync(0xffffffffu, slot, leader);
      if (won) claims[1 + p.num_blocks + slot + __popc(m & ((1u << lane) - 1))] = blk;
    }
  }
}

// 16 codes -> 16 OUT values code * s.  OUT f16: finite values are kept inside
// its range (+-65504); bf16 and f16 round to nearest where code * s does not
// fit (powers of two as scales: exact but for f16's subnormals).
template <int OUT>
__device__ __forceinline__ uint32_t widen2_scaled(uint32_t two, float s) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  float a = lo_f32<false>(h) * s, b = hi_f32<false>(h) * s;
  if constexpr (OUT == DT_BF16) {
    return pack2<true>(a, b);
  } else {
    // (a NaN code stays NaN: the comparison is false)
    if (fabsf(a) > 65504.f) a = copysignf(65504.f, a);
    if (fabsf(b) > 65504.f) b = copysignf(65504.f, b);
    return pack2<false>(a, b);
  }
}

// One block's page [num_kv_heads][head_vec 16-code vectors] widened with a
// scale per head.
template <int OUT>
__device__ __forceinline__ void widen_block_scaled(const uint4* __restrict__ src,
                                                   uint4* __restrict__ dst,
                                                   const float* __restrict__ scales, int in_vec,
                                                   int head_shift) {
  for (int u0 = threadIdx.x; u0 < in_vec; u0 += 4 * 256) {
    uint4 x[4];
    float s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u0 + e * 256 < in_vec) {
        x[e] = __ldg(src + u0 + e * 256);
        s[e] = __ldg(scales + ((u0 + e * 256) >> head_shift));
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int u = u0 + e * 256;
      if (u < in_vec) {
        const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          o[2 * q] = widen2_scaled<OUT>(w[q] & 0xFFFFu, s[e]);
          o[2 * q + 1] = widen2_scaled<OUT>(w[q] >> 16, s[e]);
        }
        st_global_v8(dst + 2 * u, o);  // (the workspace is 256-byte aligned)
      }
    }
  }
}

template <int KOUT>
__global__ void __launch_bounds__(256) widen_scaled_list_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const float* __restrict__ k_scales,
    const float* __restrict__ v_scales, uint4* __restrict__ k16, uint4* __restrict__ v16,
    const int* __restrict__ claims, int num_blocks, int num_kv_heads, int in_vec, int head_shift) {
  const int n = min(claims[0], num_blocks);
  const int* list = claims + 1 + num_blocks;
  for (int j = blockIdx.x; j < n; j += gridDim.x) {
    const int blk = list[j];
    const int64_t at = (int64_t)blk * in_vec, sc = (int64_t)blk * num_kv_heads;
    widen_block_scaled<KOUT>(k + at, k16 + 2 * at, k_scales + sc, in_vec, head_shift);
    widen_block_scaled<DT_F16>(v + at, v16 + 2 * at, v_scales + sc, in_vec, head_shift);
  }
}

// One block's page of e2m1 codes (vectors of 16, two to a microscale) widened.
template <int OUT>
__device__ __forceinline__ void widen_block_mx4(const uint2* __restrict__ src, uint4* __restrict__ dst,
                                                const uint8_t* __restrict__ scales, int in_vec) {
  for (int u0 = threadIdx.x; u0 < in_vec; u0 += 4 * 256) {
    uint2 x[4];
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u0 + e * 256 < in_vec) {
        x[e] = __ldg(src + u0 + e * 256);
        b[e] = __ldg(scales + ((u0 + e * 256) >> 1));
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int u = u0 + e * 256;
      if (u < in_vec) {
        uint32_t o[8];
        mx4_widen8<OUT == DT_BF16>(x[e].x, b[e], o);
        mx4_widen8<OUT == DT_BF16>(x[e].y, b[e], o + 4);
        st_global_v8(dst + 2 * u, o);  // (the workspace is 256-byte aligned)
      }
    }
  }
}

template <int KOUT>
__global__ void __launch_bounds__(256) widen_mx4_list_kernel(
    const uint2* __restrict__ k, const uint2* __restrict__ v, const uint8_t* __restrict__ k_scales,
    const uint8_t* __restrict__ v_scales, uint4* __restrict__ k16, uint4* __restrict__ v16,
    const int* __restrict__ claims, int num_blocks, int in_vec) {
  const int n = min(claims[0], num_blocks);
  const int* list = claims + 1 + num_blocks;
  for (int j = blockIdx.x; j < n; j += gridDim.x) {
    const int64_t at = (int64_t)list[j] * in_vec;
    widen_block_mx4<KOUT>(k + at, k16 + 2 * at, k_scales + at / 2, in_vec);
    widen_block_mx4<DT_F16>(v + at, v16 + 2 * at, v_scales + at / 2, in_vec);
  }
}

template <int SRC, int KOUT>
__global__ void __launch_bounds__(256) widen_list_kernel(const uint4* __restrict__ k,
                                                         const uint4* __restrict__ v,
                                                         uint4* __restrict__ k16,
                                                         uint4* __restrict__ v16,
                                                         const int* __restrict__ claims,
                                                         int num_blocks, int in_vec) {
  const int n = min(claims[0], num_blocks);
  const int* list = claims + 1 + num_blocks;
  const int out_vec = SRC == DT_BF16 ? in_vec : 2 * in_vec;
  for (int j = blockIdx.x; j < n; j += gridDim.x) {
    const int blk = list[j];
    if constexpr (SRC == DT_E4M3)
      widen_block<SRC, KOUT>(k + (int64_t)blk * in_vec, k16 + (int64_t)blk * out_vec, in_vec);
    widen_block<SRC, DT_F16>(v + (int64_t)blk * in_vec, v16 + (int64_t)blk * out_vec, in_vec);
  }
}

}  // namespace

cudaError_t launch_widen_claim(int cache_dt, int act_dt, const void* k_cache,
                               const void* v_cache, void* k16, void* v16, int* claims,
                               const ExtendParams& p, int head_dim, int block_size,
                               int max_total_len, int sm_count, cudaStream_t stream) {
  if (!v_cache || !v16 || !claims || p.batch <= 0 || p.num_blocks <= 0 || sm_count <= 0)
    return cudaErrorInvalidValue;
  if (cache_dt != DT_BF16 && (cache_dt != DT_E4M3 || !k_cache || !k16)) return cudaErrorInvalidValue;
  const int elem = cache_dt == DT_BF16 ? 2 : 1;
  const int in_vec = p.num_kv_heads * block_size * head_dim * elem / 16;
  const int max_nb = std::min(p.max_blocks, (std::max(max_total_len, 1) + block_size - 1) / block_size);
  dim3 grid((unsigned)((max_nb + 255) / 256), (unsigned)p.batch);
  if (grid.y > 65535) return cudaErrorInvalidValue;
  cudaError_t e = cudaMemsetAsync(claims, 0, (size_t)(1 + p.num_blocks) * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  claim_kernel<<<grid, 256, 0, stream>>>(claims, p);
  // 8 CTAs of 256 threads fill an SM
  const int ctas = std::min(8 * sm_count, p.num_blocks);
  const uint4* k = static_cast<const uint4*>(k_cache);
  const uint4* v = static_cast<const uint4*>(v_cache);
  uint4* k16v = static_cast<uint4*>(k16);
  uint4* v16v = static_cast<uint4*>(v16);
  if (cache_dt == DT_BF16)
    widen_list_kernel<DT_BF16, DT_F16><<<ctas, 256, 0, stream>>>(k, v, k16v, v16v, claims,
                                                                   p.num_blocks, in_vec);
  else if (act_dt == DT_BF16)
    widen_list_kernel<DT_E4M3, DT_BF16><<<ctas, 256, 0, stream>>>(k, v, k16v, v16v, claims,
                                                                    p.num_blocks, in_vec);
  else
    widen_list_kernel<DT_E4M3, DT_F16><<<ctas, 256, 0, stream>>>(k, v, k16v, v16v, claims,
                                                                   p.num_blocks, in_vec);
  return cudaGetLastError();
}

cudaError_t launch_widen_scaled(int act_dt, const void* k_cache, const void* v_cache,
                                const float* k_scales, const float* v_scales, void* k16, void* v16,
                                int* claims, const ExtendParams& p, int head_dim, int block_size,
                                int max_total_len, int sm_count, cudaStream_t stream) {
  if (!k_cache || !v_cache || !k_scales || !v_scales || !k16 || !v16 || !claims || p.batch <= 0 ||
      p.num_blocks <= 0 || sm_count <= 0 || p.batch > 65535)
    return cudaErrorInvalidValue;
  const int head_vec = block_size * head_dim / 16;  // a power of two
  int head_shift = 0;
  while ((1 << head_shift) < head_vec) ++head_shift;
  const int in_vec = p.num_kv_heads * head_vec;
  const int max_nb = std::min(p.max_blocks, (std::max(max_total_len, 1) + block_size - 1) / block_size);
  cudaError_t e = cudaMemsetAsync(claims, 0, (size_t)(1 + p.num_blocks) * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  claim_kernel<<<dim3((unsigned)((max_nb + 255) / 256), (unsigned)p.batch), 256, 0, stream>>>(claims, p);
  const int ctas = std::min(8 * sm_count, p.num_blocks);
  const uint4* k = static_cast<const uint4*>(k_cache);
  const uint4* v = static_cast<const uint4*>(v_cache);
  uint4* k16v = static_cast<uint4*>(k16);
  uint4* v16v = static_cast<uint4*>(v16);
  if (act_dt == DT_BF16)
    widen_scaled_list_kernel<DT_BF16><<<ctas, 256, 0, stream>>>(
        k, v, k_scales, v_scales, k16v, v16v, claims, p.num_blocks, p.num_kv_heads, in_vec, head_shift);
  else
    widen_scaled_list_kernel<DT_F16><<<ctas, 256, 0, stream>>>(
        k, v, k_scales, v_scales, k16v, v16v, claims, p.num_blocks, p.num_kv_heads, in_vec, head_shift);
  return cudaGetLastError();
}

cudaError_t launch_widen_mx4(int act_dt, const void* k_cache, const void* v_cache,
                             const uint8_t* k_scales, const uint8_t* v_scales, void* k16, void* v16,
                             int* claims, const ExtendParams& p, int head_dim, int block_size,
                             int max_total_len, int sm_count, cudaStream_t stream) {
  if (!k_cache || !v_cache || !k_scales || !v_scales || !k16 || !v16 || !claims || p.batch <= 0 ||
      p.num_blocks <= 0 || sm_count <= 0 || p.batch > 65535)
    return cudaErrorInvalidValue;
  const int in_vec = p.num_kv_heads * block_size * head_dim / 16;
  const int max_nb = std::min(p.max_blocks, (std::max(max_total_len, 1) + block_size - 1) / block_size);
  cudaError_t e = cudaMemsetAsync(claims, 0, (size_t)(1 + p.num_blocks) * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  claim_kernel<<<dim3((unsigned)((max_nb + 255) / 256), (unsigned)p.batch), 256, 0, stream>>>(claims, p);
  const int ctas = std::min(8 * sm_count, p.num_blocks);
  const uint2* k = static_cast<const uint2*>(k_cache);
  const uint2* v = static_cast<const uint2*>(v_cache);
  uint4* k16v = static_cast<uint4*>(k16);
  uint4* v16v = static_cast<uint4*>(v16);
  if (act_dt == DT_BF16)
    widen_mx4_list_kernel<DT_BF16><<<ctas, 256, 0, stream>>>(k, v, k_scales, v_scales, k16v, v16v,
                                                              claims, p.num_blocks, in_vec);
  else
    widen_mx4_list_kernel<DT_F16><<<ctas, 256, 0, stream>>>(k, v, k_scales, v_scales, k16v, v16v,
                                                             claims, p.num_blocks, in_vec);
  return cudaGetLastError();
}

cudaError_t launch_widen(int cache_dt, int act_dt, const void* k_cache, const void* v_cache,
                         void* k16, void* v16, const ExtendParams& p, int num_groups, int head_dim,
                         int block_size, int max_total_len, cudaStream_t stream) {
  if (!v_cache || !v16 || !p.group_indptr || !p.group_shared || num_groups <= 0 || p.batch <= 0)
    return cudaErrorInvalidValue;
  if (cache_dt != DT_BF16 && (cache_dt != DT_E4M3 || !k_cache || !k16)) return cudaErrorInvalidValue;
  const int elem = cache_dt == DT_BF16 ? 2 : 1;
  const int in_vec = p.num_kv_heads * block_size * head_dim * elem / 16;
  // a request's list is at most its own blocks plus its share of the shared
  // ones, both bounded by its table; about 16 blocks per CTA at the hint's length
  const int max_nb = std::min(p.max_blocks, (std::max(max_total_len, 1) + block_size - 1) / block_size);
  dim3 grid((unsigned)std::max(1, std::min(8, (max_nb + 15) / 16)), (unsigned)p.batch);
  if (grid.y > 65535) return cudaErrorInvalidValue;
  const uint4* k = static_cast<const uint4*>(k_cache);
  const uint4* v = static_cast<const uint4*>(v_cache);
  uint4* k16v = static_cast<uint4*>(k16);
  uint4* v16v = static_cast<uint4*>(v16);
  if (cache_dt == DT_BF16)
    widen_kernel<DT_BF16, DT_F16><<<grid, 256, 0, stream>>>(k, v, k16v, v16v, p, num_groups, in_vec);
  else if (act_dt == DT_BF16)
    widen_kernel<DT_E4M3, DT_BF16><<<grid, 256, 0, stream>>>(k, v, k16v, v16v, p, num_groups, in_vec);
  else
    widen_kernel<DT_E4M3, DT_F16><<<grid, 256, 0, stream>>>(k, v, k16v, v16v, p, num_groups, in_vec);
  return cudaGetLastError();
}

cudaError_t launch_extend(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                          const CUtensorMap& omap, const ExtendParams& p, int head_dim,
                          int cache_dt, int act_dt, cudaStream_t stream) {
  return launch_extend_any<false, false>(kmap, vmap, qmap, omap, p, ExtendPartialParams{},
                                         head_dim, cache_dt, act_dt, stream);
}

cudaError_t launch_extend_shared(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const CUtensorMap& qmap, const CUtensorMap& omap,
                                 const ExtendParams& p, int head_dim, int cache_dt, int act_dt,
                                 cudaStream_t stream) {
  if (!p.group_indptr || !p.group_shared) return cudaErrorInvalidValue;
  return launch_extend_any<false, true>(kmap, vmap, qmap, omap, p, ExtendPartialParams{},
                                        head_dim, cache_dt, act_dt, stream);
}

cudaError_t launch_extend_prefix_pass(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                      const CUtensorMap& qmap, const ExtendParams& p,
                                      const ExtendPartialParams& pp, int head_dim, int cache_dt,
                                      int act_dt, cudaStream_t stream) {
  if (!pp.o || !pp.lse || p.out_tma) return cudaErrorInvalidValue;
  // the partials are stored by each thread: the output map is not read
  return launch_extend_any<true, false>(kmap, vmap, qmap, qmap, p, pp, head_dim, cache_dt, act_dt,
                                        stream);
}

}  // namespace pkv
