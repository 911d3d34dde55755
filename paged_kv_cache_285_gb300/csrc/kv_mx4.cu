// A cache of e2m1 codes with a power-of-two scale for every 32 values of a row
// (microscales): quantised as rows are written, and read back.
//
// Writing.  32 values x of a row (a token and kv head, K or V) are stored as
// codes e2m1(x / s), two to a byte, the first in its low bits, and a byte
// log2(s) + 127.  s is the smallest power of two, at least 2^-126, with
// |x| <= 7 s for the finite x.  e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4 and 6: a value
// in (6 s, 7 s] becomes 6 s, off by at most one s, which is the half step between
// 4 s and 6 s too, so no value is off by more than s; a limit of 6 s would double
// the step of the 31 others to spare the largest of them less than that.  x / s is
// exact, so a code carries one rounding (to nearest even).  Infinities become
// +-6 s; a NaN takes its 32 values with it (scale byte 255), since e2m1 has none.
// Rows do not share scales: a token is written, moved and dropped by itself.
//
// Append: one warp per page (block, kv head, K or V); a lane takes 16 values, two
// lanes a scale (one shuffle joins their largest magnitudes), so that a warp reads
// 1,024 consecutive bytes of rows at once and writes 256 of codes.  Bound by memory:
// 66,000 rows (8 kv heads of 128 dims) in 55 us and read back in 52, 329 MB each way
// counting codes, 91 % of the measured copy; one token for each of a few requests 2.5 us
// (a launch and four dependent loads).
#include <algorithm>

#include "pages.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Byte of the smallest power of two s >= 2^-126 with a <= 7 s = 1.75 2^2 s (a
// finite, >= 0): a = 1.m 2^e takes 2^(e-2), or 2^(e-1) if 1.m > 1.75.
__device__ __forceinline__ uint32_t microscale_byte(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 2 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}

// Eight values (four 16-bit pairs) times inv as e2m1 codes.  bf16: multiplied as
// they are (inv is a power of two: exact, and what underflows is 0 in e2m1 anyway).
template <int AT>
__device__ __forceinline__ uint32_t quantise8(const uint32_t* w, float inv) {
  float y[8];
  if constexpr (AT == DT_BF16) {
    const uint32_t i2 = __float_as_uint(inv) >> 16 | (__float_as_uint(inv) & 0xFFFF0000u);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t z = mul_bf16x2(w[q], i2);
      y[2 * q] = lo_f32<true>(z);
      y[2 * q + 1] = hi_f32<true>(z);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      y[2 * q] = bits_to_f32<AT>(w[q] & 0xFFFFu) * inv;
      y[2 * q + 1] = bits_to_f32<AT>(w[q] >> 16) * inv;
    }
  }
  return f32x8_to_e2m1x8(y);
}

template <int AT, int HD, int BS>
__global__ void __launch_bounds__(128) append_mx4_kernel(const AppendMx4Params p) {
  constexpr int VPR = HD / 16;          // vectors of 16 values per row
  constexpr int NV = BS * VPR / 32;     // per lane
  constexpr uint32_t kInf = AT == DT_BF16 ? 0x7F80u : 0x7C00u;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  PageTask t;
  // (the warp's number through a shuffle: known to be uniform, and the page with it; 53.4 -> 52.8 us)
  if (!find_page_task<BS>(p, blockIdx.x * 4u + __shfl_sync(kFull, threadIdx.x >> 5, 0), t)) return;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(t.isv ? p.v_new : p.k_new) + t.h * HD;
  const int64_t row_elems = (int64_t)p.num_kv_heads * HD;
  uint32_t x[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + 32 * i, row = v / VPR, col = (v % VPR) * 16;
#pragma unroll
    for (int q = 0; q < 8; ++q) x[i][q] = 0u;
    if (row >= t.start && row < t.end) {
      const uint16_t* at = src + (t.first_row + row) * row_elems + col;
      if (p.in_32b) {
        ld_global_v8(at, x[i]);
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(at), b = *(reinterpret_cast<const uint4*>(at) + 1);
        x[i][0] = a.x; x[i][1] = a.y; x[i][2] = a.z; x[i][3] = a.w;
        x[i][4] = b.x; x[i][5] = b.y; x[i][6] = b.z; x[i][7] = b.w;
      }
    }
  }
  const int64_t page = (int64_t)t.blk * p.num_kv_heads + t.h;
  uint2* codes = reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.isv ? p.v_cache : p.k_cache) +
                                          page * (BS * HD / 2));
  uint8_t* scales = (t.isv ? p.v_mx : p.k_mx) + page * (BS * HD / kMxGroup);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + 32 * i, row = v / VPR;
    // the largest finite magnitude of the 32 (two lanes'): 16-bit magnitudes order
    // as integers
    uint32_t m2 = 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q) m2 = max_u16x2(m2, x[i][q] & 0x7FFF7FFFu);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    const bool nan = m > kInf;
    if (__any_sync(kFull, m >= kInf)) {  // infinities or NaN: once more without those
      m = 0u;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t lo = x[i][q] & 0x7FFFu, hi = (x[i][q] >> 16) & 0x7FFFu;
        m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
      }
      m = max(m, __shfl_xor_sync(kFull, m, 1));
    }
    const uint32_t sb = microscale_byte(bits_to_f32<AT>(m));
    const float inv = __uint_as_float((254u - sb) << 23);  // 1 / s (sb is 1 .. 253)
    const uint2 c = make_uint2(quantise8<AT>(x[i], inv), quantise8<AT>(x[i] + 4, inv));
    if (row >= t.start && row < t.end) {
      codes[v] = c;
      if ((lane & 1) == 0) scales[v >> 1] = (uint8_t)(nan ? 255u : sb);
    }
  }
}

// ---- read back --------------------------------------------------------------
// As the read-back of the other caches: a CTA takes p.rows_per_cta rows, finds
// their slots, and streams vectors of 16 codes (8 bytes in, 32 out).
constexpr int kGatherRows = 256;

template <int AT, int HD>
__global__ void __launch_bounds__(256) gather_mx4_kernel(const GatherMx4Params p) {
  constexpr int VPR = HD / 16;            // vectors per (row, head)
  __shared__ int s_blk[kGatherRows];
  __shared__ int s_off[kGatherRows];
  grid_dependency_wait();
  const int64_t row0 = (int64_t)blockIdx.x * p.rows_per_cta;
  const int rows = (int)min((int64_t)p.rows_per_cta, p.total_rows - row0);
  if (threadIdx.x < rows) {
    int blk, off;
    find_row(p, row0 + threadIdx.x, blk, off);
    s_blk[threadIdx.x] = blk;
    s_off[threadIdx.x] = off;
  }
  __syncthreads();
  const int vecs = rows * p.num_kv_heads * VPR;
  constexpr int U = 4;  // vectors in flight per thread and tensor
  for (int base = threadIdx.x; base < vecs; base += 256 * U) {
    uint2 kx[U], vx[U];
    uint32_t kb[U], vb[U];
    int blk[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int u = base + e * 256;
      blk[e] = -2;
      kx[e] = vx[e] = make_uint2(0u, 0u);
      kb[e] = vb[e] = 127u;
      if (u < vecs) {
        const int rh = u / VPR, c = u % VPR;
        const int r = (int)p.div_hkv.div((uint32_t)rh);
        const int h = rh - r * p.num_kv_heads;
        blk[e] = s_blk[r];
        if (blk[e] >= 0) {
          const int64_t row = ((((int64_t)blk[e] * p.num_kv_heads + h) << p.bs_shift) + s_off[r]);
          kx[e] = *(static_cast<const uint2*>(p.k_cache) + row * VPR + c);
          vx[e] = *(static_cast<const uint2*>(p.v_cache) + row * VPR + c);
          kb[e] = *(p.k_mx + row * (HD / kMxGroup) + c / 2);
          vb[e] = *(p.v_mx + row * (HD / kMxGroup) + c / 2);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      if (blk[e] == -2) continue;
      const int64_t u = row0 * p.num_kv_heads * VPR + base + e * 256;
      uint32_t o[8];
      mx4_widen8<AT == DT_BF16>(kx[e].x, kb[e], o);
      mx4_widen8<AT == DT_BF16>(kx[e].y, kb[e], o + 4);
      store16(p.k_out, u, o, p.out_32b);
      mx4_widen8<AT == DT_BF16>(vx[e].x, vb[e], o);
      mx4_widen8<AT == DT_BF16>(vx[e].y, vb[e], o + 4);
      store16(p.v_out, u, o, p.out_32b);
    }
  }
}

}  // namespace

cudaError_t launch_append_mx4(const AppendMx4Params& in, int act_dt, int head_dim, int block_size,
                              cudaStream_t stream) {
  AppendMx4Params p = in;
  if (!plan_pages(p, block_size)) return cudaErrorInvalidValue;
  p.in_32b = (reinterpret_cast<uintptr_t>(p.k_new) % 32 == 0 &&
              reinterpret_cast<uintptr_t>(p.v_new) % 32 == 0) ? 1 : 0;
#define PKV_APP(AT, HD, BS)                                                                       \
  if (act_dt == AT && head_dim == HD && block_size == BS)                                         \
    return launch_dependent(append_mx4_kernel<AT, HD, BS>, (p.num_tasks + 3) / 4, 128, stream, p);
  PKV_APP(DT_F16, 64, 16)
  PKV_APP(DT_F16, 64, 32)
  PKV_APP(DT_F16, 128, 16)
  PKV_APP(DT_F16, 128, 32)
  PKV_APP(DT_BF16, 64, 16)
  PKV_APP(DT_BF16, 64, 32)
  PKV_APP(DT_BF16, 128, 16)
  PKV_APP(DT_BF16, 128, 32)
#undef PKV_APP
  return cudaErrorInvalidValue;
}

cudaError_t launch_gather_mx4(const GatherMx4Params& in, int act_dt, int head_dim, cudaStream_t stream) {
  GatherMx4Params p = in;
  p.div_hkv = make_fastdiv((uint32_t)p.num_kv_heads);
  p.out_32b = (reinterpret_cast<uintptr_t>(p.k_out) % 32 == 0 &&
               reinterpret_cast<uintptr_t>(p.v_out) % 32 == 0) ? 1 : 0;
  // about 1,024 vectors a CTA, fewer where the rows would not give every SM two
  // CTAs (as for the other caches)
  const int row_vecs = p.num_kv_heads * head_dim / 16;
  p.rows_per_cta = std::min(kGatherRows, std::max(1, 1024 / row_vecs));
  while (p.rows_per_cta > 8 && p.total_rows / p.rows_per_cta < 300) p.rows_per_cta /= 2;
  const int64_t ctas = (p.total_rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned n = (unsigned)ctas;
#define PKV_GAT(AT, HD)                 \
  if (act_dt == AT && head_dim == HD) return launch_dependent(gather_mx4_kernel<AT, HD>, n, 256, stream, p);
  PKV_GAT(DT_F16, 64)
  PKV_GAT(DT_F16, 128)
  PKV_GAT(DT_BF16, 64)
  PKV_GAT(DT_BF16, 128)
#undef PKV_GAT
  return cudaErrorInvalidValue;
}

}  // namespace pkv
