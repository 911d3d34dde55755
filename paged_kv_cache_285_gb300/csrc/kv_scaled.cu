// A cache of e4m3 codes with one scale per block and kv head: quantised as it
// is written, and any cache read back into rows.
//
// Writing.  A (block, kv head) page X of at most block_size x head_dim values
// is stored as codes e4m3(x / s) and a scale s, for K and V apart.  s is the
// smallest power of two (at least 2^-126) with max |x| <= 448 s over the
// finite x:
//   * x / s is exact, so a code carries one rounding, the one to e4m3; and as
//     e4m3 is itself a floating-point format, a power of two costs none of its
//     relative precision (it moves the point where codes become subnormal by
//     at most one binary place);
//   * a page that is appended to later keeps its codes' values when its scale
//     has to grow: multiplying a code by a power of two is exact except where
//     it becomes subnormal.
// A page whose first tokens are kept (it holds positions before the request's
// new ones) takes the larger of its old scale (rounded up to a power of two)
// and the new tokens' one; when that is not the old one the kept codes are
// rewritten under it.  A page that starts with a new token takes the new
// tokens' scale whatever it held.
//
// Append: one warp per (block, kv head, K or V).  The page's new rows stay in
// registers between the pass for the maximum and the store of the codes, so
// every input is read once; there is no shared memory and no barrier.  Prompts
// are bound by memory: 63,600 rows of 8 heads x 128 dims (391 MB) in 59.8 us,
// 96 % of the measured copy; a step of one token per request by the launch and
// four dependent loads (lengths, block id, row, old scale): 2.4 us for 4
// requests (2.6 a call, which is the host's time for it).
//
// Both kernels are launched while the launch before them in the stream still
// runs and wait for its end before their first load: calls one after another
// 4.1 -> 2.6 us.  (All their loads are plain ones: read-only loads need not stay
// behind that wait.)
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void set_err(int32_t* err, int code) {
  if (err) atomicCAS(err, 0, code);
}

// max of the two 16-bit halves, unsigned
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int AT>
__device__ __forceinline__ float bits_to_f32(uint32_t b) {
  if constexpr (AT == DT_BF16) return __uint_as_float(b << 16);
  else return __half2float(__ushort_as_half((unsigned short)b));
}

// Bits of the smallest power of two s >= 2^-126 with a <= 448 s = 1.75 2^8 s
// (a finite, >= 0): a = 1.m 2^e takes 2^(e-8), or 2^(e-7) if 1.m > 1.75.
__device__ __forceinline__ uint32_t pow2_scale_bits(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1) << 23;
}

// The launch of a kernel that begins with grid_dependency_wait(): it is set up
// while the launch before it in the stream still runs.
template <typename P>
cudaError_t launch_dependent(void (*kern)(P), unsigned ctas, unsigned threads, cudaStream_t stream,
                             const P& p) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Four e4m3 codes times f (in fp32), as codes again (one rounding each).
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  const uint32_t h0 = e4m3x2_to_f16x2(c & 0xFFFFu), h1 = e4m3x2_to_f16x2(c >> 16);
  return f32x2_to_e4m3x2(lo_f32<false>(h0) * f, hi_f32<false>(h0) * f) |
         (f32x2_to_e4m3x2(lo_f32<false>(h1) * f, hi_f32<false>(h1) * f) << 16);
}

// The request whose units contain unit u: request b's start at
// q_indptr[b] / block_size + 2 b (it touches at most S / block_size + 2
// blocks).  The whole warp, 32 entries per round.
__device__ __forceinline__ int find_unit(const AppendScaledParams& p, int u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int idx = lo + lane * step;
    const int64_t v = idx < hi ? (int64_t)(*(p.q_indptr + idx) >> p.bs_shift) + 2 * (int64_t)idx
                               : INT64_MAX;
    const unsigned m = __ballot_sync(kFull, v <= u);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

template <int AT, int HD, int BS>
__global__ void __launch_bounds__(128) append_scaled_kernel(const AppendScaledParams p) {
  constexpr int VPR = HD / 8;           // 16-byte input vectors per row
  constexpr int NV = BS * VPR / 32;     // per lane
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * 4u + (threadIdx.x >> 5);
  if (task >= p.num_tasks) return;
  const bool isv = task & 1u;
  const uint32_t uh = task >> 1;
  const int unit = (int)p.div_hkv.div(uh);
  const int h = (int)(uh - (uint32_t)unit * p.div_hkv.d);
  // the unit's request and which of its touched blocks
  int b, j;
  if (p.units_per_request > 0) {
    b = (int)p.div_units.div((uint32_t)unit);
    j = unit - b * p.units_per_request;
  } else {
    if (unit < p.batch && h == 0 && !isv && lane == 0) {
      // where q_indptr falls, the search need not come to the request that does:
      // the first units (there are more than requests) look at its entries in order
      const int at = *(p.q_indptr + unit), next = *(p.q_indptr + unit + 1);
      if (at < 0 || next < at) set_err(p.err, 3);
    }
    b = find_unit(p, unit);
    j = unit - ((*(p.q_indptr + b) >> p.bs_shift) + 2 * b);
  }
  const int r0 = *(p.q_indptr + b), r1 = *(p.q_indptr + b + 1);
  const int P = *(p.prefix_lens + b);
  if (r1 == r0) return;
  const bool report = j == 0 && h == 0 && !isv && lane == 0;
  if (r0 < 0 || r1 < r0 || r1 > p.total_rows) {
    if (report) set_err(p.err, 3);
    return;
  }
  int S = r1 - r0;
  if (j < 0 || j > (S >> p.bs_shift) + 2) return;
  if (P < 0 || (int64_t)P + S > min((int64_t)p.max_blocks * BS, (int64_t)INT32_MAX - 128)) {
    if (report) set_err(p.err, 3);
    return;
  }
  if (S > p.max_suffix_len) {
    if (report) set_err(p.err, 3);
    S = p.max_suffix_len;
  }
  const int lb = (P >> p.bs_shift) + j;                 // logical block
  const int start = max(P - lb * BS, 0);                // rows [start, end) of the page are new
  const int end = min(P + S - lb * BS, BS);
  if (end <= start) return;  // (the last unit or two of a request may be empty)
  const int blk = *(p.block_tables + (int64_t)b * p.max_blocks + lb);
  if (blk < 0 || blk >= p.num_blocks) {
    if (h == 0 && !isv && lane == 0) set_err(p.err, 2);
    return;
  }
  const uint16_t* src = reinterpret_cast<const uint16_t*>(isv ? p.v_new : p.k_new) + h * HD;
  const int64_t row_elems = (int64_t)p.num_kv_heads * HD;
  const int64_t first_row = (int64_t)r0 + ((int64_t)lb * BS - P);  // new row of page row 0
  uint4 x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + 32 * i, row = v / VPR, col = (v % VPR) * 8;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= start && row < end)
      x[i] = *(reinterpret_cast<const uint4*>(src + (first_row + row) * row_elems + col));
  }
  const int64_t page = (int64_t)blk * p.num_kv_heads + h;
  float* scale_at = (isv ? p.v_scales : p.k_scales) + page;
  uint8_t* codes = static_cast<uint8_t*>(isv ? p.v_cache : p.k_cache) + page * (BS * HD);
  // the page's old scale, if it keeps tokens (start > 0 only in a request's first block)
  const float old = start > 0 ? *scale_at : 0.f;

  // ---- the largest finite magnitude: 16-bit magnitudes order as integers
  constexpr uint32_t kInf = AT == DT_BF16 ? 0x7F80u : 0x7C00u;
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    m2 = max_u16x2(m2, max_u16x2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu));
    m2 = max_u16x2(m2, max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
  }
  uint32_t m = __reduce_max_sync(kFull, max(m2 & 0xFFFFu, m2 >> 16));
  if (m >= kInf) {  // infinities or NaN among them: once more without those
    m = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = w[q] & 0x7FFFu, hi = (w[q] >> 16) & 0x7FFFu;
        m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
      }
    }
    m = __reduce_max_sync(kFull, m);
  }
  uint32_t sb = pow2_scale_bits(bits_to_f32<AT>(m));
  const uint32_t ob = __float_as_uint(old);
  bool rescale = false;
  if (old > 0.f) {  // (a NaN or negative old scale is not one: the new one stands)
    sb = max(sb, min((ob + 0x7FFFFFu) & 0xFF800000u, 0x7F000000u));
    rescale = sb != ob;
  }
  const float s = __uint_as_float(sb);
  const float inv = 1.f / s;  // exact

  // ---- kept codes under a larger scale
  if (rescale) {
    const float f = old * inv;
    for (int v = lane; v < start * (HD / 16); v += 32) {
      uint4* at = reinterpret_cast<uint4*>(codes) + v;
      uint4 c = *at;
      c.x = rescale4(c.x, f);
      c.y = rescale4(c.y, f);
      c.z = rescale4(c.z, f);
      c.w = rescale4(c.w, f);
      *at = c;
    }
  }
  // ---- the new codes
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + 32 * i, row = v / VPR;
    if (row >= start && row < end) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q >> 1] |= f32x2_to_e4m3x2(bits_to_f32<AT>(w[q] & 0xFFFFu) * inv,
                                     bits_to_f32<AT>(w[q] >> 16) * inv) << (16 * (q & 1));
      *reinterpret_cast<uint2*>(codes + v * 8) = make_uint2(o[0], o[1]);
    }
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale_at = s;
}

template <int AT, int HD, int BS>
cudaError_t launch_append_scaled_t(const AppendScaledParams& p, cudaStream_t stream) {
  return launch_dependent(append_scaled_kernel<AT, HD, BS>, (p.num_tasks + 3) / 4, 128, stream, p);
}

// ---- read back --------------------------------------------------------------
// Rows of requests out of their blocks: one CTA takes p.rows_per_cta rows;
// its first threads find each row's slot, then all threads stream the rows'
// vectors (16 codes, or 8 16-bit values), consecutive threads writing
// consecutive bytes: 16 values leave in one 32-byte store (two of 16 bytes, each
// half a sector, took 164 us where this takes 126: 832 MB at 97 % of the
// measured copy).
constexpr int kGatherRows = 256;  // at most, per CTA (one per thread)

template <int CT, int AT, bool BSC>
__device__ __forceinline__ void read16(const uint4& x, float s, uint32_t (&o)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t h = e4m3x2_to_f16x2(q & 1 ? w[q >> 1] >> 16 : w[q >> 1] & 0xFFFFu);
    float a = lo_f32<false>(h) * s, b = hi_f32<false>(h) * s;
    if constexpr (BSC && AT == DT_F16) {
      // a block's scale may put the code of a value near 65504 above it
      if (fabsf(a) > 65504.f) a = copysignf(65504.f, a);
      if (fabsf(b) > 65504.f) b = copysignf(65504.f, b);
    }
    o[q] = pack2<AT == DT_BF16>(a, b);
  }
}

// 16 values of a row, in one 32-byte store where the output is aligned to that.
__device__ __forceinline__ void store16(void* out, int64_t u, const uint32_t (&o)[8], bool aligned32) {
  uint4* at = static_cast<uint4*>(out) + 2 * u;
  if (aligned32) {
    st_global_v8(at, o);
  } else {
    at[0] = make_uint4(o[0], o[1], o[2], o[3]);
    at[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int CT, int AT, int HD, bool BSC>
__global__ void __launch_bounds__(256) gather_kernel(const GatherParams p) {
  constexpr int EPV = CT == DT_E4M3 ? 16 : 8;  // elements per vector
  constexpr int VPR = HD / EPV;                // vectors per (row, head)
  __shared__ int s_blk[kGatherRows];           // -1: no such block (zeros)
  __shared__ int s_off[kGatherRows];
  grid_dependency_wait();
  const int64_t row0 = (int64_t)blockIdx.x * p.rows_per_cta;
  const int rows = (int)min((int64_t)p.rows_per_cta, p.total_rows - row0);
  if (threadIdx.x < rows) {
    const int64_t t = row0 + threadIdx.x;
    int lo = 0, hi = p.batch;  // the request of row t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (*(p.row_indptr + mid) <= t) lo = mid;
      else hi = mid;
    }
    const int64_t pos = (int64_t)*(p.start_positions + lo) + (t - *(p.row_indptr + lo));
    int blk = -1;
    // rows that no request owns (before the first or after the last one's) are left alone
    if (t < *(p.row_indptr + lo) || t >= *(p.row_indptr + lo + 1)) {
      blk = -2;
    } else if (pos < 0 || (pos >> p.bs_shift) >= p.max_blocks) {
      set_err(p.err, 3);
    } else {
      blk = *(p.block_tables + (int64_t)lo * p.max_blocks + (pos >> p.bs_shift));
      if (blk < 0 || blk >= p.num_blocks) {
        set_err(p.err, 1);
        blk = -1;
      }
    }
    s_blk[threadIdx.x] = blk;
    s_off[threadIdx.x] = (int)(pos & ((1 << p.bs_shift) - 1));
  }
  __syncthreads();
  const int vecs = rows * p.num_kv_heads * VPR;
  constexpr int U = 4;  // vectors in flight per thread and tensor
  for (int base = threadIdx.x; base < vecs; base += 256 * U) {
    uint4 kx[U], vx[U];
    float ks[U], vs[U];
    int blk[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int u = base + e * 256;
      blk[e] = -2;
      kx[e] = vx[e] = make_uint4(0u, 0u, 0u, 0u);
      ks[e] = p.k_scale;
      vs[e] = p.v_scale;
      if (u < vecs) {
        const int rh = u / VPR, c = u % VPR;
        const int r = (int)p.div_hkv.div((uint32_t)rh);
        const int h = rh - r * p.num_kv_heads;
        blk[e] = s_blk[r];
        if (blk[e] >= 0) {
          const int64_t page = (int64_t)blk[e] * p.num_kv_heads + h;
          const int64_t at = ((page << p.bs_shift) + s_off[r]) * VPR + c;
          kx[e] = *(static_cast<const uint4*>(p.k_cache) + at);
          vx[e] = *(static_cast<const uint4*>(p.v_cache) + at);
          if constexpr (BSC) {
            ks[e] = *(p.k_scales + page);
            vs[e] = *(p.v_scales + page);
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      if (blk[e] == -2) continue;
      const int64_t u = row0 * p.num_kv_heads * VPR + base + e * 256;
      if constexpr (CT == DT_E4M3) {
        uint32_t o[8];
        read16<CT, AT, BSC>(kx[e], ks[e], o);
        store16(p.k_out, u, o, p.out_32b);
        read16<CT, AT, BSC>(vx[e], vs[e], o);
        store16(p.v_out, u, o, p.out_32b);
      } else {
        static_cast<uint4*>(p.k_out)[u] = kx[e];
        static_cast<uint4*>(p.v_out)[u] = vx[e];
      }
    }
  }
}

template <int CT, int AT, bool BSC>
cudaError_t launch_gather_t(const GatherParams& p, int head_dim, unsigned ctas, cudaStream_t stream) {
  return head_dim == 64 ? launch_dependent(gather_kernel<CT, AT, 64, BSC>, ctas, 256, stream, p)
                        : launch_dependent(gather_kernel<CT, AT, 128, BSC>, ctas, 256, stream, p);
}

}  // namespace

cudaError_t launch_append_scaled(const AppendScaledParams& in, int act_dt, int head_dim,
                                 int block_size, cudaStream_t stream) {
  AppendScaledParams p = in;
  p.bs_shift = block_size == 16 ? 4 : 5;
  // Units: candidates for touched blocks.  Bounded by the length hint for
  // every request (no search), or, when the requests' lengths differ so much
  // that this would give more, by the rows (a search over q_indptr).
  const int64_t per_request = ((int64_t)p.max_suffix_len + 2 * block_size - 2) / block_size;
  const int64_t by_hint = per_request * p.batch;
  const int64_t by_rows = p.total_rows / block_size + 2 * (int64_t)p.batch;
  const bool direct = by_hint <= by_rows;
  const int64_t tasks = std::min(by_hint, by_rows) * p.num_kv_heads * 2;
  if (tasks > INT32_MAX) return cudaErrorInvalidValue;
  p.units_per_request = direct ? (int)per_request : 0;
  p.div_units = make_fastdiv((uint32_t)std::max(p.units_per_request, 1));
  p.div_hkv = make_fastdiv((uint32_t)p.num_kv_heads);
  p.num_tasks = (uint32_t)tasks;
#define PKV_APP(AT, HD, BS)                                   \
  if (act_dt == AT && head_dim == HD && block_size == BS)     \
    return launch_append_scaled_t<AT, HD, BS>(p, stream);
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

cudaError_t launch_gather(const GatherParams& in, int cache_dt, int act_dt, int head_dim,
                          cudaStream_t stream) {
  GatherParams p = in;
  p.div_hkv = make_fastdiv((uint32_t)p.num_kv_heads);
  p.out_32b = (reinterpret_cast<uintptr_t>(p.k_out) % 32 == 0 &&
               reinterpret_cast<uintptr_t>(p.v_out) % 32 == 0) ? 1 : 0;
  // About 1,024 vectors a CTA (four per thread and tensor, in flight together):
  // 16 rows of 8 heads x 128 dims (8 rows: 146 us for 135,000 rows, 32: 127, 64:
  // 130), 256 rows of one head x 64 dims (64 rows: 18.8 us, 16: 43.6); fewer
  // where the rows would not give every SM two CTAs.
  const int row_vecs = p.num_kv_heads * head_dim / (cache_dt == DT_E4M3 ? 16 : 8);
  p.rows_per_cta = std::min(kGatherRows, std::max(1, 1024 / row_vecs));
  while (p.rows_per_cta > 8 && p.total_rows / p.rows_per_cta < 300) p.rows_per_cta /= 2;
  const int64_t ctas = (p.total_rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned n = (unsigned)ctas;
  if (cache_dt == DT_F16 && act_dt == DT_F16)
    return launch_gather_t<DT_F16, DT_F16, false>(p, head_dim, n, stream);
  if (cache_dt == DT_BF16 && act_dt == DT_BF16)
    return launch_gather_t<DT_BF16, DT_BF16, false>(p, head_dim, n, stream);
  if (cache_dt != DT_E4M3) return cudaErrorInvalidValue;
  const bool scaled = p.k_scales != nullptr;
  if (act_dt == DT_F16)
    return scaled ? launch_gather_t<DT_E4M3, DT_F16, true>(p, head_dim, n, stream)
                  : launch_gather_t<DT_E4M3, DT_F16, false>(p, head_dim, n, stream);
  if (act_dt == DT_BF16)
    return scaled ? launch_gather_t<DT_E4M3, DT_BF16, true>(p, head_dim, n, stream)
                  : launch_gather_t<DT_E4M3, DT_BF16, false>(p, head_dim, n, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
