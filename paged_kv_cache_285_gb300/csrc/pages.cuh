// Where rows lie in the pages of a cache: the pages that a call's new rows touch
// (the appends that quantise take one warp per block, kv head, and K or V), and
// the page of a row that is read back.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

namespace {

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

// The launch of a kernel that begins with grid_dependency_wait(): it is set up
// while the launch before it in the stream still runs.  cluster > 1: CTAs per
// cluster.
template <typename P>
cudaError_t launch_dependent(void (*kern)(P), unsigned ctas, unsigned threads, cudaStream_t stream,
                             const P& p, unsigned cluster = 1) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
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
    const unsigned m = __ballot_sync(0xFFFFFFFFu, v <= u);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A warp's page and the new rows that go there.
struct PageTask {
  bool isv;
  int h, blk;
  int start, end;     // rows [start, end) of the page are new
  int64_t first_row;  // the new row of page row 0 (which may lie before the request's first)
};

// The page of warp-task `task`, or false: none, or nothing that may be written
// (reported once, by one lane of one of the request's tasks).
template <int BS>
__device__ __forceinline__ bool find_page_task(const AppendScaledParams& p, uint32_t task, PageTask& t) {
  const int lane = threadIdx.x & 31;
  if (task >= p.num_tasks) return false;
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
  if (r1 == r0) return false;
  const bool report = j == 0 && h == 0 && !isv && lane == 0;
  if (r0 < 0 || r1 < r0 || r1 > p.total_rows) {
    if (report) set_err(p.err, 3);
    return false;
  }
  int S = r1 - r0;
  if (j < 0 || j > (S >> p.bs_shift) + 2) return false;
  if (P < 0 || (int64_t)P + S > min((int64_t)p.max_blocks * BS, (int64_t)INT32_MAX - 128)) {
    if (report) set_err(p.err, 3);
    return false;
  }
  if (S > p.max_suffix_len) {
    if (report) set_err(p.err, 3);
    S = p.max_suffix_len;
  }
  const int lb = (P >> p.bs_shift) + j;                 // logical block
  const int start = max(P - lb * BS, 0);
  const int end = min(P + S - lb * BS, BS);
  if (end <= start) return false;  // (the last unit or two of a request may be empty)
  const int blk = *(p.block_tables + (int64_t)b * p.max_blocks + lb);
  if (blk < 0 || blk >= p.num_blocks) {
    if (h == 0 && !isv && lane == 0) set_err(p.err, 2);
    return false;
  }
  t.isv = isv;
  t.h = h;
  t.blk = blk;
  t.start = start;
  t.end = end;
  t.first_row = (int64_t)r0 + ((int64_t)lb * BS - P);
  return true;
}

// Candidates for touched blocks (units) of a launch, in its parameters.  Bounded
// by the length hint for every request (no search), or, when the requests'
// lengths differ so much that this would give more, by the rows (a search over
// q_indptr).  False where there are too many.
inline bool plan_pages(AppendScaledParams& p, int block_size) {
  p.bs_shift = block_size == 16 ? 4 : 5;
  const int64_t per_request = ((int64_t)p.max_suffix_len + 2 * block_size - 2) / block_size;
  const int64_t by_hint = per_request * p.batch;
  const int64_t by_rows = p.total_rows / block_size + 2 * (int64_t)p.batch;
  const bool direct = by_hint <= by_rows;
  const int64_t tasks = (direct ? by_hint : by_rows) * p.num_kv_heads * 2;
  if (tasks > INT32_MAX) return false;
  p.units_per_request = direct ? (int)per_request : 0;
  p.div_units = make_fastdiv((uint32_t)(p.units_per_request > 1 ? p.units_per_request : 1));
  p.div_hkv = make_fastdiv((uint32_t)p.num_kv_heads);
  p.num_tasks = (uint32_t)tasks;
  return true;
}

// The block and the offset in it of row t of a read-back: blk -1 where there is
// no such block (reported; the row becomes zeros), -2 where no request owns the
// row (before the first or after the last one's: left alone).
__device__ __forceinline__ void find_row(const GatherParams& p, int64_t t, int& blk, int& off) {
  int lo = 0, hi = p.batch;  // the request of row t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (*(p.row_indptr + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int64_t pos = (int64_t)*(p.start_positions + lo) + (t - *(p.row_indptr + lo));
  blk = -1;
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
  off = (int)(pos & ((1 << p.bs_shift) - 1));
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

}  // namespace

}  // namespace pkv
