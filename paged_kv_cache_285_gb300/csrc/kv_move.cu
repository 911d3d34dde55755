// Moving what a cache holds: copies of whole pages (a forked request's last
// page, a request moved to other pages) and tokens of a request moved together
// (kept after an eviction, or accepted out of a tree of drafts), in any number
// of pools of any type (K, V and scales of every layer) by one launch.
//
// Both are bound by memory: each byte is read once and written once.  Copies: 9,000
// pairs of 64 KB (K and V) 172 us, the measured copy's rate; 7 pages in each of 64
// pools, which L2 holds, 3.8 us.
#include <algorithm>

#include "pages.cuh"

namespace pkv {

namespace {

// ---- pages ------------------------------------------------------------------
// One CTA takes one piece of a pair's block in one pool: every thread has two
// vectors of 32 bytes in flight, four of 16 or eight of 4, as the pool's blocks allow.
constexpr int kCopyThreads = 256, kCopyUnroll = 2;
constexpr int kPieceBytes = kCopyThreads * kCopyUnroll * 32;

template <int VEC>
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, int64_t from, int64_t to) {
  constexpr int W = VEC / 4;
  constexpr int U = kPieceBytes / (kCopyThreads * VEC) < 8 ? kPieceBytes / (kCopyThreads * VEC) : 8;
  for (int64_t at0 = from + threadIdx.x * VEC; at0 < to; at0 += (int64_t)kCopyThreads * VEC * U) {
    uint32_t x[U][W];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int64_t at = at0 + e * (kCopyThreads * VEC);
      if (at < to) {
        if constexpr (VEC == 32) {
          ld_global_v8(src + at, x[e]);
        } else if constexpr (VEC == 16) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + at);
          x[e][0] = v.x; x[e][1] = v.y; x[e][2] = v.z; x[e][3] = v.w;
        } else {
          x[e][0] = *reinterpret_cast<const uint32_t*>(src + at);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int64_t at = at0 + e * (kCopyThreads * VEC);
      if (at < to) {
        if constexpr (VEC == 32) st_global_v8(dst + at, x[e]);
        else if constexpr (VEC == 16) *reinterpret_cast<uint4*>(dst + at) = make_uint4(x[e][0], x[e][1], x[e][2], x[e][3]);
        else *reinterpret_cast<uint32_t*>(dst + at) = x[e][0];
      }
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyBlocksParams p) {
  grid_dependency_wait();
  const uint32_t rest = p.div_pieces.div(blockIdx.x);
  const uint32_t piece = blockIdx.x - rest * p.div_pieces.d;
  const uint32_t pair = p.div_pools.div(rest);
  const uint32_t k = rest - pair * p.div_pools.d;
  const int src = *(p.src + pair), dst = *(p.dst + pair);
  if (src < 0 || dst < 0) return;  // no copy
  if (src >= p.num_blocks || dst >= p.num_blocks) {
    if (threadIdx.x == 0) set_err(p.err, 1);
    return;
  }
  if (src == dst) return;
  const int64_t bytes = p.pool[k].block_bytes;
  const int64_t from = (int64_t)piece * kPieceBytes;
  if (from >= bytes) return;  // (a pool of smaller blocks than the call's largest)
  const int64_t to = min(bytes, from + kPieceBytes);
  const uint8_t* s = p.pool[k].base + src * bytes;
  uint8_t* d = p.pool[k].base + dst * bytes;
  const uint64_t a = reinterpret_cast<uint64_t>(p.pool[k].base) | (uint64_t)bytes;
  if ((a & 31) == 0) copy_piece<32>(s, d, from, to);
  else if ((a & 15) == 0) copy_piece<16>(s, d, from, to);
  else copy_piece<4>(s, d, from, to);
}

// ---- tokens moved together ----------------------------------------------------
// Row i of request b goes from position src_positions[row_indptr[b] + i] to
// dst_starts[b] + i.  The sources rise and none lies before its destination, so
// rows may be moved in passes of rising i, in place: what a pass writes lies
// behind (or at) the sources of later passes only if those were read already.
// Within a pass every load precedes a barrier and every store follows it.
//
// A CTA (or a cluster of them) takes one (request, pool, run of kv heads), a pass
// `rows` rows of it per CTA (each thread up to four 16-byte vectors, few enough
// registers for two CTAs of 512 threads or four of 256 an SM).  While a pass's
// loads are under way its threads look up the next pass's rows, so that there is
// one barrier a pass.  32 layers x 8 requests of 4,000 of 8,000 tokens (8 heads x
// 128 dims, bf16, 8.4 GB): 1.27 ms, 97 % of the measured copy; 8 layers x 6 of 4,000
// to 16,000 (fp8, 1.8 GB) 295 us, 90 %, since the longest requests' CTAs end last;
// one layer of one request, 16,000 tokens, 52 us (clusters of 8; 235 without).
// A launch whose requests all pass at once (ONE) keeps no state for passes: 34 registers
// and six CTAs of 256 an SM; 1 to 6 rows of 16 requests in 64 pools 5.3 -> 4.6 us.
// Loads of the next pass ahead of a pass's stores took registers from CTAs (306 ->
// 444 us), eight vectors a thread too (332), pointers kept from load to store 317.
constexpr int kMoveUnroll = 4;

struct RowMove {
  int src_blk, dst_blk;  // src_blk < 0: not moved
  int off;               // source offset | destination offset << 8
};

__device__ __forceinline__ RowMove find_move(const CompactParams& p, int b, int r0, int i, int dst0,
                                             bool report) {
  RowMove m;
  m.src_blk = m.dst_blk = -1;
  m.off = 0;
  const int src = *(p.src_positions + r0 + i);
  const int before = i > 0 ? *(p.src_positions + r0 + i - 1) : -1;
  const int64_t dst = (int64_t)dst0 + i;
  const int64_t held = (int64_t)p.max_blocks << p.bs_shift;
  if (src <= before || src < dst || src >= held || dst < 0) {
    if (report) set_err(p.err, 3);
    return m;
  }
  if (src == dst) return m;
  const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
  const int sb = table[src >> p.bs_shift], db = table[dst >> p.bs_shift];
  if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
    if (report) set_err(p.err, 1);
    return m;
  }
  const int mask = (1 << p.bs_shift) - 1;
  m.src_blk = sb;
  m.dst_blk = db;
  m.off = (src & mask) | ((int)(dst & mask) << 8);
  return m;
}

template <int VEC> struct MoveVec;
template <> struct MoveVec<16> { using T = uint4; };
template <> struct MoveVec<8> { using T = uint2; };
template <> struct MoveVec<4> { using T = uint32_t; };
template <> struct MoveVec<2> { using T = uint16_t; };

template <int VEC, bool CL, int NT, bool ONE>
__device__ __forceinline__ void compact_rows(const CompactParams& p, const Pool& pool, int b, int r0,
                                             int n, int dst0, int h0, int heads, bool report,
                                             RowMove (*s_row)[NT]) {
  using T = typename MoveVec<VEC>::T;
  const int vpr = (int)pool.row_bytes / VEC;       // vectors per row and head, a power of two
  const int vpr_shift = 31 - __clz(vpr);
  const int vph = vpr * p.heads;                   // per row
  const int rows = max(1, min(NT, NT * kMoveUnroll / vph));  // per CTA and pass
  const int rank = CL ? (int)(blockIdx.x & ((1u << p.cluster_shift) - 1u)) : 0;
  const int step = CL ? rows << p.cluster_shift : rows, passes = n / step + (n % step != 0);
  const int vecs = rows * vph;  // at most what the threads hold (the launcher picks p.heads so)
  auto look_up = [&](int pass) {
    if ((int)threadIdx.x < rows) {
      const uint32_t i = (uint32_t)pass * step + rank * rows + threadIdx.x;  // (may pass 2^31)
      RowMove m;
      m.src_blk = -1;
      if (i < (uint32_t)n) m = find_move(p, b, r0, (int)i, dst0, report);
      s_row[pass % 3][threadIdx.x] = m;
    }
  };
  // the vector `at` of a pass: its row's move, and its place in a block's page of
  // the pool (beside the row's offset there)
  auto place = [&](int at, int pass, RowMove& m, int& h, int& c) -> bool {
    if (at >= vecs) return false;
    const int rh = at >> vpr_shift;
    const int r = (int)p.div_heads.div((uint32_t)rh);
    c = at & (vpr - 1);
    h = rh - r * p.heads;
    m = s_row[pass % 3][r];
    return m.src_blk >= 0 && h < heads;
  };
  auto address = [&](int blk, int off, int h, int c) -> T* {
    return reinterpret_cast<T*>(pool.base) +
           ((((int64_t)blk * p.num_kv_heads + (h0 + h)) << p.bs_shift) + off) * vpr + c;
  };
  look_up(0);
  __syncthreads();
  if constexpr (ONE) {  // the longest request passes at once
    T x[kMoveUnroll];
    T* to[kMoveUnroll];
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      RowMove m;
      int h, c;
      to[e] = nullptr;
      if (place(e * NT + (int)threadIdx.x, 0, m, h, c)) {
        x[e] = *address(m.src_blk, m.off & 255, h, c);
        to[e] = address(m.dst_blk, m.off >> 8, h, c);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e)
      if (to[e]) *to[e] = x[e];
    return;
  }
  for (int pass = 0; pass < passes; ++pass) {
    T x[kMoveUnroll];
    RowMove m;
    int h, c;
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e)
      if (place(e * NT + (int)threadIdx.x, pass, m, h, c)) x[e] = *address(m.src_blk, m.off & 255, h, c);
    if (pass + 1 < passes) look_up(pass + 1);
    if constexpr (CL) cluster_sync();
    else __syncthreads();
    // (the rows are looked at once more: s_row[pass % 3] stands until every thread
    // has been through two more barriers)
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e)
      if (place(e * NT + (int)threadIdx.x, pass, m, h, c)) *address(m.dst_blk, m.off >> 8, h, c) = x[e];
  }
}

// The request with the rank-th most rows, of up to 32 (the whole warp): a request's CTAs
// take the longer the more rows it has, and those that start last should be short.
// (A count that wraps, of an invalid row_indptr, still gives each its rank.)
__device__ __forceinline__ uint32_t by_length(const CompactParams& p, int rank) {
  const int lane = threadIdx.x & 31;
  uint32_t n = 0u;
  if (lane < p.batch) n = (uint32_t)*(p.row_indptr + lane + 1) - (uint32_t)*(p.row_indptr + lane);
  int above = 0;
  for (int l = 0; l < p.batch; ++l) {
    const uint32_t other = __shfl_sync(0xFFFFFFFFu, n, l);
    above += other > n || (other == n && l < lane);
  }
  return (uint32_t)(__ffs(__ballot_sync(0xFFFFFFFFu, lane < p.batch && above == rank)) - 1);
}

template <bool CL, int NT, bool ONE>
__global__ void __launch_bounds__(NT, ONE ? 6 : 0) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ RowMove s_row[ONE ? 1 : 3][NT];
  grid_dependency_wait();
  const uint32_t item = CL ? blockIdx.x >> p.cluster_shift : blockIdx.x;
  const uint32_t rest = p.div_groups.div(item);
  const int hg = (int)(item - rest * p.div_groups.d);
  uint32_t b = p.div_pools.div(rest);
  const int k = (int)(rest - b * p.div_pools.d);
  if (!CL && p.by_length) b = by_length(p, (int)b);
  const bool report = k == 0 && hg == 0;
  const int r0 = *(p.row_indptr + b), r1 = *(p.row_indptr + b + 1), dst0 = *(p.dst_starts + b);
  if (r0 == r1) return;  // (the same for every CTA of a cluster, as the returns below)
  if (r0 < 0 || r1 < r0 || r1 > p.total_rows || dst0 < 0) {
    if (report && threadIdx.x == 0) set_err(p.err, 3);
    return;
  }
  int n = r1 - r0;
  if (n > p.max_rows) {
    if (report && threadIdx.x == 0) set_err(p.err, 3);
    n = p.max_rows;
  }
  const int h0 = hg * p.heads, heads = min(p.heads, p.num_kv_heads - h0);
  const Pool& pool = p.pool[k];
  const uint64_t a = reinterpret_cast<uint64_t>(pool.base) | pool.row_bytes;
  if ((a & 15) == 0) compact_rows<16, CL, NT, ONE>(p, pool, b, r0, n, dst0, h0, heads, report, s_row);
  else if ((a & 7) == 0) compact_rows<8, CL, NT, ONE>(p, pool, b, r0, n, dst0, h0, heads, report, s_row);
  else if ((a & 3) == 0) compact_rows<4, CL, NT, ONE>(p, pool, b, r0, n, dst0, h0, heads, report, s_row);
  else compact_rows<2, CL, NT, ONE>(p, pool, b, r0, n, dst0, h0, heads, report, s_row);
}

template <int NT>
cudaError_t launch_compact_t(CompactParams& p, int vpr, int sm_count, cudaStream_t stream) {
  // Heads per CTA: as many as let the longest request pass at once (a request of
  // few rows then takes one CTA a pool), one where no number does.
  constexpr int kHold = NT * kMoveUnroll;
  const int64_t width = (int64_t)p.max_rows * vpr;
  p.heads = (int)std::max<int64_t>(1, std::min<int64_t>(p.num_kv_heads, kHold / width));
  p.head_groups = (p.num_kv_heads + p.heads - 1) / p.heads;
  p.div_heads = make_fastdiv((uint32_t)p.heads);
  p.div_groups = make_fastdiv((uint32_t)p.head_groups);
  p.div_pools = make_fastdiv((uint32_t)p.num_pools);
  const int64_t items = (int64_t)p.batch * p.num_pools * p.head_groups;
  // Clusters of up to 8 CTAs an item where the items alone leave SMs idle and
  // their rows take several passes.
  const int64_t passes = (width * p.heads + kHold - 1) / kHold;
  int shift = 0;
  while (shift < 3 && (items << shift) < sm_count && passes > (1 << shift)) ++shift;
  p.cluster_shift = shift;
  const int64_t ctas = items << shift;
  // longest requests first where CTAs start in several rounds (8 layers x 6 requests of
  // 4,000 to 16,000 tokens: 309 -> 295 us; one round of equal ones lost 1 us of 32)
  p.by_length = p.batch > 1 && p.batch <= 32 && passes > 1 && items > (int64_t)sm_count * (1024 / NT) ? 1 : 0;
  if (ctas <= 0 || ctas > INT32_MAX) return cudaErrorInvalidValue;
  if constexpr (NT == 256) {
    // (its rows found by a thread each)
    if (passes <= 1 && p.max_rows <= NT) return launch_dependent(compact_kernel<false, NT, true>, (unsigned)ctas, NT, stream, p);
  }
  return shift > 0 ? launch_dependent(compact_kernel<true, NT, false>, (unsigned)ctas, NT, stream, p, 1u << shift)
                   : launch_dependent(compact_kernel<false, NT, false>, (unsigned)ctas, NT, stream, p);
}

}  // namespace

cudaError_t launch_copy_blocks(CopyBlocksParams& p, int num_pairs, cudaStream_t stream) {
  int64_t most = 0;
  for (int k = 0; k < p.num_pools; ++k) most = std::max(most, p.pool[k].block_bytes);
  const int64_t pieces = (most + kPieceBytes - 1) / kPieceBytes;
  if (pieces * p.num_pools > INT32_MAX) return cudaErrorInvalidValue;
  p.pieces = (int)pieces;
  p.div_pieces = make_fastdiv((uint32_t)pieces);
  p.div_pools = make_fastdiv((uint32_t)p.num_pools);
  // as many pairs a launch as a grid holds
  const int most_pairs = (int)(INT32_MAX / (pieces * p.num_pools));
  for (int left = num_pairs; left > 0;) {
    const int n = std::min(left, most_pairs);
    const cudaError_t e =
        launch_dependent(copy_blocks_kernel, (unsigned)(pieces * p.num_pools * n), kCopyThreads, stream, p);
    if (e != cudaSuccess) return e;
    left -= n;
    p.src += n;
    p.dst += n;
  }
  return cudaSuccess;
}

cudaError_t launch_compact(CompactParams& p, int sm_count, cudaStream_t stream) {
  int vpr = 1;
  for (int k = 0; k < p.num_pools; ++k) vpr = std::max(vpr, (int)p.pool[k].row_bytes / 16);
  // CTAs of 512 threads from more than two passes of 256 on (64 requests of 100 rows
  // of 256 bytes, 4 layers, 56 -> 48 us with 256; 16 of 1,000, one layer, 39 -> 31
  // with 512)
  return (int64_t)p.max_rows * vpr > 2 * 256 * kMoveUnroll ? launch_compact_t<512>(p, vpr, sm_count, stream)
                                                        : launch_compact_t<256>(p, vpr, sm_count, stream);
}

}  // namespace pkv
