// C ABI of libpkv.so: argument validation, split planning, TMA descriptors and
// launches.  Every check runs on the host before anything is enqueued.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "../../include/pkv.h"
#include "internal.h"

using namespace pkv;

// Device error word: first data error seen by any kernel (see pkv.h).
__device__ int32_t g_pkv_error_word = 0;

namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
  std::once_flag once;
  int sm_count = 0;
  int32_t* err = nullptr;
  cudaError_t init_error = cudaSuccess;
  // side stream of the shared-prefix decode, created on first use: its
  // prefix pass runs there, beside the decode of the members' own tokens on
  // the caller's stream (fork / join events order both against the caller's
  // stream; the mutex keeps concurrent callers' fork and join apart)
  std::once_flag side_once;
  std::mutex side_mu;
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  cudaError_t side_error = cudaSuccess;
};
DeviceState g_dev[kMaxDevices];

DeviceState* device_state(cudaError_t* e) {
  int dev = 0;
  *e = cudaGetDevice(&dev);
  if (*e != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= kMaxDevices) {
    *e = cudaErrorInvalidDevice;
    return nullptr;
  }
  DeviceState* s = &g_dev[dev];
  std::call_once(s->once, [s, dev]() {
    cudaError_t r = cudaDeviceGetAttribute(&s->sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (r == cudaSuccess) r = cudaGetSymbolAddress(reinterpret_cast<void**>(&s->err), g_pkv_error_word);
    s->init_error = r;
  });
  *e = s->init_error;
  return s->init_error == cudaSuccess ? s : nullptr;
}

cudaError_t side_stream(DeviceState* s) {
  std::call_once(s->side_once, [s]() {
    int least = 0, greatest = 0;
    cudaError_t r = cudaDeviceGetStreamPriorityRange(&least, &greatest);
    if (r == cudaSuccess) r = cudaStreamCreateWithPriority(&s->side, cudaStreamNonBlocking, greatest);
    if (r == cudaSuccess) r = cudaEventCreateWithFlags(&s->fork, cudaEventDisableTiming);
    if (r == cudaSuccess) r = cudaEventCreateWithFlags(&s->join, cudaEventDisableTiming);
    s->side_error = r;
  });
  return s->side_error;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, []() {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

int elem_bytes(pkv_dtype d) { return d == PKV_FP8_E4M3 ? 1 : 2; }

bool valid_dtype(pkv_dtype d) { return d == PKV_F16 || d == PKV_BF16 || d == PKV_FP8_E4M3; }

pkv_status check_desc(const pkv_cache_desc* d) {
  if (!d) return PKV_ERR_INVALID_ARG;
  if (d->num_blocks <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0 || d->block_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (!valid_dtype(d->cache_dtype)) return PKV_ERR_INVALID_ARG;
  if (!(d->head_dim == 64 || d->head_dim == 128)) return PKV_ERR_UNSUPPORTED;
  if (!(d->block_size == 16 || d->block_size == 32)) return PKV_ERR_UNSUPPORTED;
  if (d->cache_dtype == PKV_FP8_E4M3) {
    if (!(std::isfinite(d->k_scale) && d->k_scale > 0.f && std::isfinite(d->v_scale) &&
          d->v_scale > 0.f))
      return PKV_ERR_INVALID_ARG;
  }
  if ((int64_t)d->num_blocks * d->num_kv_heads > (int64_t)INT32_MAX) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

pkv_status check_act(const pkv_cache_desc* d, pkv_dtype act) {
  if (act != PKV_F16 && act != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (d->cache_dtype != PKV_FP8_E4M3 && d->cache_dtype != act) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// One 16-token tile of one kv head per TMA box row group:
// dims {head_dim, block_size, num_blocks*Hkv}, box {min(128B row) , 16, 1}.
pkv_status make_page_map(CUtensorMap* m, const void* base, const pkv_cache_desc* d) {
  auto enc = encode_fn();
  if (!enc) return PKV_ERR_CUDA;
  const int elem = elem_bytes(d->cache_dtype);
  const int rowb = d->head_dim * elem;
  const int chunkb = rowb < 128 ? rowb : 128;
  cuuint64_t dims[3] = {(cuuint64_t)d->head_dim, (cuuint64_t)d->block_size,
                        (cuuint64_t)d->num_blocks * (cuuint64_t)d->num_kv_heads};
  cuuint64_t strides[2] = {(cuuint64_t)rowb, (cuuint64_t)rowb * (cuuint64_t)d->block_size};
  cuuint32_t box[3] = {(cuuint32_t)(chunkb / elem), (cuuint32_t)kSubTokens, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUtensorMapDataType dt =
      elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const CUtensorMapSwizzle sw =
      chunkb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

// Query rows of the extend call as a 3-D map {head_dim, num_q_heads, rows}:
// one box {64, group, 128 / group} is the 64-dim column block of a row tile of
// (suffix token, head of the group) rows, 128-byte swizzled.
pkv_status make_q_map(CUtensorMap* m, const void* q, int head_dim, int num_q_heads,
                      int total_rows, int group) {
  auto enc = encode_fn();
  if (!enc) return PKV_ERR_CUDA;
  cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)num_q_heads, (cuuint64_t)total_rows};
  cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2u, (cuuint64_t)head_dim * 2u * (cuuint64_t)num_q_heads};
  cuuint32_t box[3] = {64u, (cuuint32_t)group, (cuuint32_t)(128 / group)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(q), dims, strides, box,
                   estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Work decomposition of an extend launch: rows of one (request, kv head) in
// tiles of `tok` suffix tokens x `group` heads, a work item = a pair of tiles,
// one persistent CTA per SM.  False if the item count overflows.
bool plan_extend(ExtendParams& p, int batch, int num_kv_heads, int group, int max_rows_per_request,
                 int sm_count) {
  p.group = group;
  p.tok = 128 / group;
  p.kchunks = 1;
  p.kchunk_keys = 0;
  p.tiles_per_head = ceil_div((int64_t)max_rows_per_request, p.tok);
  const int64_t pairs = (p.tiles_per_head + 1) / 2;
  const int64_t items = pairs * num_kv_heads * batch;
  if (items > INT32_MAX || pairs * num_kv_heads > UINT32_MAX / 2) return false;
  p.num_items = (int)items;
  p.div_pairs = make_fastdiv((uint32_t)pairs);
  p.div_hkv = make_fastdiv((uint32_t)num_kv_heads);
  p.div_req = make_fastdiv((uint32_t)(pairs * num_kv_heads));
  p.num_ctas = (int)std::min<int64_t>(items, sm_count > 0 ? sm_count : 1);
  return true;
}

// How an extend call with a window and / or block scales takes its items: in
// whole tiles or, where every request's rows fit one row tile, in half tiles; and
// with its key tiles split over a cluster of `splits` CTAs when the items are too
// few to fill the GPU.  The estimate, in us, at 128 dims: a key tile costs 1.80
// (half tiles: 1.43), a CTA a fixed part of 5.5, or 9.5 where parts are combined
// (clusters and half tiles); 152 SMs hold 152, 152, 144 and 120 CTAs in clusters
// of 1, 2, 4 and 8.  Measured (us at 1 / 2 / 4 / 8 CTAs): whole tiles, 64 items of
// 254 tiles 458 / 259 / 278 / 365, 128 of up to 21 tiles 43 / 53 / 62 / 107, 8 of
// 63 tiles 115 / 66 / 39 / 25; the last in half tiles 100 / 55 / 33 / 22.5, and
// 512 of 1 to 4 tiles 44 whole, 56 in half tiles.  (Two of these at each end
// again with launches set up early: 257, 44; the order is the same.)
void plan_view_items(ExtendParams& p, int max_total_len, int sm_count) {
  int64_t tiles = ((int64_t)max_total_len + 127) / 128;
  if (p.window > 0)
    tiles = std::min<int64_t>(tiles, ((int64_t)p.window + 2 * p.tok + 15 + 127) / 128 + 1 +
                                         ((int64_t)p.sink_tokens + 127) / 128);
  const double sms = sm_count > 0 ? sm_count : 152;
  double best = 1e30;
  for (int half = 0; half <= (p.tiles_per_head <= 1 ? 1 : 0); ++half) {
    for (int c = 1; c <= 8; c *= 2) {
      if ((int64_t)p.num_items * c > INT32_MAX || (c > 1 && tiles < c)) break;
      const double slots = c == 8 ? sms * 120 / 152 : c == 4 ? sms * 144 / 152 : sms;
      const double cost = std::ceil(p.num_items * c / slots) *
                          ((double)((tiles + c - 1) / c) * (half ? 1.43 : 1.80) +
                           (c > 1 || half ? 9.5 : 5.5));
      if (cost < 0.93 * best) {  // (not for less than a few per cent)
        best = cost;
        p.splits = c;
        p.half = half;
      }
    }
  }
}

// Softmax scale in base 2 with an fp8 cache's k_scale folded in (scores are
// computed on the codes), and the output scale (v_scale for fp8, else 1).
float score_scale_log2(const pkv_cache_desc* d, float sm_scale) {
  const double kscale = d->cache_dtype == PKV_FP8_E4M3 ? (double)d->k_scale : 1.0;
  return (float)((double)sm_scale * kscale * 1.4426950408889634);
}
float output_scale(const pkv_cache_desc* d) {
  return d->cache_dtype == PKV_FP8_E4M3 ? d->v_scale : 1.0f;
}

struct DecodePlan {
  int chunk = 0;
  int splits = 0;
  size_t ws_bytes = 0;
  size_t ws_lse_offset = 0;
  size_t ws_span_offset = 0;  // cascade: int2 (first own token, length) per request
  bool cluster = false;       // window / block-scaled: the splits form clusters, no workspace
  int num_cuts = 0;           // window / block-scaled: splits of different lengths
  int cut[kMaxCuts + 1] = {};
};

// The workspace of a plan's partials: O and LSE per (request, head, split).
void size_partials(DecodePlan& pl, const pkv_cache_desc* d, int batch, int hq) {
  const size_t o_bytes = (size_t)batch * hq * pl.splits * d->head_dim * sizeof(float);
  pl.ws_lse_offset = (o_bytes + 255) & ~(size_t)255;
  pl.ws_bytes = pl.ws_lse_offset + (size_t)batch * hq * pl.splits * sizeof(float);
}

// Split plan: the sequence is cut into runs of `chunk` tokens (a multiple of
// 16).  Automatic: aim for about six waves of two CTAs per SM over the worst
// case batch*Hkv*max_seq_len, runs between 128 and 4096 tokens.
DecodePlan plan_decode(const pkv_cache_desc* d, int batch, int hq, int max_seq_len,
                       int forced, int sm_count) {
  DecodePlan pl;
  const int max_sub = max_seq_len > 0 ? ceil_div(max_seq_len, kSubTokens) : 1;
  int chunk_sub;
  if (forced > 0) {
    chunk_sub = ceil_div(max_sub, forced);
  } else {
    const int64_t work = (int64_t)max_sub * batch * d->num_kv_heads;
    const int64_t target = 6LL * 2LL * (sm_count > 0 ? sm_count : 148);
    chunk_sub = ceil_div(work, target);
    if (chunk_sub < 8) chunk_sub = 8;
    if (chunk_sub > 256) chunk_sub = 256;
  }
  if (chunk_sub < 1) chunk_sub = 1;
  pl.chunk = chunk_sub * kSubTokens;
  pl.splits = ceil_div(max_sub, chunk_sub);
  if (pl.splits < 1) pl.splits = 1;
  if (pl.splits > 1) size_partials(pl, d, batch, hq);
  return pl;
}

}  // namespace

extern "C" {

pkv_status pkv_chain_hash(const int32_t* tokens, const int32_t* token_indptr, int32_t batch,
                          int32_t block_size, const uint64_t* salts, uint64_t* hashes,
                          int32_t max_blocks, cudaStream_t stream) {
  if (batch < 0 || block_size <= 0 || block_size > 4096 || max_blocks < 0) return PKV_ERR_INVALID_ARG;
  if (batch == 0 || max_blocks == 0) return PKV_OK;
  if (!tokens || !token_indptr || !hashes) return PKV_ERR_INVALID_ARG;
  if (!aligned(hashes, 8) || (salts && !aligned(salts, 8)) || !aligned(tokens, 4))
    return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  ChainHashParams p;
  p.tokens = tokens;
  p.token_indptr = token_indptr;
  p.salts = salts;
  p.hashes = hashes;
  p.err = ds->err;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  e = launch_chain_hash(p, batch, stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

const char* pkv_status_string(pkv_status s) {
  switch (s) {
    case PKV_OK: return "PKV_OK";
    case PKV_ERR_INVALID_ARG: return "PKV_ERR_INVALID_ARG";
    case PKV_ERR_UNSUPPORTED: return "PKV_ERR_UNSUPPORTED";
    case PKV_ERR_WORKSPACE: return "PKV_ERR_WORKSPACE";
    case PKV_ERR_CUDA: return "PKV_ERR_CUDA";
    case PKV_ERR_NO_SPACE: return "PKV_ERR_NO_SPACE";
    default: return "PKV_ERR_UNKNOWN";
  }
}

int32_t pkv_version(void) { return 20100; }

pkv_status pkv_get_device_error(int32_t* word, int32_t clear, cudaStream_t stream) {
  if (!word) return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  int32_t host = 0;
  if (cudaMemcpyAsync(&host, ds->err, sizeof(int32_t), cudaMemcpyDeviceToHost, stream) != cudaSuccess)
    return PKV_ERR_CUDA;
  if (clear && cudaMemsetAsync(ds->err, 0, sizeof(int32_t), stream) != cudaSuccess)
    return PKV_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return PKV_ERR_CUDA;
  *word = host;
  return PKV_OK;
}

pkv_status pkv_kv_append(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                         const void* k_new, const void* v_new, pkv_dtype act_dtype,
                         const int64_t* slot_mapping, int32_t num_tokens, cudaStream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!k_cache || !v_cache || !k_new || !v_new || !slot_mapping) return PKV_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
    return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  AppendParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_new = k_new;
  p.v_new = v_new;
  p.slots = slot_mapping;
  p.err = ds->err;
  p.num_tokens = num_tokens;
  p.num_kv_heads = desc->num_kv_heads;
  p.head_dim = desc->head_dim;
  p.block_size = desc->block_size;
  p.num_blocks = desc->num_blocks;
  p.k_scale = desc->k_scale;
  p.v_scale = desc->v_scale;
  e = launch_append(p, (int)desc->cache_dtype, (int)act_dtype, stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t pkv_decode_workspace_bytes(const pkv_cache_desc* desc, int32_t batch, int32_t num_q_heads,
                                  int32_t max_seq_len, int32_t num_splits) {
  if (check_desc(desc) != PKV_OK || batch <= 0 || num_q_heads <= 0 || max_seq_len < 0 ||
      num_splits < 0)
    return 0;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  const int sms = ds ? ds->sm_count : 0;
  return plan_decode(desc, batch, num_q_heads, max_seq_len, num_splits, sms).ws_bytes;
}

}  // extern "C"

// Plan of a shared-prefix decode: the decode split plan over the requests'
// own tokens, plus workspace slots for the shared prefix's partials (one per
// key chunk, at most kMaxPrefixChunks, chunks of at least kMinPrefixChunk keys)
// per (request, head), always merged.
constexpr int kMaxPrefixChunks = 8;
constexpr int kMinPrefixChunk = 256;
int prefix_slots_for(int max_prefix_len) {
  const int by_len = ceil_div(std::max(max_prefix_len, 1), kMinPrefixChunk);
  return std::min(kMaxPrefixChunks, std::max(1, by_len));
}
static DecodePlan plan_cascade(const pkv_cache_desc* d, int batch, int hq, int max_prefix_len,
                               int max_suffix_len, int forced, int sm_count) {
  // a member's own tokens start at its group's prefix rounded down to whole
  // blocks: up to block_size - 1 more than seq_len - prefix
  DecodePlan pl = plan_decode(d, batch, hq, max_suffix_len + d->block_size - 1, forced, sm_count);
  const size_t slots = (size_t)pl.splits + prefix_slots_for(max_prefix_len);
  pl.ws_lse_offset = align256((size_t)batch * hq * slots * d->head_dim * sizeof(float));
  pl.ws_span_offset = align256(pl.ws_lse_offset + (size_t)batch * hq * slots * sizeof(float));
  pl.ws_bytes = pl.ws_span_offset + (size_t)batch * 2 * sizeof(int32_t);
  return pl;
}

extern "C" {

size_t pkv_shared_prefix_decode_workspace_bytes(const pkv_cache_desc* desc, int32_t batch,
                                                int32_t num_q_heads, int32_t max_prefix_len,
                                                int32_t max_suffix_len, int32_t num_splits) {
  if (check_desc(desc) != PKV_OK || batch <= 0 || num_q_heads <= 0 || max_prefix_len < 0 ||
      max_suffix_len < 0 || num_splits < 0)
    return 0;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  const int sms = ds ? ds->sm_count : 0;
  return plan_cascade(desc, batch, num_q_heads, max_prefix_len, max_suffix_len, num_splits, sms)
      .ws_bytes;
}

pkv_status pkv_paged_decode_attn_shared_prefix(
    const pkv_cache_desc* desc, void* k_cache, void* v_cache, const void* k_new, const void* v_new,
    const void* q, void* out, pkv_dtype act_dtype, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
    float sm_scale, const int32_t* group_indptr, const int32_t* group_prefix_lens,
    int32_t num_groups, int32_t max_group_size, int32_t max_prefix_len, int32_t max_suffix_len,
    int32_t num_splits, float* lse_out, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (batch < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || num_groups < 0 ||
      max_group_size < 0 || max_prefix_len < 0 || max_suffix_len < 0 || num_splits < 0 ||
      !std::isfinite(sm_scale) || !(sm_scale > 0.f))
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int group = num_q_heads / desc->num_kv_heads;
  if (!extend_supported(desc->head_dim, (int)desc->cache_dtype, (int)act_dtype, group))
    return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (num_groups == 0 || max_group_size == 0) return PKV_ERR_INVALID_ARG;
  if (batch > 65535 || desc->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !q || !out || !block_tables || !seq_lens || !group_indptr ||
      !group_prefix_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 2))
    return PKV_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return PKV_ERR_INVALID_ARG;
  if (k_new && (!aligned(k_new, 16) || !aligned(v_new, 16))) return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  const DecodePlan pl = plan_cascade(desc, batch, num_q_heads, max_prefix_len, max_suffix_len,
                                     num_splits, ds->sm_count);
  if (!workspace || workspace_bytes < pl.ws_bytes || !aligned(workspace, 256))
    return PKV_ERR_WORKSPACE;
  if (pl.splits > 65535) return PKV_ERR_UNSUPPORTED;
  CUtensorMap kmap, vmap, qmap;
  if ((st = make_page_map(&kmap, k_cache, desc)) != PKV_OK) return st;
  if ((st = make_page_map(&vmap, v_cache, desc)) != PKV_OK) return st;
  if ((st = make_q_map(&qmap, q, desc->head_dim, num_q_heads, batch, group)) != PKV_OK) return st;
  float* ws_o = reinterpret_cast<float*>(workspace);
  float* ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.ws_lse_offset);
  const int prefix_slots = prefix_slots_for(max_prefix_len);
  const int slots = pl.splits + prefix_slots;
  const float scale_log2 = score_scale_log2(desc, sm_scale);

  // 1. the shared prefixes, once per group, on the tensor cores -> one
  //    partial per key chunk in the first prefix_slots slots (on the side
  //    stream, beside step 2)
  ExtendParams pe{};
  pe.q_indptr = group_indptr;
  pe.prefix_lens = group_prefix_lens;
  pe.block_tables = block_tables;
  pe.q = q;
  pe.out = nullptr;
  pe.lse_out = nullptr;
  pe.err = ds->err;
  pe.max_blocks = max_blocks_per_seq;
  pe.num_blocks = desc->num_blocks;
  pe.batch = num_groups;
  pe.num_q_heads = num_q_heads;
  pe.num_kv_heads = desc->num_kv_heads;
  pe.out_32b = 0;
  pe.bs_shift = desc->block_size == 16 ? 4 : 5;
  pe.total_rows = batch;
  pe.scale_log2 = scale_log2;
  pe.out_scale = output_scale(desc);
  if (!plan_extend(pe, num_groups, desc->num_kv_heads, group, max_group_size, ds->sm_count))
    return PKV_ERR_UNSUPPORTED;
  // The prefix's keys in chunks of whole key tiles when the groups give few
  // work items: the pass runs beside the own-token decode and should take
  // about a quarter of the SMs (measured on the shared-prompt layer: 32 items
  // of 8 key tiles beside the decode, 55 us per call; 128 items of 2 tiles run
  // before it, 75 us).  Each chunk's partial is one more term of the LSE
  // merge; at most prefix_slots chunks.
  const int key_tiles = std::max(1, ceil_div(max_prefix_len, 128));
  const int quarter = std::max(1, (ds->sm_count > 0 ? ds->sm_count : 4) / 4);
  const int want = std::max(1, quarter / pe.num_items);
  const int chunk_tiles = ceil_div(key_tiles, std::min(std::min(want, prefix_slots), key_tiles));
  pe.kchunks = ceil_div(key_tiles, chunk_tiles);
  pe.kchunk_keys = chunk_tiles * 128;
  {
    const int64_t items = (int64_t)pe.num_items * pe.kchunks;
    const uint32_t pairs = (uint32_t)((pe.tiles_per_head + 1) / 2);
    if (items > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    pe.num_items = (int)items;
    pe.div_pairs = make_fastdiv(pairs * (uint32_t)pe.kchunks);
    pe.div_req = make_fastdiv(pairs * (uint32_t)pe.kchunks * (uint32_t)desc->num_kv_heads);
    pe.num_ctas = (int)std::min<int64_t>(items, ds->sm_count > 0 ? ds->sm_count : 1);
  }
  ExtendPartialParams pp{};
  pp.o = ws_o;
  pp.lse = ws_lse;
  pp.o_stride = (int64_t)slots * desc->head_dim;
  pp.lse_stride = slots;
  if (side_stream(ds) != cudaSuccess) return PKV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(ds->side_mu);
  e = cudaEventRecord(ds->fork, stream);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  e = cudaStreamWaitEvent(ds->side, ds->fork, 0);
  if (e == cudaSuccess)
    e = launch_extend_prefix_pass(kmap, vmap, qmap, pe, pp, desc->head_dim,
                                  (int)desc->cache_dtype, (int)act_dtype, ds->side);
  // join even after a failure, so that the caller's stream (or a capture in
  // progress) never keeps the side stream forked
  const cudaError_t ej = cudaEventRecord(ds->join, ds->side);
  if (e != cudaSuccess || ej != cudaSuccess) {
    cudaStreamWaitEvent(stream, ds->join, 0);
    return PKV_ERR_CUDA;
  }

  // 2. each request's own tokens (current token appended first) -> the slots
  //    after the prefix's, then, once the prefix pass has joined, the merge
  //    of all of them
  DecodeParams p;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.q = q;
  p.out = out;
  p.lse_out = lse_out;
  p.ws_o = ws_o;
  p.ws_lse = ws_lse;
  p.err = ds->err;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = desc->num_blocks;
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = desc->num_kv_heads;
  p.group = group;
  p.bs_shift = desc->block_size == 16 ? 4 : 5;
  p.chunk = pl.chunk;
  p.num_splits = pl.splits;
  p.scale_log2 = scale_log2;
  p.out_scale = output_scale(desc);
  DecodeExtraParams ap{};
  ap.k_new = k_new;
  ap.v_new = v_new;
  ap.k_cache = k_cache;
  ap.v_cache = v_cache;
  ap.k_scale = desc->k_scale;
  ap.v_scale = desc->v_scale;
  ap.k_rcp = (float)(1.0 / (double)desc->k_scale);
  ap.v_rcp = (float)(1.0 / (double)desc->v_scale);
  ap.group_indptr = group_indptr;
  ap.group_prefix_lens = group_prefix_lens;
  ap.num_groups = num_groups;
  ap.ws_span = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + pl.ws_span_offset);
  ap.prefix_slots = prefix_slots;
  ap.prefix_chunk = pe.kchunk_keys;
  ap.prefix_chunks = pe.kchunks;
  e = launch_decode_cascade(kmap, vmap, p, ap, desc->head_dim, (int)desc->cache_dtype,
                            (int)act_dtype, stream, ds->join);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// What a decode or extend call sees: scales per block and kv head (null:
// none), and a window with sink tokens (window 0: every token).
struct AttnView {
  const float* k_scales;
  const float* v_scales;
  int32_t window;
  int32_t sink_tokens;
};

static pkv_status check_view(const pkv_cache_desc* desc, const AttnView& w, bool scaled) {
  if (w.window < 0 || w.sink_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (!scaled) return PKV_OK;
  if (desc->cache_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}
static pkv_status check_scales(const float* k_scales, const float* v_scales) {
  if (!k_scales || !v_scales || !aligned(k_scales, 4) || !aligned(v_scales, 4))
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

// The desc of a block-scaled cache: its per-tensor scales are not used.
static pkv_cache_desc scaled_desc(const pkv_cache_desc* desc) {
  pkv_cache_desc d = *desc;
  d.k_scale = d.v_scale = 1.f;
  return d;
}

// Most tokens that the decode kernel goes over for a query that sees
// max_seq_len tokens under a window: whole 16-token tiles of the sinks and of
// the window (which may begin and end inside a tile).
static int visible_bound(int max_seq_len, int window, int sink_tokens) {
  if (window <= 0) return max_seq_len;
  const int64_t tiles = ((int64_t)window + kSubTokens - 1) / kSubTokens + 1 +
                        ((int64_t)sink_tokens + kSubTokens - 1) / kSubTokens;
  return (int)std::min<int64_t>(max_seq_len, tiles * kSubTokens);
}

// Split plan of a decode call through a view, from what a CTA and an SM do (us;
// four CTAs fit an SM): a CTA alone goes through r1 tokens per us (100 at 128
// dims, 160 at 64: the latency of its four warps' tiles), an SM through its
// share of the bandwidth, whatever its CTAs (in a window, 1.25 times its share
// while others have fewer).  A launch costs its full rounds of CTAs, then the last
// round (5.5 more each), and a fixed part: 5, 6 for splits joined in a cluster, 8
// with a merge launch (and more for long rows of partials).  Under a window the sequences are taken as all of the bound's
// length, else for a third as that, for the rest as spread evenly up to it.
// Against the plain plan's runs (128 to 4,096 tokens, six rounds): block-scaled,
// 16 x 4,096 tokens 39 -> 31 us, 8 x 5,000-20,000 50 -> 47, 1 x 100,000 69 -> 45,
// 128 x 100-300 27.5 -> 21; windows: 32 x 1,024 (bf16) 37.6 -> 26.7, 128 x 4,096
// (fp8) 179 -> 168.  (Since launches are set up while the one before runs: 29.3,
// 46.2, 42.1, 17.1 with CTAs of two warps; 26.2, 167.  With no more
// than its share for an SM of a window's last round, and 7 for a cluster: bf16 8 x
// 1,024 11.3 us where it is 9.7 now, 24 x 1,024 27.1 and 21.8, 4 x 4,096 17.3 and
// 15.1, 1 x 4,096 9.1 and 9.5.)
//
// With a quarter of a round of items or more, a launch ends unevenly: the CTAs of
// its last round are few, and a CTA alone reads at r1.  Splits of falling length
// (each 0.45 to 0.78 of the one before; a split's CTAs start after all of the one
// before) end it with short ones.  Block-scaled, lengths spread up to n, equal
// splits -> falling ones: 64 x 4,096 62.5 -> 56.2 us, 32 x 4,096 38.8 -> 34.4, 128 x
// 4,096 109 -> 103, 32 x 1,500 22.5 -> 17.5, 20 x 8,192 46.6 -> 42.5, 100 x 8,192
// 165 -> 164, d64 128 x 4,096 86.6 -> 71.9, 64 heads 64 x 4,096 66.0 -> 59.6; all of
// one length: 76 x 4,096 115 -> 106, 100 x 8,192 268 -> 251, but 24 x 2,048 23.9 ->
// 27.4.  Where many short sequences make several rounds of their own the short
// splits only cost (256 x 1,024 59 -> 64, 400 x 2,048 155 -> 162: excluded).  In a
// window the lengths are the same: taken from 0.9 MB of K and V an item on, up to
// 1.5 rounds (fp8 40 x 4,096 62.7 -> 54.9, 100 x 4,096 130 -> 122, bf16 64 x 4,096
// 154 -> 146; excluded: fp8 64 x 2,048 50.1 -> 52.5, 128 x 4,096 of 64 heads 165 ->
// 170).
static DecodePlan plan_view(const pkv_cache_desc* d, int batch, int hq, int max_seq_len, int window,
                            int sink_tokens, int forced, int sm_count) {
  // (so far below 2^31 that whole splits stay below it too)
  const int len = std::min(visible_bound(max_seq_len, window, sink_tokens), INT32_MAX - (1 << 21));
  const int tiles = std::max(1, ceil_div(len, kSubTokens));
  if (forced > 0 || tiles <= 4) return plan_decode(d, batch, hq, len, forced > 0 ? forced : 1, sm_count);
  const int sms = sm_count > 0 ? sm_count : 152;
  const double items = (double)batch * d->num_kv_heads * ((hq / d->num_kv_heads + 7) / 8);
  const double r1 = d->head_dim != 128 ? 160.0 : window > 0 ? 90.0 : 100.0;
  const double over = window > 0 ? 1.25 : 1.0;
  const double sm_rate = 44600.0 / (2.0 * d->head_dim * elem_bytes(d->cache_dtype));
  const double slots = 4.0 * sms;
  double best = 1e30;
  int best_s = 1;
  bool best_cluster = false;
  // at most about two rounds of CTAs beyond one per item, of 64 tokens at least
  const int most = (int)std::min<double>(std::max(1, tiles / 4), 2.0 * slots / items + 8.0);
  for (int s = 1; s <= most; s += s < 16 ? 1 : s / 8) {
    const int chunk = ceil_div(tiles, s);
    if (s > 1 && ceil_div(tiles, chunk) != s) continue;  // the same plan as a smaller s
    const double tokens = 16.0 * chunk;
    const double ctas = items * s, full = std::floor(ctas / slots), rest = ctas - full * slots;
    double cost = full * (tokens * 4 / sm_rate + 5.5);
    if (rest > 0)
      cost += std::max(tokens / std::min(r1, over * sm_rate / std::ceil(rest / sms)),
                       rest * tokens / (sm_rate * sms)) + 5.5;
    if (window <= 0) {
      const double some = items * (s + 1) * 0.5, k = std::min(4.0, std::ceil(some / sms));
      const double one = tokens / std::min(r1, sm_rate / k);
      const double spread = std::max(one, items * len * 0.5 / (sm_rate * sms) + 0.5 * one) +
                            2.0 * some / slots;
      cost = 0.35 * cost + 0.65 * spread;
    }
    const bool cl = s >= 2 && s <= 8 && (s & (s - 1)) == 0 && items * s <= 0.75 * slots;
    cost += s == 1 ? 5.0 : cl ? 6.0 : 8.0 + 0.2 * std::max(0, s - 8);
    if (cost < best) {
      best = cost;
      best_s = s;
      best_cluster = cl;
    }
  }
  DecodePlan pl = plan_decode(d, batch, hq, len, best_s, sm_count);
  if (best_cluster && pl.splits == best_s) {
    pl.cluster = true;
    pl.ws_bytes = 0;
  }
  // splits of falling length: see above
  const double fill = items / slots;
  const bool falling = window > 0 ? fill <= 1.5 && 2.0 * len * d->head_dim * elem_bytes(d->cache_dtype) >= 0.9e6
                                  : len >= 1000 && fill <= len / 800.0;
  if (fill >= 0.25 && falling) {
    const double ratio = std::min(0.78, std::max(0.45, 0.45 + 0.75 * (0.75 - fill)));
    int k = kMaxCuts;
    double first = 0;
    for (; k > 1; --k) {  // the last one of 192 tokens at least
      first = len * (1 - ratio) / (1 - std::pow(ratio, k));
      if (first * std::pow(ratio, k - 1) >= 192) break;
    }
    if (k > 1) {
      pl = DecodePlan{};
      pl.splits = pl.num_cuts = k;
      double at = 0;
      for (int i = 0; i <= kMaxCuts; ++i, at += first, first *= ratio)
        pl.cut[i] = i < k    ? (int)(at / kSubTokens + 0.5) * kSubTokens
                    : i == k ? tiles * kSubTokens
                             : INT32_MAX;
      pl.chunk = pl.cut[1];
      size_partials(pl, d, batch, hq);
    }
  }
  return pl;
}

// Bytes that serve the automatic plan of every batch up to `batch` with every bound
// up to max_seq_len (plans come and go with both: 512 requests of 4,096 tokens take
// one split each and no workspace, 400 take partials).  plan_view's splits: at most
// 2 slots / items + 8, and of 64 tokens at least; those of falling length at most
// kMaxCuts, of 192.  Both bounds, times the batch, grow with it.
static size_t view_workspace_bound(const pkv_cache_desc* d, int batch, int hq, int max_seq_len,
                                   int window, int sink_tokens, int sm_count) {
  static_assert(kMaxCuts <= 8, "the bound below");
  const int len = std::min(visible_bound(max_seq_len, window, sink_tokens), INT32_MAX - (1 << 21));
  const int tiles = ceil_div(len, kSubTokens);
  if (tiles / 4 < 2) return 0;
  const double ctas = (double)d->num_kv_heads * ((hq / d->num_kv_heads + 7) / 8);  // of a request's split
  const double slots = 4.0 * (sm_count > 0 ? sm_count : 152);
  const double splits = std::min((double)batch * (tiles / 4), 2.0 * slots / ctas + 8.0 * batch);
  const size_t rows = (size_t)splits * (size_t)hq;  // partials: splits of all requests x heads
  return align256(rows * d->head_dim * sizeof(float)) + rows * sizeof(float);
}

// Decode, optionally with the current token's K/V (k_new/v_new, [B][Hkv][D]
// act dtype) appended to position seq_len-1 inside the decode kernel, or
// through a view (a window and / or scales per block).
static pkv_status decode_common(const pkv_cache_desc* desc, const void* k_cache,
                                const void* v_cache, const void* k_new, const void* v_new,
                                const void* q, void* out, pkv_dtype act_dtype,
                                const int32_t* block_tables, int32_t max_blocks_per_seq,
                                const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                                float sm_scale, int32_t max_seq_len, int32_t num_splits,
                                float* lse_out, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream, const AttnView* view = nullptr) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (batch < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || max_seq_len < 0 ||
      num_splits < 0 || !std::isfinite(sm_scale))
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int group = num_q_heads / desc->num_kv_heads;
  if (batch == 0) return PKV_OK;
  if (batch > 65535 || desc->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !q || !out || !block_tables || !seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 4) || !aligned(out, 2))
    return PKV_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return PKV_ERR_INVALID_ARG;
  if (k_new && (!aligned(k_new, 16) || !aligned(v_new, 16))) return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  const DecodePlan pl =
      view ? plan_view(desc, batch, num_q_heads, max_seq_len, view->window, view->sink_tokens,
                       num_splits, ds->sm_count)
           : plan_decode(desc, batch, num_q_heads, max_seq_len, num_splits, ds->sm_count);
  if (pl.ws_bytes > 0 && (!workspace || workspace_bytes < pl.ws_bytes || !aligned(workspace, 256)))
    return PKV_ERR_WORKSPACE;
  if (pl.splits > 65535) return PKV_ERR_UNSUPPORTED;
  CUtensorMap kmap, vmap;
  if ((st = make_page_map(&kmap, k_cache, desc)) != PKV_OK) return st;
  if ((st = make_page_map(&vmap, v_cache, desc)) != PKV_OK) return st;
  DecodeParams p;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.q = q;
  p.out = out;
  p.lse_out = lse_out;
  p.ws_o = pl.ws_bytes ? reinterpret_cast<float*>(workspace) : nullptr;
  p.ws_lse = pl.ws_bytes ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + pl.ws_lse_offset)
                         : nullptr;
  p.err = ds->err;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = desc->num_blocks;
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = desc->num_kv_heads;
  p.group = group;
  p.bs_shift = desc->block_size == 16 ? 4 : 5;
  p.chunk = pl.chunk;
  p.num_splits = pl.splits;
  p.scale_log2 = score_scale_log2(desc, sm_scale);
  p.out_scale = output_scale(desc);
  DecodeExtraParams ap{};
  ap.k_new = k_new;
  ap.v_new = v_new;
  ap.k_cache = const_cast<void*>(k_cache);
  ap.v_cache = const_cast<void*>(v_cache);
  ap.k_scale = desc->k_scale;
  ap.v_scale = desc->v_scale;
  ap.k_rcp = (float)(1.0 / (double)desc->k_scale);
  ap.v_rcp = (float)(1.0 / (double)desc->v_scale);
  if (view) {
    ap.window = view->window;
    ap.sink_tokens = view->sink_tokens;
    ap.k_scales = view->k_scales;
    ap.v_scales = view->v_scales;
    ap.join_cluster = pl.cluster ? 1 : 0;
    // Short sequences, one CTA each and more of them than fit at once in CTAs of
    // four warps: twice as many of half the size overlap their fixed costs (setup,
    // first copy, epilogue).  Block-scaled, 8 kv heads, four warps -> two: 128 x 64
    // tokens 11.1 -> 8.4 us, 512 x 64 39.8 -> 28.0, 256 x 128 24.5 -> 19.3, 128 x 300
    // 19.0 -> 17.3, 512 x 300 55.4 -> 46.3; 64 x 300 (fewer than a round) 10.0 -> 11.6,
    // 256 x 600 43.0 -> 43.5, 256 x 1,024 58.5 -> 65.5.  Windows: fp8 512 x 128 65.3 ->
    // 51.3, 128 x 256 26.6 -> 22.3, bf16 256 x 128 46.1 -> 42.8, 128 x 256 37.0 -> 38.2.
    const int64_t ctas = (int64_t)batch * desc->num_kv_heads * ((group + 7) / 8);
    ap.two_warps = !pl.cluster && pl.splits == 1 && pl.chunk <= 400 && ctas > 4 * ds->sm_count ? 1 : 0;
    ap.num_cuts = pl.num_cuts;
    std::copy(pl.cut, pl.cut + kMaxCuts + 1, ap.cut);
    e = launch_decode_window(kmap, vmap, p, ap, desc->head_dim, (int)desc->cache_dtype,
                             (int)act_dtype, stream);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  }
  e = launch_decode(kmap, vmap, p, ap, desc->head_dim, (int)desc->cache_dtype, (int)act_dtype,
                    stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_paged_decode_attn(const pkv_cache_desc* desc, const void* k_cache,
                                 const void* v_cache, const void* q, void* out,
                                 pkv_dtype act_dtype, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 int32_t batch, int32_t num_q_heads, float sm_scale,
                                 int32_t max_seq_len, int32_t num_splits, float* lse_out,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return decode_common(desc, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, block_tables,
                       max_blocks_per_seq, seq_lens, batch, num_q_heads, sm_scale, max_seq_len,
                       num_splits, lse_out, workspace, workspace_bytes, stream);
}

pkv_status pkv_paged_decode_attn_append(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                                        const void* k_new, const void* v_new, const void* q,
                                        void* out, pkv_dtype act_dtype,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, int32_t batch,
                                        int32_t num_q_heads, float sm_scale, int32_t max_seq_len,
                                        int32_t num_splits, float* lse_out, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  if (!k_new || !v_new) return PKV_ERR_INVALID_ARG;
  return decode_common(desc, k_cache, v_cache, k_new, v_new, q, out, act_dtype, block_tables,
                       max_blocks_per_seq, seq_lens, batch, num_q_heads, sm_scale, max_seq_len,
                       num_splits, lse_out, workspace, workspace_bytes, stream);
}

size_t pkv_decode_window_workspace_bytes(const pkv_cache_desc* desc, int32_t batch,
                                         int32_t num_q_heads, int32_t max_seq_len, int32_t window,
                                         int32_t sink_tokens, int32_t num_splits) {
  if (check_desc(desc) != PKV_OK || batch <= 0 || num_q_heads <= 0 || max_seq_len < 0 ||
      window < 0 || sink_tokens < 0 || num_splits < 0)
    return 0;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  const int sm_count = ds ? ds->sm_count : 0;
  if (num_splits > 0)
    return plan_view(desc, batch, num_q_heads, max_seq_len, window, sink_tokens, num_splits, sm_count)
        .ws_bytes;
  return view_workspace_bound(desc, batch, num_q_heads, max_seq_len, window, sink_tokens, sm_count);
}

pkv_status pkv_paged_decode_attn_window(const pkv_cache_desc* desc, const void* k_cache,
                                        const void* v_cache, const void* q, void* out,
                                        pkv_dtype act_dtype, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                        int32_t batch, int32_t num_q_heads, float sm_scale,
                                        int32_t max_seq_len, int32_t window, int32_t sink_tokens,
                                        int32_t num_splits, float* lse_out, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  const AttnView view{nullptr, nullptr, window, sink_tokens};
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_view(desc, view, false);
  if (st != PKV_OK) return st;
  if (window == 0) return PKV_ERR_INVALID_ARG;
  return decode_common(desc, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, block_tables,
                       max_blocks_per_seq, seq_lens, batch, num_q_heads, sm_scale, max_seq_len,
                       num_splits, lse_out, workspace, workspace_bytes, stream, &view);
}

pkv_status pkv_paged_decode_attn_block_scaled(
    const pkv_cache_desc* desc, const void* k_cache, const void* v_cache, const float* k_scales,
    const float* v_scales, const void* q, void* out, pkv_dtype act_dtype,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
    int32_t batch, int32_t num_q_heads, float sm_scale, int32_t max_seq_len, int32_t window,
    int32_t sink_tokens, int32_t num_splits, float* lse_out, void* workspace,
    size_t workspace_bytes, cudaStream_t stream) {
  const AttnView view{k_scales, v_scales, window, sink_tokens};
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_view(desc, view, true);
  if (st == PKV_OK && batch > 0) st = check_scales(k_scales, v_scales);
  if (st != PKV_OK) return st;
  const pkv_cache_desc d = scaled_desc(desc);
  return decode_common(&d, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, block_tables,
                       max_blocks_per_seq, seq_lens, batch, num_q_heads, sm_scale, max_seq_len,
                       num_splits, lse_out, workspace, workspace_bytes, stream, &view);
}

pkv_status pkv_kv_append_block_scaled(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                                      float* k_scales, float* v_scales, const void* k_new,
                                      const void* v_new, pkv_dtype act_dtype,
                                      const int32_t* q_indptr, const int32_t* prefix_lens,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      int32_t batch, int32_t total_rows, int32_t max_suffix_len,
                                      cudaStream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (desc->cache_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
  if (batch < 0 || max_blocks_per_seq <= 0 || total_rows < 0 || max_suffix_len < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0 || max_suffix_len == 0) return PKV_OK;
  if ((st = check_scales(k_scales, v_scales)) != PKV_OK) return st;
  if (!k_cache || !v_cache || !k_new || !v_new || !q_indptr || !prefix_lens || !block_tables)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  AppendScaledParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.k_new = k_new;
  p.v_new = v_new;
  p.q_indptr = q_indptr;
  p.prefix_lens = prefix_lens;
  p.block_tables = block_tables;
  p.err = ds->err;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = desc->num_blocks;
  p.num_kv_heads = desc->num_kv_heads;
  p.batch = batch;
  p.total_rows = total_rows;
  p.max_suffix_len = max_suffix_len;
  e = launch_append_scaled(p, (int)act_dtype, desc->head_dim, desc->block_size, stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_kv_gather(const pkv_cache_desc* desc, const void* k_cache, const void* v_cache,
                         const float* k_scales, const float* v_scales, void* k_out, void* v_out,
                         pkv_dtype act_dtype, const int32_t* row_indptr,
                         const int32_t* start_positions, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, int32_t batch, int32_t total_rows,
                         cudaStream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (batch < 0 || max_blocks_per_seq <= 0 || total_rows < 0) return PKV_ERR_INVALID_ARG;
  if ((k_scales == nullptr) != (v_scales == nullptr)) return PKV_ERR_INVALID_ARG;
  if (k_scales) {
    if (desc->cache_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
    if ((st = check_scales(k_scales, v_scales)) != PKV_OK) return st;
  }
  if (batch == 0 || total_rows == 0) return PKV_OK;
  if (!k_cache || !v_cache || !k_out || !v_out || !row_indptr || !start_positions || !block_tables)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  GatherParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.k_out = k_out;
  p.v_out = v_out;
  p.row_indptr = row_indptr;
  p.start_positions = start_positions;
  p.block_tables = block_tables;
  p.err = ds->err;
  p.total_rows = total_rows;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = desc->num_blocks;
  p.num_kv_heads = desc->num_kv_heads;
  p.batch = batch;
  p.bs_shift = desc->block_size == 16 ? 4 : 5;
  p.k_scale = desc->k_scale;
  p.v_scale = desc->v_scale;
  e = launch_gather(p, (int)desc->cache_dtype, (int)act_dtype, desc->head_dim, stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t pkv_extend_workspace_bytes(const pkv_cache_desc* desc, int32_t batch, int32_t num_q_heads,
                                  int32_t total_q_rows, int32_t max_total_len) {
  // every dtype, fp8 included, is read straight from the cache: no scratch
  (void)desc; (void)batch; (void)num_q_heads; (void)total_q_rows; (void)max_total_len;
  return 0;
}

}  // extern "C"

// Shared-prefix extend: the groups (null group_indptr: plain extend).
struct ExtendGroups {
  const int32_t* group_indptr;
  const int32_t* group_shared;
  int32_t num_groups;
  int32_t max_group_rows;
};

// Extend, optionally with the suffix's K/V (k_new/v_new, [rows][Hkv][D] in
// the act dtype) written into the cache before the extend kernel runs, or
// (groups) with the rows of each group's requests packed into shared tiles.
// Workspace the shared-prefix extend can use: f16 copies of the pools (the same
// block ids) into which the call widens the pages it reads, so that the kernel
// takes them as f16 instead of converting every tile -- the V pool of a bf16
// cache, the K and V pools of an fp8 cache (K first); none for an f16 cache.
static size_t shared_prefix_pool16_bytes(const pkv_cache_desc* d) {
  return align256((size_t)d->num_blocks * d->num_kv_heads * d->block_size * d->head_dim * 2);
}
static size_t shared_prefix_widen_bytes(const pkv_cache_desc* d) {
  if (d->cache_dtype == PKV_BF16) return shared_prefix_pool16_bytes(d);
  if (d->cache_dtype == PKV_FP8_E4M3) return 2 * shared_prefix_pool16_bytes(d);
  return 0;
}
// The plain extend's optional workspace: the same pools, then a counter, a
// claim flag per block and a list of the blocks claimed (requests may share
// blocks without the call knowing it).
static size_t plain_widen_bytes(const pkv_cache_desc* d) {
  const size_t pools = shared_prefix_widen_bytes(d);
  return pools ? pools + align256((1 + 2 * (size_t)d->num_blocks) * sizeof(int32_t)) : 0;
}

static pkv_status extend_common(const pkv_cache_desc* desc, const void* k_cache,
                                const void* v_cache, const void* k_new, const void* v_new,
                                const void* q, void* out, pkv_dtype act_dtype,
                                const int32_t* q_indptr, const int32_t* prefix_lens,
                                const int32_t* block_tables, int32_t max_blocks_per_seq,
                                int32_t batch, int32_t num_q_heads, float sm_scale,
                                int32_t total_q_rows, int32_t max_suffix_len,
                                int32_t max_total_len, float* lse_out, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream,
                                const ExtendGroups* groups = nullptr,
                                const AttnView* view = nullptr) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if ((st = check_act(desc, act_dtype)) != PKV_OK) return st;
  if (batch < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || total_q_rows < 0 ||
      max_suffix_len < 0 || max_total_len < 0 || !std::isfinite(sm_scale) || !(sm_scale > 0.f))
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int group = num_q_heads / desc->num_kv_heads;
  if (!extend_supported(desc->head_dim, (int)desc->cache_dtype, (int)act_dtype, group))
    return PKV_ERR_UNSUPPORTED;
  // no call needs scratch; either may take one to widen the pages it reads
  // once instead of per tile (a plain call whose workspace is smaller than
  // that, such as the 0 bytes of pkv_extend_workspace_bytes, does without)
  const size_t plain_bytes = groups ? 0 : plain_widen_bytes(desc);
  const bool widen_plain = !groups && workspace != nullptr && plain_bytes > 0 &&
                           workspace_bytes >= plain_bytes && aligned(workspace, 256) &&
                           batch <= 65535;
  const bool scaled = view && view->k_scales;
  const size_t widen_bytes = groups ? shared_prefix_widen_bytes(desc) : 0;
  // (the widening pass takes one CTA row per request: larger batches keep the
  // per-tile conversion)
  const bool widen = groups && workspace != nullptr && widen_bytes > 0 && batch <= 65535;
  if (widen && (workspace_bytes < widen_bytes || !aligned(workspace, 256))) return PKV_ERR_WORKSPACE;
  if (groups) {
    if (groups->num_groups < 0 || groups->max_group_rows < 0 || groups->num_groups > batch)
      return PKV_ERR_INVALID_ARG;
    if (batch > 0 && groups->num_groups == 0) return PKV_ERR_INVALID_ARG;
  }
  const int32_t rows_hint = groups ? groups->max_group_rows : max_suffix_len;
  if (batch == 0 || total_q_rows == 0 || rows_hint == 0) return PKV_OK;
  if (!k_cache || !v_cache || !q || !out || !block_tables || !q_indptr || !prefix_lens)
    return PKV_ERR_INVALID_ARG;
  if (groups && (!groups->group_indptr || !groups->group_shared)) return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16))
    return PKV_ERR_INVALID_ARG;
  cudaError_t e;
  DeviceState* ds = device_state(&e);
  if (!ds) return PKV_ERR_CUDA;
  CUtensorMap kmap, vmap, qmap, omap;
  if ((st = make_page_map(&kmap, k_cache, desc)) != PKV_OK) return st;
  if ((st = make_page_map(&vmap, v_cache, desc)) != PKV_OK) return st;
  if ((st = make_q_map(&qmap, q, desc->head_dim, num_q_heads, total_q_rows, group)) != PKV_OK)
    return st;
  // the output has q's shape and layout: the same map over out
  if ((st = make_q_map(&omap, out, desc->head_dim, num_q_heads, total_q_rows, group)) != PKV_OK)
    return st;
  ExtendParams p{};
  p.q_indptr = q_indptr;
  p.prefix_lens = prefix_lens;
  p.block_tables = block_tables;
  p.group_indptr = groups ? groups->group_indptr : nullptr;
  p.group_shared = groups ? groups->group_shared : nullptr;
  p.q = q;
  p.out = out;
  p.lse_out = lse_out;
  p.err = ds->err;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = desc->num_blocks;
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = desc->num_kv_heads;
  p.out_32b = aligned(out, 32) ? 1 : 0;
  p.out_tma = 1;
  p.bs_shift = desc->block_size == 16 ? 4 : 5;
  p.total_rows = total_q_rows;
  p.scale_log2 = score_scale_log2(desc, sm_scale);
  p.out_scale = output_scale(desc);
  p.window = view ? view->window : 0;
  p.sink_tokens = view ? view->sink_tokens : 0;
  // work items per (request or group, kv head): pairs of row tiles
  if (!plan_extend(p, groups ? groups->num_groups : batch, desc->num_kv_heads, group, rows_hint,
                   ds->sm_count))
    return PKV_ERR_UNSUPPORTED;
  if (groups) {
    int cache_dt = (int)desc->cache_dtype;
    if (widen) {
      // the pages the call reads, widened in the workspace (same block ids),
      // then read by the kernel through maps over those pools: V as f16, an
      // fp8 cache's K in the queries' type; the scales of an fp8 cache stay
      // folded into p's softmax and output scales
      pkv_cache_desc d16 = *desc;
      d16.cache_dtype = PKV_F16;
      const bool fp8 = desc->cache_dtype == PKV_FP8_E4M3;
      void* k16 = fp8 ? workspace : nullptr;
      void* v16 = static_cast<uint8_t*>(workspace) + (fp8 ? shared_prefix_pool16_bytes(desc) : 0);
      if (fp8 && (st = make_page_map(&kmap, k16, &d16)) != PKV_OK) return st;
      if ((st = make_page_map(&vmap, v16, &d16)) != PKV_OK) return st;
      e = launch_widen(fp8 ? DT_E4M3 : DT_BF16, (int)act_dtype, k_cache, v_cache, k16, v16, p,
                       groups->num_groups, desc->head_dim, desc->block_size, max_total_len, stream);
      if (e != cudaSuccess) return PKV_ERR_CUDA;
      // K bf16 (cache or widened) with f16 V; an fp8 cache under f16 queries
      // is then an f16 cache
      cache_dt = act_dtype == PKV_BF16 ? DT_BF16_V16 : DT_F16;
    }
    e = launch_extend_shared(kmap, vmap, qmap, omap, p, desc->head_dim, cache_dt, (int)act_dtype,
                             stream);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  }
  if (k_new) {
    // the suffix's K/V first (its slots computed from the extend layout), then
    // the extend kernel reads them back; two launches in stream order
    AppendParams ap{};
    ap.k_cache = const_cast<void*>(k_cache);
    ap.v_cache = const_cast<void*>(v_cache);
    ap.k_new = k_new;
    ap.v_new = v_new;
    ap.slots = nullptr;
    ap.err = ds->err;
    ap.num_tokens = total_q_rows;
    ap.num_kv_heads = desc->num_kv_heads;
    ap.head_dim = desc->head_dim;
    ap.block_size = desc->block_size;
    ap.num_blocks = desc->num_blocks;
    ap.k_scale = desc->k_scale;
    ap.v_scale = desc->v_scale;
    ap.q_indptr = q_indptr;
    ap.prefix_lens = prefix_lens;
    ap.block_tables = block_tables;
    ap.batch = batch;
    ap.max_blocks = max_blocks_per_seq;
    e = launch_append(ap, (int)desc->cache_dtype, (int)act_dtype, stream);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
  }
  int cache_dt = (int)desc->cache_dtype;
  bool widen_pages = widen_plain;
  if (view) {
    plan_view_items(p, max_total_len, ds->sm_count);
    if (p.splits > 1 || p.half) p.out_tma = 0;  // (every row leaves with its parts' sum)
    const int64_t units = total_q_rows / (2 * p.tok) + (int64_t)batch;
    p.num_blocks_dyn = p.num_items;
    p.div_rows = make_fastdiv((uint32_t)(2 * p.tok));
    if (units * desc->num_kv_heads * 2 < p.num_items) {
      p.by_rows = 1;
      p.num_units = (int)units;
      p.num_blocks_dyn = (int)(units * desc->num_kv_heads);
    }
    // Widening pays where many pairs of row tiles would convert the same pages:
    // one pair per key tile costs 15 % (4 requests of 1,900 rows x 4 heads, 59
    // pairs: 804 against 957 us), the pass itself three launches and three
    // times the pages' bytes (300 rows, 10 pairs: 140 against 132; 16 rows: 123
    // against 68).
    if (p.splits > 1 || p.half || (p.tiles_per_head + 1) / 2 < 16) widen_pages = false;
    if (scaled && !widen_pages) {
      p.k_scales = view->k_scales;
      p.v_scales = view->v_scales;
    }
  }
  if (widen_pages) {
    // the pages the call reads, each block widened once (claimed in the
    // workspace) into 16-bit pools read through maps over them
    pkv_cache_desc d16 = *desc;
    d16.cache_dtype = PKV_F16;
    const bool fp8 = desc->cache_dtype == PKV_FP8_E4M3;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    void* k16 = fp8 ? base : nullptr;
    void* v16 = base + (fp8 ? shared_prefix_pool16_bytes(desc) : 0);
    int32_t* claims = reinterpret_cast<int32_t*>(base + shared_prefix_widen_bytes(desc));
    if (fp8 && (st = make_page_map(&kmap, k16, &d16)) != PKV_OK) return st;
    if ((st = make_page_map(&vmap, v16, &d16)) != PKV_OK) return st;
    if (scaled)
      e = launch_widen_scaled((int)act_dtype, k_cache, v_cache, view->k_scales, view->v_scales, k16,
                              v16, claims, p, desc->head_dim, desc->block_size, max_total_len,
                              ds->sm_count, stream);
    else
      e = launch_widen_claim(fp8 ? DT_E4M3 : DT_BF16, (int)act_dtype, k_cache, v_cache, k16, v16,
                             claims, p, desc->head_dim, desc->block_size, max_total_len,
                             ds->sm_count, stream);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    cache_dt = act_dtype == PKV_BF16 ? DT_BF16_V16 : DT_F16;
  }
  if (view)
    e = launch_extend_view(kmap, vmap, qmap, omap, p, desc->head_dim, cache_dt, (int)act_dtype,
                           stream);
  else
    e = launch_extend(kmap, vmap, qmap, omap, p, desc->head_dim, cache_dt, (int)act_dtype, stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" {

pkv_status pkv_paged_extend_attn(const pkv_cache_desc* desc, const void* k_cache,
                                 const void* v_cache, const void* q, void* out,
                                 pkv_dtype act_dtype, const int32_t* q_indptr,
                                 const int32_t* prefix_lens, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, int32_t batch, int32_t num_q_heads,
                                 float sm_scale, int32_t total_q_rows, int32_t max_suffix_len,
                                 int32_t max_total_len, float* lse_out, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  return extend_common(desc, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, q_indptr,
                       prefix_lens, block_tables, max_blocks_per_seq, batch, num_q_heads,
                       sm_scale, total_q_rows, max_suffix_len, max_total_len, lse_out, workspace,
                       workspace_bytes, stream);
}

pkv_status pkv_paged_extend_attn_window(const pkv_cache_desc* desc, const void* k_cache,
                                        const void* v_cache, const void* q, void* out,
                                        pkv_dtype act_dtype, const int32_t* q_indptr,
                                        const int32_t* prefix_lens, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, int32_t batch,
                                        int32_t num_q_heads, float sm_scale, int32_t total_q_rows,
                                        int32_t max_suffix_len, int32_t max_total_len,
                                        int32_t window, int32_t sink_tokens, float* lse_out,
                                        void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
  const AttnView view{nullptr, nullptr, window, sink_tokens};
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_view(desc, view, false);
  if (st != PKV_OK) return st;
  if (window == 0) return PKV_ERR_INVALID_ARG;
  return extend_common(desc, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, q_indptr,
                       prefix_lens, block_tables, max_blocks_per_seq, batch, num_q_heads,
                       sm_scale, total_q_rows, max_suffix_len, max_total_len, lse_out, workspace,
                       workspace_bytes, stream, nullptr, &view);
}

size_t pkv_extend_block_scaled_workspace_bytes(const pkv_cache_desc* desc) {
  if (check_desc(desc) != PKV_OK || desc->cache_dtype != PKV_FP8_E4M3) return 0;
  return plain_widen_bytes(desc);
}

pkv_status pkv_paged_extend_attn_block_scaled(
    const pkv_cache_desc* desc, const void* k_cache, const void* v_cache, const float* k_scales,
    const float* v_scales, const void* q, void* out, pkv_dtype act_dtype, const int32_t* q_indptr,
    const int32_t* prefix_lens, const int32_t* block_tables, int32_t max_blocks_per_seq,
    int32_t batch, int32_t num_q_heads, float sm_scale, int32_t total_q_rows,
    int32_t max_suffix_len, int32_t max_total_len, int32_t window, int32_t sink_tokens,
    float* lse_out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const AttnView view{k_scales, v_scales, window, sink_tokens};
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_view(desc, view, true);
  if (st == PKV_OK && batch > 0) st = check_scales(k_scales, v_scales);
  if (st != PKV_OK) return st;
  const pkv_cache_desc d = scaled_desc(desc);
  return extend_common(&d, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, q_indptr,
                       prefix_lens, block_tables, max_blocks_per_seq, batch, num_q_heads,
                       sm_scale, total_q_rows, max_suffix_len, max_total_len, lse_out, workspace,
                       workspace_bytes, stream, nullptr, &view);
}

size_t pkv_extend_widen_workspace_bytes(const pkv_cache_desc* desc) {
  if (check_desc(desc) != PKV_OK) return 0;
  return plain_widen_bytes(desc);
}

size_t pkv_extend_shared_prefix_workspace_bytes(const pkv_cache_desc* desc) {
  if (check_desc(desc) != PKV_OK) return 0;
  return shared_prefix_widen_bytes(desc);
}

pkv_status pkv_paged_extend_attn_shared_prefix(
    const pkv_cache_desc* desc, const void* k_cache, const void* v_cache, const void* q, void* out,
    pkv_dtype act_dtype, const int32_t* q_indptr, const int32_t* prefix_lens,
    const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t batch, int32_t num_q_heads,
    float sm_scale, int32_t total_q_rows, const int32_t* group_indptr,
    const int32_t* group_shared_lens, int32_t num_groups, int32_t max_group_rows,
    int32_t max_total_len, float* lse_out, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
  const ExtendGroups groups{group_indptr, group_shared_lens, num_groups, max_group_rows};
  return extend_common(desc, k_cache, v_cache, nullptr, nullptr, q, out, act_dtype, q_indptr,
                       prefix_lens, block_tables, max_blocks_per_seq, batch, num_q_heads,
                       sm_scale, total_q_rows, max_group_rows, max_total_len, lse_out, workspace,
                       workspace_bytes, stream, &groups);
}

pkv_status pkv_paged_extend_attn_append(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                                        const void* k_new, const void* v_new, const void* q,
                                        void* out, pkv_dtype act_dtype, const int32_t* q_indptr,
                                        const int32_t* prefix_lens, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, int32_t batch,
                                        int32_t num_q_heads, float sm_scale, int32_t total_q_rows,
                                        int32_t max_suffix_len, int32_t max_total_len,
                                        float* lse_out, cudaStream_t stream) {
  if (!k_new || !v_new) return PKV_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return PKV_ERR_INVALID_ARG;
  return extend_common(desc, k_cache, v_cache, k_new, v_new, q, out, act_dtype, q_indptr,
                       prefix_lens, block_tables, max_blocks_per_seq, batch, num_q_heads,
                       sm_scale, total_q_rows, max_suffix_len, max_total_len, lse_out, nullptr, 0,
                       stream);
}

}  // extern "C"
