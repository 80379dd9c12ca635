// tv_api.cu -- the C ABI of libtv (include/tv.h): argument checks on the host,
// launch configuration, TMA tensor maps, and launches on the caller's stream.
// The library allocates nothing and never synchronises.
#include <cfloat>
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/tv.h"
#include "tv_device.cuh"
#include "tv_launch.h"

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

int sm_count() {
  static thread_local int cached_dev = -1, cached_n = 148;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cached_n;
  if (dev == cached_dev) return cached_n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return cached_n;
  cached_dev = dev;
  cached_n = n;
  return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct AttnPlan {
  int group;        // query heads per KV head
  int lanes;        // CTAs per virtual CTA (m-tile pairs of one layer)
  int vctas;        // virtual CTAs
  int min_tiles;    // fewest key tiles per virtual CTA
  size_t workspace; // counters + partial-result slots
};

// Fewest 128-key tiles a virtual CTA is given: below this a unit is not split
// further, since a split piece costs about this much in fixed work (its Q
// load, the pipeline fill and its partial-result write).  Timed at 2, 3, 4,
// 5, 6 and 9: only the short-prefix MHA line (32 heads x 9 tiles) moved, and
// 3 was fastest there (each unit then splits into three whole ranges).
constexpr int kMinTiles = 3;

// Launch plan for `sms` SMs (one persistent CTA per SM).  A layer of `lanes`
// CTAs takes the m-tile pairs (256 packed rows) of a (sequence, KV head): as
// many lanes as the largest tree has pairs, so that the CTAs reading the
// same K/V tiles run together.  The virtual CTAs (sms / lanes of them, fewer
// when the host hints bound the work below kMinTiles tiles each) share the
// line of key tiles equally on the device.  Workspace: two arrival counters
// per CTA, then two partial-result slots per CTA.
bool plan_attention(const tv_attn_params* p, int sms, AttnPlan* out) {
  if (!p || sms < 1) return false;
  if (p->batch < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1) return false;
  if (p->num_q_heads % p->num_kv_heads) return false;
  if (p->head_dim != 64 && p->head_dim != 128) return false;
  if (p->block_size != TV_BLOCK_SIZE) return false;
  if (p->max_nodes < 1 || p->max_nodes > TV_MAX_NODES) return false;
  if (p->total_nodes < p->batch || p->num_blocks < 1 || p->max_blocks_per_seq < 1) return false;
  if (p->max_prefix_len < 0) return false;
  if ((p->max_prefix_len + 15) / 16 > p->max_blocks_per_seq) return false;
  if (p->out_dtype != TV_OUT_BF16 && p->out_dtype != TV_OUT_FP32) return false;
  if (static_cast<int64_t>(p->num_blocks) * p->num_kv_heads * 16 >= (1ll << 31)) return false;
  if (static_cast<int64_t>(p->total_nodes) * p->num_q_heads >= (1ll << 31)) return false;
  AttnPlan pl;
  pl.group = p->num_q_heads / p->num_kv_heads;
  const long long mpairs = (static_cast<long long>(p->max_nodes) * pl.group + 255) / 256;
  pl.lanes = static_cast<int>(std::min<long long>(mpairs, sms));
  const long long layers = (mpairs + pl.lanes - 1) / pl.lanes;
  const long long tiles = (p->max_prefix_len + 127) / 128 + (p->max_nodes + 127) / 128;
  const long long wmax = static_cast<long long>(p->batch) * p->num_kv_heads * layers * tiles;
  if (wmax >= (1ll << 31)) return false;  // the device schedule counts tiles in 32 bits
  pl.min_tiles = kMinTiles;
  // at most 4096 virtual CTAs: the device computes range boundaries with
  // fp32 products of v r < 4096^2 = 2^24 (exact integers)
  pl.vctas = static_cast<int>(
      std::max(1ll, std::min<long long>({sms / pl.lanes, wmax / kMinTiles, 4096ll})));
  const size_t ctas = static_cast<size_t>(pl.vctas) * pl.lanes;
  pl.workspace = (ctas * 8 + 255) / 256 * 256 + 2 * ctas * tv::attn_slot_bytes(p->head_dim);
  *out = pl;
  return true;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides_bytes, const cuuint32_t* box,
            CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, type, rank, const_cast<void*>(base), dims,
            strides_bytes, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor map of a paged pool whose box is one 16-token page of one KV head.
// E4M3: (128 bytes, 16 rows, pages).  bf16: (64 columns, 8 rows, halves, 2 row
// groups, pages), landing as [8-row group][64-column half][8 rows][128 B].
bool encode_pool(CUtensorMap* m, const void* pool, int D, uint64_t pages, bool fp8) {
  if (fp8) {
    const cuuint64_t dims[3] = {128, 16, pages};
    const cuuint64_t str[2] = {128, 2048};
    const cuuint32_t box[3] = {128, 16, 1};
    return encode(m, pool, 3, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_UINT8);
  }
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t halves = static_cast<cuuint64_t>(D) / 64;
  const cuuint64_t dims[5] = {64, 8, halves, 2, pages};
  const cuuint64_t str[4] = {row, 128, row * 8, row * 16};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(halves), 2, 1};
  return encode(m, pool, 5, dims, str, box);
}

// Shortest range of the chunk attention's line that a CTA is given.
constexpr int kMinRange = 14;

struct ChunkPlan {
  int unit_tokens;  // tokens of a unit
  int vctas;        // CTAs (ranges of the line of key tiles)
  size_t workspace; // counters + partial-result slots
};

// Launch plan of the chunk attention for `sms` SMs: a unit is as many whole
// tokens as give at most 256 packed rows; the CTAs share the line of work
// (at most `wmax` by the host hints) in ranges of at least kMinRange.
// Workspace: a ticket counter per CTA, then two partial-result slots per CTA.
bool plan_chunk(const tv_chunk_params* p, int sms, ChunkPlan* out) {
  if (!p || sms < 1) return false;
  if (p->batch < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1) return false;
  if (p->num_q_heads % p->num_kv_heads || p->num_q_heads / p->num_kv_heads > 256) return false;
  if (p->head_dim != 64 && p->head_dim != 128) return false;
  if (p->block_size != TV_BLOCK_SIZE) return false;
  if (p->total_tokens < 0 || p->num_blocks < 1 || p->max_blocks_per_seq < 1) return false;
  if (p->max_len < 0 || p->max_len > INT32_MAX - 256) return false;
  if ((p->max_len + 15) / 16 > p->max_blocks_per_seq) return false;
  if (p->window < 0 || p->sinks < 0) return false;
  if (!(p->softmax_scale >= 0.0f && p->softmax_scale <= FLT_MAX)) return false;
  if (p->out_dtype != TV_OUT_BF16 && p->out_dtype != TV_OUT_FP32) return false;
  if (static_cast<int64_t>(p->num_blocks) * p->num_kv_heads * 16 >= (1ll << 31)) return false;
  if (static_cast<int64_t>(p->total_tokens) * p->num_q_heads >= (1ll << 31)) return false;
  ChunkPlan pl;
  pl.unit_tokens = 256 / (p->num_q_heads / p->num_kv_heads);
  const int64_t units = p->total_tokens / pl.unit_tokens + static_cast<int64_t>(std::min(p->batch, p->total_tokens));
  int64_t tiles = (static_cast<int64_t>(p->max_len) + 127) / 128;
  if (p->window > 0)  // the sinks' tiles, and the tiles that a unit's windows meet
    tiles = std::min(tiles, (static_cast<int64_t>(p->sinks) + 127) / 128 +
                                (static_cast<int64_t>(p->window) + pl.unit_tokens + 253) / 128);
  const int64_t wmax =
      units * p->num_kv_heads * (std::max<int64_t>(tiles, 1) * tv::kChunkTileCost + tv::kChunkPieceCost);
  if (wmax >= (1ll << 31)) return false;  // counted in 32 bits
  // at most 4096 CTAs: the range boundaries are fp32 products below 2^24
  pl.vctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sms, wmax / kMinRange, 4096})));
  pl.workspace = (static_cast<size_t>(pl.vctas) * 4 + 255) / 256 * 256 +
                 2 * static_cast<size_t>(pl.vctas) * tv::chunk_slot_bytes(p->head_dim);
  *out = pl;
  return true;
}

}  // namespace

extern "C" {

const char* tv_status_string(int s) {
  switch (s) {
    case TV_OK: return "TV_OK";
    case TV_ERR_INVALID_ARG: return "TV_ERR_INVALID_ARG";
    case TV_ERR_UNSUPPORTED: return "TV_ERR_UNSUPPORTED";
    case TV_ERR_WORKSPACE: return "TV_ERR_WORKSPACE";
    case TV_ERR_CUDA: return "TV_ERR_CUDA";
    case TV_ERR_BAD_TREE: return "TV_ERR_BAD_TREE";
    case TV_ERR_DEVICE_TIMEOUT: return "TV_ERR_DEVICE_TIMEOUT";
    case TV_ERR_NO_PAGE: return "TV_ERR_NO_PAGE";
    default: return "TV_ERR_UNKNOWN";
  }
}

int tv_version(void) { return TV_VERSION; }

namespace {
// One thread block waits on an mbarrier that nothing arrives at, through the
// kernels' bounded wait, and reports the outcome.
__global__ void selftest_wait_timeout_kernel(int32_t* status, unsigned long long* waited_ns,
                                             unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    tv::mbar_init(&bar, 1);
    tv::fence_mbar_init();
  }
  __syncthreads();
  const unsigned long long t0 = tv::global_ns();
  const bool done = tv::mbar_wait(&bar, 0, nullptr, limit_ns);
  if (threadIdx.x == 0) {
    *status = done ? tv::kOk : tv::kDeviceTimeout;
    *waited_ns = tv::global_ns() - t0;
  }
}
}  // namespace

int tv_selftest_wait_timeout(int32_t* status, unsigned long long* waited_ns,
                             unsigned long long limit_ns, cudaStream_t stream) {
  if (!status || !waited_ns) return TV_ERR_INVALID_ARG;
  if (limit_ns < 1000000ull || limit_ns > 1000000000ull) return TV_ERR_INVALID_ARG;
  selftest_wait_timeout_kernel<<<1, 32, 0, stream>>>(status, waited_ns, limit_ns);
  return cudaGetLastError() == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

size_t tv_tree_attention_workspace_size(const tv_attn_params* p) {
  AttnPlan pl;
  if (!plan_attention(p, sm_count(), &pl)) return 0;
  return pl.workspace;
}

int tv_tree_attention_plan(const tv_attn_params* p, int32_t sms, tv_attn_plan* out) {
  if (!out) return TV_ERR_INVALID_ARG;
  AttnPlan pl;
  if (!plan_attention(p, sms > 0 ? sms : sm_count(), &pl)) return TV_ERR_INVALID_ARG;
  out->ctas = pl.vctas * pl.lanes;
  out->lanes = pl.lanes;
  out->virtual_ctas = pl.vctas;
  out->min_tiles = pl.min_tiles;
  out->workspace_bytes = pl.workspace;
  return TV_OK;
}

}  // extern "C"

namespace {

struct Fp8Scales {
  const float *q, *kp, *vp, *kn, *vn;
};

// The shared path of tv_tree_attention and tv_tree_attention_fp8: checks,
// tensor maps, arguments, the status and counter memsets and the launch.
int attention_call(const tv_attn_params* p, const Fp8Scales* f8, const void* q_nodes,
                   const void* k_prefix_blocks, const void* v_prefix_blocks,
                   const int32_t* block_table, const void* k_nodes, const void* v_nodes,
                   const int32_t* parent, const int32_t* prefix_lens,
                   const int32_t* node_offsets, void* out, int32_t* status, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (f8 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  AttnPlan pl;
  if (!plan_attention(p, sm_count(), &pl)) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes,
                        v_nodes, parent, prefix_lens, node_offsets, out, status};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  if (f8) {
    const void* sc[] = {f8->q, f8->kp, f8->vp, f8->kn, f8->vn};
    for (const void* q : sc)
      if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  }
  if (!workspace || workspace_bytes < pl.workspace || !aligned16(workspace))
    return TV_ERR_WORKSPACE;

  const int D = p->head_dim, Hkv = p->num_kv_heads;
  tv::AttnMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (f8) {
    // E4M3 codes, one byte each, 128-byte rows.  Pool: (128 bytes, 16 rows,
    // pages), box = one page (2 KB).  Tree K/V: (128 bytes, nodes, KV heads),
    // box = 8 nodes of one head (1 KB).  128-byte swizzle.
    const cuuint64_t pdims[3] = {128, 16, static_cast<cuuint64_t>(p->num_blocks) * Hkv};
    const cuuint64_t pstr[2] = {128, 2048};
    const cuuint32_t pbox[3] = {128, 16, 1};
    if (!encode(&maps.k_pool, k_prefix_blocks, 3, pdims, pstr, pbox, CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return TV_ERR_CUDA;
    if (!encode(&maps.v_pool, v_prefix_blocks, 3, pdims, pstr, pbox, CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return TV_ERR_CUDA;
    const cuuint64_t ndims[3] = {128, static_cast<cuuint64_t>(p->total_nodes), static_cast<cuuint64_t>(Hkv)};
    const cuuint64_t nstr[2] = {static_cast<cuuint64_t>(Hkv) * 128, 128};
    const cuuint32_t nbox[3] = {128, 8, 1};
    if (!encode(&maps.k_nodes, k_nodes, 3, ndims, nstr, nbox, CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return TV_ERR_CUDA;
    if (!encode(&maps.v_nodes, v_nodes, 3, ndims, nstr, nbox, CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return TV_ERR_CUDA;
  } else {
    // Paged pool as a 5-D tensor so that one box is one 16-token page of one
    // KV head, landing in shared memory as [8-row group][64-column half][8
    // rows][128 B]: dims (64 columns, 8 rows, halves, 2 row groups, pages),
    // box (64, 8, halves, 2, 1).
    const int halves = D / 64;
    {
      const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(halves), 2,
                                  static_cast<cuuint64_t>(p->num_blocks) * Hkv};
      const cuuint64_t str[4] = {static_cast<cuuint64_t>(D) * 2, 128,
                                 static_cast<cuuint64_t>(D) * 2 * 8, static_cast<cuuint64_t>(D) * 2 * 16};
      const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(halves), 2, 1};
      if (!encode(&maps.k_pool, k_prefix_blocks, 5, dims, str, box)) return TV_ERR_CUDA;
      if (!encode(&maps.v_pool, v_prefix_blocks, 5, dims, str, box)) return TV_ERR_CUDA;
    }
    // Tree K/V as a 4-D tensor (64 columns, nodes, halves, KV heads); a box
    // is 8 consecutive nodes of one head: [half][8 rows][128 B].
    {
      const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(p->total_nodes),
                                  static_cast<cuuint64_t>(halves), static_cast<cuuint64_t>(Hkv)};
      const cuuint64_t str[3] = {static_cast<cuuint64_t>(D) * 2 * Hkv, 128,
                                 static_cast<cuuint64_t>(D) * 2};
      const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(halves), 1};
      if (!encode(&maps.k_nodes, k_nodes, 4, dims, str, box)) return TV_ERR_CUDA;
      if (!encode(&maps.v_nodes, v_nodes, 4, dims, str, box)) return TV_ERR_CUDA;
    }
  }

  const size_t ctas = static_cast<size_t>(pl.vctas) * pl.lanes;
  tv::AttnArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = static_cast<const uint16_t*>(q_nodes);
  a.block_table = block_table;
  a.parent = parent;
  a.prefix_lens = prefix_lens;
  a.node_offsets = node_offsets;
  a.out = out;
  a.status = status;
  a.counters = static_cast<int32_t*>(workspace);
  a.slots = static_cast<uint8_t*>(workspace) + (ctas * 8 + 255) / 256 * 256;
  a.batch = p->batch;
  a.hq = p->num_q_heads;
  a.hkv = Hkv;
  a.group = pl.group;
  a.head_dim = D;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.max_nodes = p->max_nodes;
  a.max_prefix_len = p->max_prefix_len;
  a.total_nodes = p->total_nodes;
  a.lanes = pl.lanes;
  a.vctas = pl.vctas;
  a.min_tiles = pl.min_tiles;
  a.out_fp32 = p->out_dtype == TV_OUT_FP32 ? 1 : 0;
  const float scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(D));
  a.scale_log2 = scale * 1.4426950408889634f;
  if (f8) {
    a.fp8 = 1;
    a.q_scale = f8->q;
    a.kp_scale = f8->kp;
    a.vp_scale = f8->vp;
    a.kn_scale = f8->kn;
    a.vn_scale = f8->vn;
  }

  // status and the arrival counters of split units start at zero
  if (cudaMemsetAsync(status, 0, sizeof(int32_t) * p->batch, stream) != cudaSuccess)
    return TV_ERR_CUDA;
  if (cudaMemsetAsync(a.counters, 0, ctas * 8, stream) != cudaSuccess) return TV_ERR_CUDA;
  if (tv::launch_tree_attention(a, maps, stream) != 0) return TV_ERR_CUDA;
  return TV_OK;
}

}  // namespace

extern "C" {

int tv_tree_attention(const tv_attn_params* p, const uint16_t* q_nodes,
                      const uint16_t* k_prefix_blocks, const uint16_t* v_prefix_blocks,
                      const int32_t* block_table, const uint16_t* k_nodes,
                      const uint16_t* v_nodes, const int32_t* parent,
                      const int32_t* prefix_lens, const int32_t* node_offsets, void* out,
                      int32_t* status, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
  return attention_call(p, nullptr, q_nodes, k_prefix_blocks, v_prefix_blocks, block_table,
                        k_nodes, v_nodes, parent, prefix_lens, node_offsets, out, status,
                        workspace, workspace_bytes, stream);
}

int tv_tree_attention_fp8(const tv_attn_params* p, const uint8_t* q_nodes, const float* q_scale,
                          const uint8_t* k_prefix_blocks, const float* k_prefix_scale,
                          const uint8_t* v_prefix_blocks, const float* v_prefix_scale,
                          const int32_t* block_table, const uint8_t* k_nodes,
                          const float* k_nodes_scale, const uint8_t* v_nodes,
                          const float* v_nodes_scale, const int32_t* parent,
                          const int32_t* prefix_lens, const int32_t* node_offsets, void* out,
                          int32_t* status, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  const Fp8Scales sc = {q_scale, k_prefix_scale, v_prefix_scale, k_nodes_scale, v_nodes_scale};
  return attention_call(p, &sc, q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes,
                        v_nodes, parent, prefix_lens, node_offsets, out, status, workspace,
                        workspace_bytes, stream);
}

size_t tv_accept_workspace_size(const tv_accept_params* p) {
  if (!p || p->vocab < 1 || p->vocab >= (1 << 18) || p->total_nodes < 1) return 0;
  return tv::accept_workspace_bytes(p->vocab, p->total_nodes);
}

int tv_accept(const tv_accept_params* p, const float* target, const float* draft_probs,
              const int32_t* draft_tokens, const int32_t* parent, const int32_t* node_offsets,
              const float* uniforms, const uint32_t* retained_mask, int32_t* accepted_len,
              int32_t* path, int32_t* bonus_token, int32_t* status, float* debug_pq,
              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return tv_accept_ex(p, nullptr, target, draft_probs, draft_tokens, parent, node_offsets,
                      uniforms, retained_mask, accepted_len, path, bonus_token, status, debug_pq,
                      workspace, workspace_bytes, stream);
}

int tv_accept_ex(const tv_accept_params* p, const tv_accept_options* opt, const float* target,
                 const float* draft_probs, const int32_t* draft_tokens, const int32_t* parent,
                 const int32_t* node_offsets, const float* uniforms,
                 const uint32_t* retained_mask, int32_t* accepted_len, int32_t* path,
                 int32_t* bonus_token, int32_t* status, float* debug_pq, void* workspace,
                 size_t workspace_bytes, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (opt && opt->test != TV_TEST_RATIO && opt->test != TV_TEST_LOG_CLAMP &&
      opt->test != TV_TEST_MULTI)
    return TV_ERR_INVALID_ARG;
  if (opt && !(opt->log_clamp >= 0.0f && opt->log_clamp <= 88.0f)) return TV_ERR_INVALID_ARG;
  if (opt && opt->gamma && !aligned16(opt->gamma)) return TV_ERR_INVALID_ARG;
  if (p->batch < 1 || p->vocab < 1 || p->vocab >= (1 << 18)) return TV_ERR_INVALID_ARG;
  if (p->max_nodes < 1 || p->max_nodes > TV_MAX_NODES || p->max_nodes > tv::accept_max_nodes())
    return TV_ERR_INVALID_ARG;
  if (p->kind != TV_INPUT_PROBS && p->kind != TV_INPUT_LOGITS) return TV_ERR_INVALID_ARG;
  if (p->total_nodes < p->batch) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {target, draft_probs, draft_tokens, parent, node_offsets, uniforms,
                        accepted_len, path, bonus_token, status};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  if ((retained_mask && !aligned16(retained_mask)) || (debug_pq && !aligned16(debug_pq)))
    return TV_ERR_INVALID_ARG;
  tv::AcceptArgs a;
  a.target = target;
  a.draft = draft_probs;
  a.tokens = draft_tokens;
  a.parent = parent;
  a.node_offsets = node_offsets;
  a.uniforms = uniforms;
  a.mask = retained_mask;
  a.accepted_len = accepted_len;
  a.path = path;
  a.bonus_token = bonus_token;
  a.status = status;
  a.debug_pq = debug_pq;
  a.vocab = p->vocab;
  a.max_nodes = p->max_nodes;
  a.kind = p->kind;
  a.batch = p->batch;
  a.total_nodes = p->total_nodes;
  a.test = opt ? opt->test : TV_TEST_RATIO;
  a.log_clamp = (opt && opt->log_clamp > 0.0f) ? opt->log_clamp : 20.0f;
  a.gamma = opt ? opt->gamma : nullptr;
  // per-row statistics (logits input or a retained-set mask) need workspace
  if (p->kind == TV_INPUT_LOGITS || retained_mask) {
    const size_t need = tv::accept_workspace_bytes(p->vocab, p->total_nodes);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return TV_ERR_WORKSPACE;
  }
  if (tv::launch_accept(a, workspace, stream) != 0) return TV_ERR_CUDA;
  return TV_OK;
}

}  // extern "C"

namespace {

// The shared path of tv_commit_kv and tv_commit_kv_fp8 (k_scale non-null).
int commit_call(const tv_commit_params* p, const void* k_nodes, const float* k_nodes_scale,
                const void* v_nodes, const float* v_nodes_scale, const int32_t* parent,
                const int32_t* node_offsets, const int32_t* accepted_len, const int32_t* path,
                const int32_t* block_table, const int32_t* prefix_lens, void* k_pool,
                float* k_scale, void* v_pool, float* v_scale, int32_t* new_prefix_lens,
                int32_t* status, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->batch < 1 || p->num_kv_heads < 1 || p->block_size != TV_BLOCK_SIZE ||
      p->max_blocks_per_seq < 1 || p->num_blocks < 1 || p->max_nodes < 1 ||
      p->max_nodes > TV_MAX_NODES || p->total_nodes < p->batch)
    return TV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->num_blocks) * p->num_kv_heads * 16 >= (1ll << 31))
    return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {k_nodes, v_nodes, parent, node_offsets, accepted_len, path,
                        block_table, prefix_lens, k_pool, v_pool, new_prefix_lens, status};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  if (static_cast<const void*>(new_prefix_lens) == static_cast<const void*>(prefix_lens))
    return TV_ERR_INVALID_ARG;
  tv::CommitArgs a;
  a.k_nodes = k_nodes;
  a.v_nodes = v_nodes;
  a.k_nodes_scale = k_nodes_scale;
  a.v_nodes_scale = v_nodes_scale;
  a.parent = parent;
  a.node_offsets = node_offsets;
  a.accepted_len = accepted_len;
  a.path = path;
  a.block_table = block_table;
  a.prefix_lens = prefix_lens;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.new_prefix_lens = new_prefix_lens;
  a.status = status;
  a.batch = p->batch;
  a.hkv = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.max_nodes = p->max_nodes;
  a.total_nodes = p->total_nodes;
  return tv::launch_commit(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

int tv_commit_kv(const tv_commit_params* p, const uint16_t* k_nodes, const uint16_t* v_nodes,
                 const int32_t* parent, const int32_t* node_offsets, const int32_t* accepted_len,
                 const int32_t* path, const int32_t* block_table, const int32_t* prefix_lens,
                 uint16_t* k_prefix_blocks, uint16_t* v_prefix_blocks, int32_t* new_prefix_lens,
                 int32_t* status, cudaStream_t stream) {
  return commit_call(p, k_nodes, nullptr, v_nodes, nullptr, parent, node_offsets, accepted_len, path,
                     block_table, prefix_lens, k_prefix_blocks, nullptr, v_prefix_blocks, nullptr,
                     new_prefix_lens, status, stream);
}

int tv_commit_kv_fp8(const tv_commit_params* p, const uint8_t* k_nodes, const float* k_nodes_scale,
                     const uint8_t* v_nodes, const float* v_nodes_scale, const int32_t* parent,
                     const int32_t* node_offsets, const int32_t* accepted_len,
                     const int32_t* path, const int32_t* block_table, const int32_t* prefix_lens,
                     uint8_t* k_prefix_blocks, float* k_prefix_scale, uint8_t* v_prefix_blocks,
                     float* v_prefix_scale, int32_t* new_prefix_lens, int32_t* status,
                     cudaStream_t stream) {
  const void* sc[] = {k_nodes_scale, v_nodes_scale, k_prefix_scale, v_prefix_scale};
  for (const void* q : sc)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  return commit_call(p, k_nodes, k_nodes_scale, v_nodes, v_nodes_scale, parent, node_offsets,
                     accepted_len, path, block_table, prefix_lens, k_prefix_blocks, k_prefix_scale,
                     v_prefix_blocks, v_prefix_scale, new_prefix_lens, status, stream);
}

int tv_retained_set(const tv_retain_params* p, const float* draft_probs, uint32_t* retained_mask,
                    uint64_t* z_fixed, float* z, int32_t* kept, cudaStream_t stream) {
  if (!p || p->rows < 1 || p->rows > 65535 || p->vocab < 1 || p->vocab > (1 << 18))
    return TV_ERR_INVALID_ARG;
  if (!(p->mass >= 0x1p-40f && p->mass <= 32.0f)) return TV_ERR_INVALID_ARG;  // NaN fails too
  if (!draft_probs || !retained_mask || !aligned16(draft_probs) || !aligned16(retained_mask))
    return TV_ERR_INVALID_ARG;
  if ((z_fixed && !aligned16(z_fixed)) || (z && !aligned16(z)) || (kept && !aligned16(kept)))
    return TV_ERR_INVALID_ARG;
  tv::RetainArgs a;
  a.draft = draft_probs;
  a.mask = retained_mask;
  a.z_fixed = reinterpret_cast<unsigned long long*>(z_fixed);
  a.z = z;
  a.kept = kept;
  a.threshold = static_cast<unsigned long long>(std::floor(static_cast<double>(p->mass) * 0x1p40));
  a.rows = p->rows;
  a.vocab = p->vocab;
  if (a.threshold < 1) return TV_ERR_INVALID_ARG;
  return tv::launch_retained_set(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

size_t tv_chunk_attention_workspace_size(const tv_chunk_params* p) {
  ChunkPlan pl;
  if (!plan_chunk(p, sm_count(), &pl)) return 0;
  return pl.workspace;
}

namespace {

// The shared path of tv_chunk_attention and tv_chunk_attention_fp8 (q_scale
// non-null): checks, tensor maps, arguments and the launch.
int chunk_call(const tv_chunk_params* p, bool fp8, const void* q, const float* q_scale,
               const void* k_pool, const float* k_scale, const void* v_pool, const float* v_scale,
               const int32_t* block_table, const int32_t* seq_lens, const int32_t* token_offsets,
               void* out, int32_t* status, void* workspace, size_t workspace_bytes,
               cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (fp8 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->num_kv_heads > 0 && p->num_q_heads / p->num_kv_heads > 256) return TV_ERR_UNSUPPORTED;
  ChunkPlan pl;
  if (!plan_chunk(p, sm_count(), &pl)) return TV_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(p->num_q_heads) * p->head_dim;
  const int64_t elem = fp8 ? 1 : 2;
  const int64_t stride = p->q_stride ? p->q_stride : row;
  if (stride < row || stride >= (1ll << 38) || stride * elem % 16) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {k_pool, v_pool, block_table, seq_lens, token_offsets, status};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return TV_ERR_INVALID_ARG;
  if (p->total_tokens > 0 && (!q || !out)) return TV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out)) return TV_ERR_INVALID_ARG;
  if (fp8) {
    if (p->total_tokens > 0 && !q_scale) return TV_ERR_INVALID_ARG;
    if (!k_scale || !v_scale || !aligned16(q_scale) || !aligned16(k_scale) || !aligned16(v_scale))
      return TV_ERR_INVALID_ARG;
  }
  if (!workspace || workspace_bytes < pl.workspace || !aligned16(workspace))
    return TV_ERR_WORKSPACE;
  tv::ChunkMaps maps;
  const uint64_t pages = static_cast<uint64_t>(p->num_blocks) * p->num_kv_heads;
  if (!encode_pool(&maps.k_pool, k_pool, p->head_dim, pages, fp8) ||
      !encode_pool(&maps.v_pool, v_pool, p->head_dim, pages, fp8))
    return TV_ERR_CUDA;
  tv::ChunkArgs a;
  std::memset(&a, 0, sizeof a);
  a.q_tokens = std::min(pl.unit_tokens, p->total_tokens);
  if (p->total_tokens > 0) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p->head_dim), static_cast<cuuint64_t>(p->num_q_heads),
                                static_cast<cuuint64_t>(p->total_tokens)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(p->head_dim * elem), static_cast<cuuint64_t>(stride * elem)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem),
                               static_cast<cuuint32_t>(p->num_q_heads / p->num_kv_heads),
                               static_cast<cuuint32_t>(a.q_tokens)};
    if (!encode(&maps.q, q, 3, dims, str, box,
                fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16))
      return TV_ERR_CUDA;
  }
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.token_offsets = token_offsets;
  a.out = out;
  a.status = status;
  a.counters = static_cast<int32_t*>(workspace);
  a.slots = static_cast<uint8_t*>(workspace) + (static_cast<size_t>(pl.vctas) * 4 + 255) / 256 * 256;
  a.batch = p->batch;
  a.hq = p->num_q_heads;
  a.hkv = p->num_kv_heads;
  a.group = p->num_q_heads / p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.max_len = p->max_len;
  a.total_tokens = p->total_tokens;
  a.unit_tokens = pl.unit_tokens;
  a.vctas = pl.vctas;
  a.min_range = kMinRange;
  // a window of max_len or more hides nothing; neither count overflows in the kernel
  a.window = p->window >= p->max_len ? 0 : p->window;
  a.sinks = std::min(p->sinks, p->max_len);
  a.out_fp32 = p->out_dtype == TV_OUT_FP32 ? 1 : 0;
  a.fp8 = fp8 ? 1 : 0;
  const float scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(p->head_dim));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q_scale = q_scale;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return tv::launch_chunk_attention(a, maps, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

int tv_chunk_attention(const tv_chunk_params* p, const uint16_t* q, const uint16_t* k_pool,
                       const uint16_t* v_pool, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* token_offsets, void* out,
                       int32_t* status, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  return chunk_call(p, false, q, nullptr, k_pool, nullptr, v_pool, nullptr, block_table, seq_lens,
                    token_offsets, out, status, workspace, workspace_bytes, stream);
}

int tv_chunk_attention_fp8(const tv_chunk_params* p, const uint8_t* q, const float* q_scale,
                           const uint8_t* k_pool, const float* k_scale, const uint8_t* v_pool,
                           const float* v_scale, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* token_offsets, void* out,
                           int32_t* status, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  return chunk_call(p, true, q, q_scale, k_pool, k_scale, v_pool, v_scale, block_table, seq_lens,
                    token_offsets, out, status, workspace, workspace_bytes, stream);
}

namespace {

// The shared path of tv_append_kv, tv_append_kv_fp8 and tv_read_kv_fp8.
int cache_call(const tv_cache_params* p, bool read, const void* k_new, const void* v_new,
               const int32_t* block_table, const int32_t* seq_lens, const int32_t* token_offsets,
               const void* k_pool, const float* k_scale, const void* v_pool, const float* v_scale,
               bool fp8, int32_t* status, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->batch < 1 || p->num_kv_heads < 1 || p->block_size != TV_BLOCK_SIZE ||
      p->max_blocks_per_seq < 1 || p->num_blocks < 1 || p->total_tokens < 0)
    return TV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->num_blocks) * p->num_kv_heads * 16 >= (1ll << 31))
    return TV_ERR_INVALID_ARG;
  if (p->num_kv_heads >= (1 << 24) || static_cast<int64_t>(p->total_tokens) * p->num_kv_heads >= (1ll << 31))
    return TV_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  const int64_t stride = p->kv_stride ? p->kv_stride : row;
  if (stride < row || stride >= (1ll << 38) || stride % 8) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {block_table, seq_lens, token_offsets, k_pool, v_pool, status};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  if (p->total_tokens > 0 && (!k_new || !v_new)) return TV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new)) return TV_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale || !aligned16(k_scale) || !aligned16(v_scale)))
    return TV_ERR_INVALID_ARG;
  tv::CacheArgs a;
  a.k_new = const_cast<void*>(k_new);
  a.v_new = const_cast<void*>(v_new);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.token_offsets = token_offsets;
  a.k_pool = const_cast<void*>(k_pool);
  a.v_pool = const_cast<void*>(v_pool);
  a.k_scale = const_cast<float*>(k_scale);
  a.v_scale = const_cast<float*>(v_scale);
  a.status = status;
  a.kv_stride = static_cast<size_t>(stride);
  a.batch = p->batch;
  a.hkv = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.max_blocks_per_seq = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.total_tokens = p->total_tokens;
  a.read = read ? 1 : 0;
  a.tile_shift = 0;
  return tv::launch_cache(a, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

int tv_append_kv(const tv_cache_params* p, const uint16_t* k_new, const uint16_t* v_new,
                 const int32_t* block_table, const int32_t* seq_lens,
                 const int32_t* token_offsets, uint16_t* k_pool, uint16_t* v_pool,
                 int32_t* status, cudaStream_t stream) {
  return cache_call(p, false, k_new, v_new, block_table, seq_lens, token_offsets, k_pool, nullptr,
                    v_pool, nullptr, false, status, stream);
}

int tv_append_kv_fp8(const tv_cache_params* p, const uint16_t* k_new, const uint16_t* v_new,
                     const int32_t* block_table, const int32_t* seq_lens,
                     const int32_t* token_offsets, uint8_t* k_pool, float* k_scale,
                     uint8_t* v_pool, float* v_scale, int32_t* status, cudaStream_t stream) {
  return cache_call(p, false, k_new, v_new, block_table, seq_lens, token_offsets, k_pool, k_scale,
                    v_pool, v_scale, true, status, stream);
}

int tv_read_kv_fp8(const tv_cache_params* p, const uint8_t* k_pool, const float* k_scale,
                   const uint8_t* v_pool, const float* v_scale, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* token_offsets, uint16_t* k_out,
                   uint16_t* v_out, int32_t* status, cudaStream_t stream) {
  return cache_call(p, true, k_out, v_out, block_table, seq_lens, token_offsets, k_pool, k_scale,
                    v_pool, v_scale, true, status, stream);
}

int tv_quantize_rows(const tv_quant_params* p, const uint16_t* x, uint8_t* codes, float* scale,
                     cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->tokens < 0 || p->heads < 1) return TV_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(p->heads) * p->head_dim;
  const int64_t stride = p->stride ? p->stride : row;
  if (stride < row || stride >= (1ll << 38) || stride % 8) return TV_ERR_INVALID_ARG;
  if (p->tokens == 0) return TV_OK;
  const void* ptrs[] = {x, codes, scale};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  tv::QuantArgs a;
  a.x = x;
  a.codes = codes;
  a.scale = scale;
  a.stride = static_cast<size_t>(stride);
  a.tokens = p->tokens;
  a.heads = p->heads;
  a.head_dim = p->head_dim;
  return tv::launch_quantise_rows(a, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

int tv_penalize_logits(const tv_penalty_params* p, const void* logits,
                       const int32_t* draft_tokens, const int32_t* parent,
                       const int32_t* node_offsets, const int32_t* history,
                       const int32_t* history_offsets, const int32_t* prompt_lens,
                       const float* repetition, const float* presence, const float* frequency,
                       const int32_t* bias_ids, const float* bias_values,
                       const int32_t* bias_offsets, const uint32_t* allowed_mask, float* out,
                       int32_t* status, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->batch < 1 || p->batch > 65535 || p->vocab < 1 || p->vocab >= (1 << 18)) return TV_ERR_INVALID_ARG;
  if (p->max_nodes < 1 || p->max_nodes > TV_MAX_NODES || p->total_nodes < p->batch) return TV_ERR_INVALID_ARG;
  if (p->logits_dtype != TV_OUT_BF16 && p->logits_dtype != TV_OUT_FP32) return TV_ERR_INVALID_ARG;
  if (p->total_history < 0 || p->total_history > (1 << 30) || p->total_bias < 0 || p->total_bias > (1 << 30))
    return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {logits, draft_tokens, parent, node_offsets, out, status};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return TV_ERR_INVALID_ARG;
  const void* optional[] = {history, history_offsets, prompt_lens, repetition, presence, frequency,
                            bias_ids, bias_values, bias_offsets, allowed_mask};
  for (const void* q : optional)
    if (q && !aligned16(q)) return TV_ERR_INVALID_ARG;
  if (history && !history_offsets) return TV_ERR_INVALID_ARG;
  if (bias_ids && (!bias_values || !bias_offsets)) return TV_ERR_INVALID_ARG;
  // in place with fp32 logits, which no other row's output may lie over (a bf16
  // row is half as long as its output)
  const uint64_t entries = static_cast<uint64_t>(p->total_nodes) * p->vocab;
  const uint64_t in0 = reinterpret_cast<uintptr_t>(logits), out0 = reinterpret_cast<uintptr_t>(out);
  const bool bf16 = p->logits_dtype == TV_OUT_BF16;
  if ((bf16 || in0 != out0) && in0 < out0 + entries * 4 && out0 < in0 + entries * (bf16 ? 2 : 4))
    return TV_ERR_INVALID_ARG;
  tv::PenaltyArgs a;
  a.logits = logits;
  a.out = out;
  a.tokens = draft_tokens;
  a.parent = parent;
  a.node_offsets = node_offsets;
  // an empty list may have no address, but its extents are checked
  a.history = history;
  a.history_offsets = history || p->total_history == 0 ? history_offsets : nullptr;
  a.prompt_lens = prompt_lens;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.bias_offsets = bias_ids || p->total_bias == 0 ? bias_offsets : nullptr;
  a.allowed_mask = allowed_mask;
  a.status = status;
  a.batch = p->batch;
  a.vocab = p->vocab;
  a.max_nodes = p->max_nodes;
  a.total_nodes = p->total_nodes;
  a.total_history = p->total_history;
  a.total_bias = p->total_bias;
  a.bf16 = p->logits_dtype == TV_OUT_BF16 ? 1 : 0;
  return tv::launch_penalty(a, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

namespace {

// The bytes [p, p + n) and [q, q + m) have some in common.
bool overlap(const void* p, uint64_t n, const void* q, uint64_t m) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n && m && a < b + m && b < a + n;
}

struct Span {
  const void* p;
  uint64_t bytes;
};
// Some output has bytes in common with an input or with another output.
template <size_t N, size_t M>
bool clash(const Span (&outs)[N], const Span (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j)
      if (outs[i].p && outs[j].p && overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
    for (size_t j = 0; j < M; ++j)
      if (outs[i].p && ins[j].p && overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
  }
  return false;
}

// Rows of `row` elements, `stride` apart.
struct RowSpan {
  const uint16_t* p;
  int64_t row, stride;
};
// Some element of `rows` rows of x lies in one of y.  Rows of one stride that
// interleave (the slices of a fused projection) do not, if they miss each other
// within a stride.
bool rows_overlap(const RowSpan& x, const RowSpan& y, int64_t rows) {
  const uint64_t n = static_cast<uint64_t>((rows - 1) * x.stride + x.row) * 2;
  const uint64_t m = static_cast<uint64_t>((rows - 1) * y.stride + y.row) * 2;
  if (!overlap(x.p, n, y.p, m)) return false;
  if (x.stride != y.stride) return true;
  const int64_t bytes = reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p);
  if (bytes % 2) return true;
  const int64_t apart = ((bytes / 2) % x.stride + x.stride) % x.stride;
  return apart < x.row || apart + y.row > x.stride;
}

}  // namespace

int tv_rotate_qk(const tv_rotate_params* p, const uint16_t* q, const uint16_t* k,
                 const void* q_weight, const void* k_weight, const int32_t* positions,
                 const double* frequencies, uint16_t* q_out, uint16_t* k_out,
                 cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->tokens < 0 || p->tokens > (1 << 30) || p->num_q_heads < 1 || p->num_kv_heads < 0) return TV_ERR_INVALID_ARG;
  if (p->num_q_heads > (1 << 20) || p->num_kv_heads > (1 << 20)) return TV_ERR_INVALID_ARG;
  const int64_t heads = static_cast<int64_t>(p->num_q_heads) + p->num_kv_heads;
  if (p->tokens * heads >= (1ll << 40)) return TV_ERR_INVALID_ARG;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 2) return TV_ERR_INVALID_ARG;
  if (p->interleaved != 0 && p->interleaved != 1) return TV_ERR_INVALID_ARG;
  if (p->num_axes < 1 || p->num_axes > TV_MAX_POSITION_AXES) return TV_ERR_INVALID_ARG;
  if (p->weight_dtype != TV_OUT_BF16 && p->weight_dtype != TV_OUT_FP32) return TV_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f && p->eps <= FLT_MAX) || !(p->scale >= 0.0f && p->scale <= FLT_MAX)) return TV_ERR_INVALID_ARG;
  for (int i = 0; i < p->rotary_dim / 2; ++i)
    if (p->axis_of_pair[i] >= p->num_axes) return TV_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(p->num_q_heads) * p->head_dim;
  const int64_t k_row = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  const int64_t strides[4] = {p->q_stride ? p->q_stride : q_row, p->k_stride ? p->k_stride : k_row,
                              p->q_out_stride ? p->q_out_stride : q_row, p->k_out_stride ? p->k_out_stride : k_row};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < (i % 2 ? k_row : q_row) || strides[i] >= (1ll << 38) || strides[i] % 8) return TV_ERR_INVALID_ARG;
  if (p->tokens == 0) return TV_OK;
  const bool keys = p->num_kv_heads > 0;
  if (!q || !q_out || (keys && (!k || !k_out))) return TV_ERR_INVALID_ARG;
  if (p->rotary_dim > 0 && (!positions || !frequencies)) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, q_weight, k_weight, positions, frequencies, q_out, k_out};
  for (const void* x : ptrs)
    if (!aligned16(x)) return TV_ERR_INVALID_ARG;
  const RowSpan qs{q, q_row, strides[0]}, ks{k, k_row, strides[1]}, qo{q_out, q_row, strides[2]}, ko{k_out, k_row, strides[3]};
  const bool q_here = q == q_out && strides[0] == strides[2], k_here = k == k_out && strides[1] == strides[3];
  if (!q_here && rows_overlap(qs, qo, p->tokens)) return TV_ERR_INVALID_ARG;
  if (keys && ((!k_here && rows_overlap(ks, ko, p->tokens)) || rows_overlap(qo, ko, p->tokens) ||
               rows_overlap(qs, ko, p->tokens) || rows_overlap(ks, qo, p->tokens)))
    return TV_ERR_INVALID_ARG;
  const uint64_t weight = p->head_dim * (p->weight_dtype == TV_OUT_FP32 ? 4ull : 2ull);
  const auto all_rows = [&](const RowSpan& x) { return static_cast<uint64_t>((p->tokens - 1) * x.stride + x.row) * 2; };
  const Span small[] = {{q_weight, weight}, {keys ? k_weight : nullptr, weight},
                        {p->rotary_dim > 0 ? positions : nullptr, static_cast<uint64_t>(p->num_axes) * p->tokens * 4},
                        {frequencies, p->rotary_dim * 4ull}};
  if (clash({{q_out, all_rows(qo)}}, small) || (keys && clash({{k_out, all_rows(ko)}}, small))) return TV_ERR_INVALID_ARG;
  tv::RotateArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = q;
  a.k = k;
  a.q_weight = q_weight;
  a.k_weight = keys ? k_weight : nullptr;
  a.positions = positions;
  a.frequencies = frequencies;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = static_cast<size_t>(strides[0]);
  a.k_stride = static_cast<size_t>(strides[1]);
  a.q_out_stride = static_cast<size_t>(strides[2]);
  a.k_out_stride = static_cast<size_t>(strides[3]);
  a.tokens = p->tokens;
  a.hq = p->num_q_heads;
  a.hkv = p->num_kv_heads;
  a.head_dim = p->head_dim;
  a.rotary_dim = p->rotary_dim;
  a.axes = p->num_axes;
  a.interleaved = p->interleaved;
  a.weight_fp32 = p->weight_dtype == TV_OUT_FP32 ? 1 : 0;
  a.eps = p->eps;
  a.scale = p->scale > 0.0f ? p->scale : 1.0f;
  std::memcpy(a.axis, p->axis_of_pair, sizeof a.axis);
  return tv::launch_rotate(a, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

namespace {

bool beam_valid(const tv_beam_params* p) {
  if (!p || p->batch < 1 || p->batch > 65535 || p->vocab < 1 || p->vocab >= (1 << 18)) return false;
  if (p->beams < 1 || p->beams > tv::beam_max_beams() || p->select < 1 || p->select > tv::beam_max_select()) return false;
  if (p->logits_dtype != TV_OUT_BF16 && p->logits_dtype != TV_OUT_FP32) return false;
  if (p->end_token < -1 || p->end_token >= p->vocab) return false;
  if (!(p->length_penalty >= -4.0f && p->length_penalty <= 4.0f)) return false;  // NaN fails too
  return p->logits_stride == 0 || (p->logits_stride >= p->vocab && p->logits_stride < (1ll << 38));
}

// The sizes and parts of a call, and the bytes of its workspace: the parts' maxima
// and sums and the rows' factors (whole 256 each), and all.
tv::BeamArgs beam_args(const tv_beam_params* p, size_t* stats, size_t* factors, size_t* bytes) {
  tv::BeamArgs a;
  std::memset(&a, 0, sizeof a);
  a.stride = static_cast<size_t>(p->logits_stride ? p->logits_stride : p->vocab);
  a.batch = p->batch;
  a.beams = p->beams;
  a.select = p->select;
  a.vocab = p->vocab;
  a.bf16 = p->logits_dtype == TV_OUT_BF16 ? 1 : 0;
  a.end_token = p->end_token;
  a.length_penalty = p->length_penalty;
  tv::plan_beam_parts(a, sm_count());
  const size_t parts = static_cast<size_t>(p->batch) * p->beams * a.parts;
  *stats = (parts * 8 + 255) / 256 * 256;
  *factors = (static_cast<size_t>(p->batch) * p->beams * 8 + 255) / 256 * 256;
  *bytes = *stats + *factors + parts * p->select * 8;
  return a;
}

}  // namespace

size_t tv_beam_select_workspace_size(const tv_beam_params* p) {
  if (!beam_valid(p)) return 0;
  size_t stats, factors, bytes;
  beam_args(p, &stats, &factors, &bytes);
  return bytes;
}

int tv_beam_select(const tv_beam_params* p, const void* logits, const float* scores,
                   const int32_t* lengths, const int32_t* finished, int32_t* tokens,
                   int32_t* parents, float* scores_out, int32_t* lengths_out,
                   int32_t* finished_out, int32_t* status, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  if (!beam_valid(p)) return TV_ERR_INVALID_ARG;
  const void* ptrs[] = {logits, scores, tokens, parents, scores_out, status};
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return TV_ERR_INVALID_ARG;
  const void* optional[] = {lengths, finished, lengths_out, finished_out};
  for (const void* x : optional)
    if (!aligned16(x)) return TV_ERR_INVALID_ARG;
  if (!lengths && (lengths_out || p->length_penalty != 0.0f)) return TV_ERR_INVALID_ARG;
  // (a request's merge reads its input while another's writes)
  const uint64_t in = static_cast<uint64_t>(p->batch) * p->beams * 4, out = static_cast<uint64_t>(p->batch) * p->select * 4;
  size_t stats, factors, bytes;
  tv::BeamArgs a = beam_args(p, &stats, &factors, &bytes);
  const uint64_t x = ((static_cast<uint64_t>(p->batch) * p->beams - 1) * a.stride + p->vocab) * (a.bf16 ? 2 : 4);
  if (clash({{tokens, out}, {parents, out}, {scores_out, out}, {lengths_out, out}, {finished_out, out}, {status, p->batch * 4ull},
             {workspace, bytes}},
            {{logits, x}, {scores, in}, {lengths, in}, {finished, in}}))
    return TV_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < bytes || !aligned16(workspace)) return TV_ERR_WORKSPACE;
  a.logits = logits;
  a.scores = scores;
  a.lengths = lengths;
  a.finished = finished;
  a.tokens = tokens;
  a.parents = parents;
  a.scores_out = scores_out;
  a.lengths_out = lengths_out;
  a.finished_out = finished_out;
  a.status = status;
  a.stats = static_cast<float2*>(workspace);
  a.power = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + stats);
  a.lists = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + stats + factors);
  return tv::launch_beam_select(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

namespace {

bool pages_valid(const tv_page_params* p) {
  return p && p->rows >= 1 && p->rows <= 65536 && p->block_size == TV_BLOCK_SIZE && p->max_blocks_per_seq >= 1 &&
         p->max_blocks_per_seq <= (1 << 27) && p->num_blocks >= 1 && p->num_blocks <= (1 << 30) &&
         static_cast<int64_t>(p->rows) * p->max_blocks_per_seq < (1ll << 31);  // needs are summed in 32 bits
}

tv::PageArgs page_args(const tv_page_params* p, const int32_t* block_table, const int32_t* ref_counts, int32_t* status) {
  tv::PageArgs a;
  std::memset(&a, 0, sizeof a);
  a.block_table = const_cast<int32_t*>(block_table);
  a.ref_counts = const_cast<int32_t*>(ref_counts);
  a.status = status;
  a.rows = p->rows;
  a.width = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  return a;
}

// Bytes of the workspace's first two parts, whole 256 each: free pages in order, and
// the first child of every row; the counts of the pool's segments and, of a large
// pool, the needs of pieces of rows follow.
size_t page_list_bytes(const tv_page_params* p) { return (static_cast<size_t>(p->num_blocks) * 4 + 255) / 256 * 256; }
size_t page_first_bytes(const tv_page_params* p) { return (static_cast<size_t>(p->rows) * 4 + 255) / 256 * 256; }
size_t page_need_bytes(const tv_page_params* p) { return p->num_blocks < tv::kManyPages ? 0 : static_cast<size_t>(p->rows) * tv::kMaxCuts * 4; }
void page_workspace(const tv_page_params* p, void* workspace, tv::PageArgs* a) {
  uint8_t* at = static_cast<uint8_t*>(workspace);
  a->list = reinterpret_cast<int32_t*>(at);
  a->first = reinterpret_cast<int32_t*>(at + page_list_bytes(p));
  a->counts = reinterpret_cast<int32_t*>(at + page_list_bytes(p) + page_first_bytes(p));
  a->needs = a->counts + tv::kPageSegments;
}

template <size_t N>
bool all_given(const void* const (&ptrs)[N]) {
  for (const void* x : ptrs)
    if (!x || !aligned16(x)) return false;
  return true;
}

}  // namespace

size_t tv_pages_workspace_size(const tv_page_params* p) {
  return pages_valid(p) ? page_list_bytes(p) + page_first_bytes(p) + tv::kPageSegments * 4 + page_need_bytes(p) : 0;
}

int tv_alloc_pages(const tv_page_params* p, int32_t* block_table, int32_t* ref_counts,
                   const int32_t* begin, const int32_t* end, int32_t* status, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  if (!pages_valid(p)) return TV_ERR_INVALID_ARG;
  if (!all_given({block_table, ref_counts, end, status}) || !aligned16(begin)) return TV_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < tv_pages_workspace_size(p) || !aligned16(workspace)) return TV_ERR_WORKSPACE;
  const uint64_t word = static_cast<uint64_t>(p->rows) * 4;
  if (clash({{block_table, word * p->max_blocks_per_seq}, {ref_counts, p->num_blocks * 4ull}, {status, word},
             {workspace, tv_pages_workspace_size(p)}},
            {{begin, word}, {end, word}}))
    return TV_ERR_INVALID_ARG;
  tv::PageArgs a = page_args(p, block_table, ref_counts, status);
  a.begin = begin;
  a.end = end;
  page_workspace(p, workspace, &a);
  return tv::launch_alloc_pages(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

int tv_free_pages(const tv_page_params* p, int32_t* block_table, int32_t* ref_counts,
                  const int32_t* keep_begin, const int32_t* keep_end, int32_t* status,
                  cudaStream_t stream) {
  if (!pages_valid(p) || p->sinks < 0) return TV_ERR_INVALID_ARG;
  if (!all_given({block_table, ref_counts, status}) || !aligned16(keep_begin) || !aligned16(keep_end))
    return TV_ERR_INVALID_ARG;
  const uint64_t word = static_cast<uint64_t>(p->rows) * 4;
  if (clash({{block_table, word * p->max_blocks_per_seq}, {ref_counts, p->num_blocks * 4ull}, {status, word}},
            {{keep_begin, word}, {keep_end, word}}))
    return TV_ERR_INVALID_ARG;
  tv::PageArgs a = page_args(p, block_table, ref_counts, status);
  a.keep_begin = keep_begin;
  a.keep_end = keep_end;
  a.sinks = p->sinks;
  return tv::launch_free_pages(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

int tv_fork_pages(const tv_page_params* p, const int32_t* block_table,
                  const int32_t* seq_lens, const int32_t* parents, int32_t* ref_counts,
                  int32_t* block_table_out, int32_t* seq_lens_out, int32_t* copies,
                  int32_t* status, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  if (!pages_valid(p) || p->new_rows < 1 || p->new_rows > 65536) return TV_ERR_INVALID_ARG;
  if (!all_given({block_table, seq_lens, parents, ref_counts, block_table_out, seq_lens_out, copies, status}))
    return TV_ERR_INVALID_ARG;
  const uint64_t row = static_cast<uint64_t>(p->max_blocks_per_seq) * 4, rows = p->rows, children = p->new_rows;
  if (clash({{ref_counts, p->num_blocks * 4ull}, {block_table_out, children * row}, {seq_lens_out, children * 4},
             {copies, children * 12}, {status, children * 4}, {workspace, tv_pages_workspace_size(p)}},
            {{block_table, rows * row}, {seq_lens, rows * 4}, {parents, children * 4}}))
    return TV_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < tv_pages_workspace_size(p) || !aligned16(workspace)) return TV_ERR_WORKSPACE;
  tv::PageArgs a = page_args(p, block_table, ref_counts, status);
  a.new_rows = p->new_rows;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.table_out = block_table_out;
  a.lens_out = seq_lens_out;
  a.copies = copies;
  page_workspace(p, workspace, &a);
  return tv::launch_fork_pages(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

int tv_compact_pages(const tv_page_params* p, const int32_t* block_table,
                     const int32_t* ref_counts, int32_t* block_table_out,
                     int32_t* ref_counts_out, int32_t* page_map, int32_t* moves,
                     int32_t* count, int32_t* status, cudaStream_t stream) {
  if (!pages_valid(p)) return TV_ERR_INVALID_ARG;
  if (!all_given({block_table, ref_counts, block_table_out, ref_counts_out, page_map, moves, count, status}))
    return TV_ERR_INVALID_ARG;
  const uint64_t table = static_cast<uint64_t>(p->rows) * p->max_blocks_per_seq * 4, pages = p->num_blocks * 4ull;
  const uint64_t move_bytes = (p->num_blocks > 1 ? p->num_blocks / 2 : 1) * 12ull;
  if (clash({{block_table_out, table}, {ref_counts_out, pages}, {page_map, pages}, {moves, move_bytes}, {count, 8},
             {status, p->rows * 4ull}},
            {{block_table == block_table_out ? nullptr : block_table, table},
             {ref_counts == ref_counts_out ? nullptr : ref_counts, pages}}))
    return TV_ERR_INVALID_ARG;
  tv::PageArgs a = page_args(p, block_table, ref_counts, status);
  a.table_out = block_table_out;
  a.refs_out = ref_counts_out;
  a.page_map = page_map;
  a.copies = moves;
  a.count = count;
  return tv::launch_compact_pages(a, stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

namespace {

// The shared path of tv_copy_pages and tv_copy_pages_fp8 (scales given).
int copy_call(const tv_copy_params* p, const int32_t* copies, const int32_t* count, bool fp8, void* k_pool,
              float* k_scale, void* v_pool, float* v_scale, int32_t* status, cudaStream_t stream) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_ERR_UNSUPPORTED;
  if (p->entries < 0 || p->layers < 1 || p->num_kv_heads < 1 || p->block_size != TV_BLOCK_SIZE || p->num_blocks < 1)
    return TV_ERR_INVALID_ARG;
  if (p->layers > (1 << 16) || p->num_kv_heads > (1 << 16) ||
      static_cast<int64_t>(p->num_blocks) * p->num_kv_heads * 16 >= (1ll << 31))
    return TV_ERR_INVALID_ARG;
  if (p->entries == 0) return TV_OK;
  if (!all_given({copies, k_pool, v_pool}) || !aligned16(status) || reinterpret_cast<uintptr_t>(count) % 4)
    return TV_ERR_INVALID_ARG;
  if (fp8 && !all_given({k_scale, v_scale})) return TV_ERR_INVALID_ARG;
  tv::CopyArgs a;
  std::memset(&a, 0, sizeof a);
  a.copies = copies;
  a.count = count;
  a.pool[0] = k_pool;
  a.pool[1] = v_pool;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.status = status;
  a.row_bytes = p->head_dim * (fp8 ? 1 : 2);
  a.scale_stride = static_cast<size_t>(p->num_blocks) * p->num_kv_heads * 16;
  a.layer_stride = a.scale_stride * a.row_bytes;
  a.entries = p->entries;
  a.layers = p->layers;
  a.num_blocks = p->num_blocks;
  a.hkv = p->num_kv_heads;
  const uint64_t pool = a.layer_stride * p->layers, scales = fp8 ? a.scale_stride * p->layers * 4 : 0;
  if (clash({{k_pool, pool}, {v_pool, pool}, {k_scale, scales}, {v_scale, scales}, {status, p->entries * 4ull}},
            {{copies, p->entries * 12ull}, {count, 4}}))
    return TV_ERR_INVALID_ARG;
  return tv::launch_copy_pages(a, sm_count(), stream) == 0 ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

int tv_copy_pages(const tv_copy_params* p, const int32_t* copies, const int32_t* count,
                  uint16_t* k_pool, uint16_t* v_pool, int32_t* status, cudaStream_t stream) {
  return copy_call(p, copies, count, false, k_pool, nullptr, v_pool, nullptr, status, stream);
}

int tv_copy_pages_fp8(const tv_copy_params* p, const int32_t* copies, const int32_t* count,
                      uint8_t* k_pool, float* k_scale, uint8_t* v_pool, float* v_scale,
                      int32_t* status, cudaStream_t stream) {
  return copy_call(p, copies, count, true, k_pool, k_scale, v_pool, v_scale, status, stream);
}
