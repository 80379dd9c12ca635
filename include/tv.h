/*
 * tv.h -- C ABI of libtv: the target-model tree-verification step of
 * speculative decoding, on one GB300 GPU (sm_103a).
 *
 * Sources (four web pages on speculative decoding; titles abbreviated):
 *   [EC]  "端云协同推测解码中草稿模型动态生成与验证并行化：探究树形注意力机制与显存碎片整理联合加速"
 *         (edge-cloud speculative decoding; tree attention; KV defragmentation)
 *   [LLM] "端侧大模型推测解码草稿模型动态剪枝策略：详解基于重要性采样的树形验证并行加速机制"
 *         (on-device LLM draft pruning; importance-sampling correction)
 *   [MM]  "端侧多模态大模型推测解码草稿模型动态剪枝：详解基于重要性采样的树形验证并行加速策略"
 *         (on-device multimodal draft pruning; importance-sampled tree verification)
 *
 * General rules for every entry point
 *   - The caller owns every buffer.  The library allocates nothing, frees
 *     nothing and never synchronises the device or the stream; all work is
 *     enqueued on the caller's stream in order.
 *   - Pointers are DEVICE pointers unless a comment says "host".
 *   - Inputs are read only.  Outputs are fully written when the call returns
 *     TV_OK and the enqueued work completes.
 *   - Argument errors are found on the host and returned before anything is
 *     enqueued.  Data errors found on the device (a bad parent index, an
 *     out-of-range block id or token) are reported per sequence in the
 *     device-side `status` array; the kernels never trap.
 *   - Stateless and re-entrant: concurrent calls on different streams are
 *     safe when their workspaces differ.
 *
 * Tree convention (shared by both entry points)
 *   Sequence b owns tree nodes node_offsets[b] .. node_offsets[b+1]-1 of the
 *   flattened node arrays ([EC] appendix B: cumulative lengths over the
 *   flattened tree).  parent[] holds LOCAL indices (0 .. N_b-1): parent of
 *   the root (local node 0) is -1 and 0 <= parent[i] < i for i >= 1
 *   ([EC] appendix B, Tree_Parent_Idx, -1 at the root).  Node 0 is the last
 *   committed token; nodes >= 1 are draft tokens.
 */
#ifndef TV_H_
#define TV_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h> /* cudaStream_t */

#ifdef __cplusplus
extern "C" {
#endif

#define TV_VERSION 100     /* 1.0.0 */
#define TV_MAX_NODES 512   /* largest tree (nodes per sequence) */
#define TV_BLOCK_SIZE 16   /* tokens per page of the paged prefix KV pool */

typedef enum {
  TV_OK = 0,
  TV_ERR_INVALID_ARG = 1,    /* null pointer, bad size or layout (host) */
  TV_ERR_UNSUPPORTED = 2,    /* valid but not implemented (e.g. head_dim) */
  TV_ERR_WORKSPACE = 3,      /* workspace missing or smaller than required */
  TV_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
  TV_ERR_BAD_TREE = 5,       /* device: malformed tree, block id or token */
  TV_ERR_DEVICE_TIMEOUT = 6, /* device: a bounded wait ran out */
  TV_ERR_NO_PAGE = 7         /* device: no pool page for a position to commit */
} tv_status;

/* Human-readable name of a status code (static string, never NULL). */
const char* tv_status_string(int status);
/* TV_VERSION of the loaded library. */
int tv_version(void);

/* Self-test of the device-timeout path.  Every wait of the library's kernels
 * on an mbarrier is bounded (2 s); when one runs out the kernel records
 * TV_ERR_DEVICE_TIMEOUT in the sequence's status, releases what it holds and
 * returns, so the context stays usable.  This entry point enqueues one
 * kernel that waits on an mbarrier nothing ever arrives at, through the same
 * bounded wait, with the limit `limit_ns` (1 ms .. 1 s), then writes the
 * outcome: status[0] = TV_ERR_DEVICE_TIMEOUT (or TV_OK had the wait ended)
 * and waited_ns[0] = the nanoseconds it waited.  status, waited_ns: device
 * pointers (int32, uint64), 4- and 8-byte aligned.  Returns
 * TV_ERR_INVALID_ARG (nothing enqueued) for a NULL pointer or a limit out of
 * range, TV_ERR_CUDA if the launch fails, else TV_OK. */
int tv_selftest_wait_timeout(int32_t* status, unsigned long long* waited_ns,
                             unsigned long long limit_ns, cudaStream_t stream);

/* ========================================================================
 * Tree attention
 *
 * For every sequence b, tree node i (local) and query head h, with KV head
 * kvh = floor(h / (Hq/Hkv)):
 *
 *   out[n0+i][h] = sum_k softmax_k(scale * q.k_k) * v_k
 *
 * over the key list [prefix tokens 0 .. L_b-1 ; tree nodes j of sequence b]
 * where every prefix token is visible and tree node j is visible iff j is an
 * ancestor of i or j == i: the tree mask M_tree[i,j] = 0 iff j is an ancestor
 * of i or j = i, -inf otherwise ([EC] §2.2.2).  The committed prefix KV is
 * stored once in a paged pool and reached through block_table ([MM] §3.2
 * common-prefix merging; [LLM] §2.3.1 cuSeqLens + block_table).  One launch
 * handles every sequence, every head and every node ([MM] §3.2: one kernel
 * for all branches).  Inputs bf16, accumulation and softmax fp32, output bf16
 * (or fp32, out_dtype).
 * ====================================================================== */
typedef enum { TV_OUT_BF16 = 0, TV_OUT_FP32 = 1 } tv_out_dtype;

typedef struct {
  int32_t batch;              /* B >= 1                                        */
  int32_t num_q_heads;        /* Hq                                            */
  int32_t num_kv_heads;       /* Hkv; Hq % Hkv == 0                            */
  int32_t head_dim;           /* D: 64 or 128                                  */
  int32_t block_size;         /* tokens per page: must be TV_BLOCK_SIZE (16)   */
  int32_t max_blocks_per_seq; /* row stride of block_table                     */
  int32_t num_blocks;         /* pages in the pool                             */
  int32_t max_nodes;          /* upper bound of N_b (<= TV_MAX_NODES)          */
  int32_t total_nodes;        /* node_offsets[batch] (host copy)               */
  int32_t max_prefix_len;     /* upper bound of L_b (host hint for the grid)   */
  float softmax_scale;        /* 0 => 1/sqrt(D)                                */
  int32_t out_dtype;          /* tv_out_dtype of `out`: bf16 (0) or fp32 (1).
                                 The bf16 output is the fp32 result rounded
                                 once to nearest even.                         */
} tv_attn_params;             /* host struct */

/* Bytes of device workspace tv_tree_attention needs for these parameters on
 * the current device (0 if the parameters are invalid).  The workspace holds
 * two arrival counters per CTA (zeroed by every call, on the stream) and two
 * partial-result slots per CTA: when the line of key tiles is cut inside a
 * unit (256 packed rows of one sequence and KV head), every piece but the
 * last to finish leaves its unnormalised output and (max, sum) per row there,
 * and the last merges them in a fixed order.  About 2 * SMs * (256 * D * 4 + 2 KB) bytes: 40.5 MB at
 * D = 128 on 152 SMs. */
size_t tv_tree_attention_workspace_size(const tv_attn_params* params);

/* Launch plan of tv_tree_attention (host only; nothing is enqueued):
 * persistent CTAs (at most one per SM) in virtual CTAs of `lanes` CTAs, one
 * lane per m-tile pair of a layer of a (sequence, KV head); the virtual CTAs
 * share the line of key tiles (sequence, KV head, layer, tile) in equal
 * contiguous ranges of at least min_tiles tiles, computed on the device from
 * prefix_lens and node_offsets. */
typedef struct {
  int32_t ctas;            /* CTAs launched = virtual_ctas * lanes          */
  int32_t lanes;           /* CTAs per virtual CTA                          */
  int32_t virtual_ctas;    /* at most SMs / lanes                           */
  int32_t min_tiles;       /* fewest 128-key tiles per virtual CTA          */
  size_t workspace_bytes;  /* = tv_tree_attention_workspace_size on `sms`   */
} tv_attn_plan;

/* The plan for `sms` SMs (sms <= 0: the current device's count, 148 when no
 * device is visible).  Returns TV_OK, or TV_ERR_INVALID_ARG for invalid
 * parameters or a NULL `plan`. */
int tv_tree_attention_plan(const tv_attn_params* params, int32_t sms, tv_attn_plan* plan);

/* Layouts (all row-major, contiguous):
 *   q_nodes          bf16 [total_nodes][Hq][D]
 *   k_prefix_blocks  bf16 [num_blocks][Hkv][block_size][D]   (paged pool)
 *   v_prefix_blocks  bf16 [num_blocks][Hkv][block_size][D]
 *   block_table      int32 [batch][max_blocks_per_seq]: page of logical block
 *                    t/16 of sequence b; entries past ceil(L_b/16) unused
 *   k_nodes, v_nodes bf16 [total_nodes][Hkv][D]   (K/V of the tree tokens)
 *   parent           int32 [total_nodes]  local parent, -1 at each root
 *   prefix_lens      int32 [batch]        L_b >= 0 (<= max_prefix_len)
 *   node_offsets     int32 [batch+1]      cumulative node counts, N_b >= 1
 *   out              bf16 or fp32 (out_dtype) [total_nodes][Hq][D]
 *   status           int32 [batch]        per-sequence TV_OK / TV_ERR_BAD_TREE /
 *                                         TV_ERR_DEVICE_TIMEOUT (device)
 *   workspace        device bytes >= tv_tree_attention_workspace_size()
 *                    (TV_ERR_WORKSPACE otherwise); contents need no
 *                    initialisation; calls that overlap on the GPU need
 *                    distinct workspaces
 * bf16 pointers are passed as uint16_t (bf16 bit patterns).  All device
 * pointers must be 16-byte aligned.  A sequence whose tree or block ids are
 * malformed gets status TV_ERR_BAD_TREE and an all-zero output. */
int tv_tree_attention(const tv_attn_params* params, const uint16_t* q_nodes,
                      const uint16_t* k_prefix_blocks, const uint16_t* v_prefix_blocks,
                      const int32_t* block_table, const uint16_t* k_nodes,
                      const uint16_t* v_nodes, const int32_t* parent,
                      const int32_t* prefix_lens, const int32_t* node_offsets, void* out,
                      int32_t* status, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream);

/* ------------------------------------------------------------------------
 * FP8 tree attention ([EC] §9.2: FP8 mixed-precision tree verification,
 * E4M3 values with fp32 accumulation and one scale per 128-element block).
 *
 * The same attention as tv_tree_attention (same mask, key list, layouts of
 * the index arrays, output, status and workspace), on E4M3 inputs: q_nodes,
 * the pools and the tree K/V hold one-byte E4M3 codes (OCP layout: bias 7,
 * subnormals, NaN at S.1111.111, no infinities), and every row of D codes
 * (a token of one head: the 128-element block at D = 128) carries one fp32
 * scale; the value is code x scale.  head_dim must be 128
 * (TV_ERR_UNSUPPORTED otherwise).
 *   q_nodes          u8 [total_nodes][Hq][128],        q_scale fp32 [total_nodes][Hq]
 *   k_prefix_blocks  u8 [num_blocks][Hkv][16][128],    k_prefix_scale fp32 [num_blocks][Hkv][16]
 *   v_prefix_blocks  u8 [num_blocks][Hkv][16][128],    v_prefix_scale fp32 [num_blocks][Hkv][16]
 *   k_nodes, v_nodes u8 [total_nodes][Hkv][128],       k_nodes_scale, v_nodes_scale fp32 [total_nodes][Hkv]
 * Arithmetic: S = Q K^T on the tensor cores over the codes (E4M3 x E4M3,
 * fp32 accumulation), each score times its query row's and key row's scale;
 * fp32 online softmax; each V row converted to fp16 as code x scale (the
 * exact product rounded once), P rounded to fp16 (the row sum adds the
 * rounded values), P V in fp16 with fp32 accumulation.  The dequantised V
 * values must lie in the fp16 range (|code x scale| <= 65504, i.e. a V scale
 * of at most 146 for codes up to 448); larger ones become infinite.  All
 * device pointers 16-byte aligned (the scale arrays 4-byte). */
int tv_tree_attention_fp8(const tv_attn_params* params, const uint8_t* q_nodes,
                          const float* q_scale, const uint8_t* k_prefix_blocks,
                          const float* k_prefix_scale, const uint8_t* v_prefix_blocks,
                          const float* v_prefix_scale, const int32_t* block_table,
                          const uint8_t* k_nodes, const float* k_nodes_scale,
                          const uint8_t* v_nodes, const float* v_nodes_scale,
                          const int32_t* parent, const int32_t* prefix_lens,
                          const int32_t* node_offsets, void* out, int32_t* status,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Tree attention for callers that cannot allocate (no counterpart on the
 * pages: an engineering addition of this library).
 *
 * Same inputs, outputs, layouts, semantics and status codes as
 * tv_tree_attention, but no workspace argument: the device scratch the plan
 * needs (tv_tree_attention_workspace_size: arrival counters and
 * partial-result slots) comes from a fixed device array inside the library,
 * so a caller that may not call cudaMalloc (code running under stream
 * capture, an operator inside an engine that owns all device memory, a
 * service that forbids allocation after start-up) can still use it.  This
 * entry point allocates nothing and calls no allocating routine.
 *   - The array is TV_NO_ALLOC_SCRATCH_BYTES (64 MiB) of device memory; every
 *     GPU on which this entry point runs holds it until the process exits.
 *   - A call whose scratch would not fit
 *     (tv_tree_attention_workspace_size(params) > TV_NO_ALLOC_SCRATCH_BYTES)
 *     returns TV_ERR_WORKSPACE before anything is enqueued.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current and keeps it for the
 *     life of the process; make that first call before any stream capture on
 *     the device, and do not reset the device's primary context afterwards.
 *   - Every call uses the same array and it keeps the last call's contents;
 *     the arrival counters that must start at zero are cleared by each call
 *     on its stream.  Calls that overlap on the GPU (other streams, other host
 *     threads) race on the array: serialise them. */
#define TV_NO_ALLOC_SCRATCH_BYTES (64u << 20)
int tv_tree_attention_no_alloc(const tv_attn_params* params, const uint16_t* q_nodes,
                               const uint16_t* k_prefix_blocks, const uint16_t* v_prefix_blocks,
                               const int32_t* block_table, const uint16_t* k_nodes,
                               const uint16_t* v_nodes, const int32_t* parent,
                               const int32_t* prefix_lens, const int32_t* node_offsets,
                               void* out, int32_t* status, cudaStream_t stream);

/* ========================================================================
 * Fused accept pass ([EC] §2.2.3; [LLM] §2.2.1-§2.2.2, §7.1)
 *
 * Per tree b, for every draft node i >= 1 with parent j:
 *   p = target probability of token x_i in row j (probs given, or softmax of
 *       the logits row, fp32), q = draft probability of x_i in row j.
 *   Pruning renormalisation when retained_mask is given: on the retained set
 *   R_j, p~ = p / Z_j and q~ = q / Z_j (log space: add log(1/Z_j)); off R_j
 *   p~ = q~ = 0 (log space: -inf).  Z_j = the retained draft mass, summed
 *   exactly in 2^-40 fixed point and rounded once to fp32.  Without a mask
 *   p~ = p, q~ = q.
 *   Test: a_i = fl32(u_i * q~) < p~  (u < min(1, p~/q~), strict, NaN rejects).
 * Walk: the deepest node whose whole root path is accepted (cut at the first
 *   rejection), ties to the smallest index; accepted_len = its depth.
 * Bonus token: from the cut node j*: if j* has children, the residual
 *   max(0, p~ - q~) of row j*; if it is a leaf or the residual is all zero,
 *   p~ of row j*; if that is all zero too, the smallest index of max p~.
 *   The draw is an exact inverse CDF in 2^-40 fixed point: quanta
 *   f_v = floor(min(r_v, 32) * 2^40), S = sum f_v (uint64),
 *   t = floor(u_0 * S), token = min v with f_0 + .. + f_v > t.
 * ====================================================================== */
typedef enum { TV_INPUT_PROBS = 0, TV_INPUT_LOGITS = 1 } tv_input_kind;

typedef struct {
  int32_t batch;        /* B >= 1                                           */
  int32_t vocab;        /* V, 1 <= V < 2^18                                 */
  int32_t max_nodes;    /* row stride of `path`; >= every N_b, <= TV_MAX_NODES */
  int32_t total_nodes;  /* node_offsets[batch] (host copy)                  */
  int32_t kind;         /* tv_input_kind: the form of `target`              */
} tv_accept_params;     /* host struct */

/* Bytes of device workspace tv_accept needs when the target rows are logits
 * or a retained_mask is given (per-row partial statistics); with
 * probabilities and no mask the workspace may be NULL. */
size_t tv_accept_workspace_size(const tv_accept_params* params);

/* Layouts:
 *   target        fp32 [total_nodes][V]  row j = target next-token
 *                 probabilities (or logits) after node j
 *   draft_probs   fp32 [total_nodes][V]  row j = draft probabilities after node j
 *   draft_tokens  int32 [total_nodes]    token of node i (node 0 unused)
 *   parent, node_offsets                 as for tree attention
 *   uniforms      fp32 [total_nodes]     u_i in [0,1) tests node i >= 1;
 *                                        u at each root is the bonus draw u_0
 *   retained_mask uint32 [total_nodes][ceil(V/32)] or NULL: bit v%32 of word
 *                 v/32 of row j set iff v is in R_j
 *   accepted_len  int32 [batch]          accepted draft tokens (-1 on error)
 *   path          int32 [batch][max_nodes]: local ids of the accepted path at
 *                 depths 1..accepted_len, then -1
 *   bonus_token   int32 [batch]          (-1 on error)
 *   status        int32 [batch]
 *   debug_pq      fp32 [total_nodes][2] or NULL: (p~, q~) used by the test of
 *                 each node (0, 0 at roots)
 *   workspace     device bytes >= tv_accept_workspace_size() for logits input
 *                 or with a mask (else may be NULL)
 * All device pointers 16-byte aligned; V * 4 a multiple of 16 is not required. */
int tv_accept(const tv_accept_params* params, const float* target, const float* draft_probs,
              const int32_t* draft_tokens, const int32_t* parent, const int32_t* node_offsets,
              const float* uniforms, const uint32_t* retained_mask, int32_t* accepted_len,
              int32_t* path, int32_t* bonus_token, int32_t* status, float* debug_pq,
              void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Accept-test variants (tv_accept_ex; tv_accept is tv_accept_ex with NULL
 * options, i.e. TV_TEST_RATIO and no calibration factor):
 *   TV_TEST_RATIO      a_i = fl32(u_i * q~) < fl32(gamma_b * p~): the test
 *                      u < min(1, gamma * p/q) with the calibration factor of
 *                      [MM] §3.3 (gamma = exp(-lambda KL) computed by the
 *                      caller, one per sequence; gamma = 1 is the plain test).
 *   TV_TEST_LOG_CLAMP  the log-space test of [LLM] §10.2:
 *                      r = clamp(log p~ - log q~ + log gamma_b, -L, L) in fp32,
 *                      a_i = u_i < (r >= 0 ? 1 : exp(r)); p~ = 0 or a NaN r
 *                      rejects (a pruned token never passes).
 * For these two the walk and the bonus draw are unchanged (the residual
 * max(0, p~ - q~)).
 *   TV_TEST_MULTI      multi-candidate verification with residual updates
 *                      (multi-step speculative sampling of SpecInfer, which
 *                      the pages cite; the pages only say "resample at the
 *                      rejection"): from the root, the children c of the
 *                      current node j are tried in increasing index order
 *                      against the current target distribution cur (at first
 *                      p~_j): accept iff fl32(u_c * q~_j(x_c)) <
 *                      fl32(gamma_b * cur(x_c)), and the first accepted child
 *                      becomes the current node.  A rejection replaces cur by
 *                      fl32(r / N) with r = max(0, fl32(cur - q~_j)) and N the
 *                      fp32 of the exact 2^-40 fixed-point sum of r (cur is
 *                      kept when that sum is 0).  When every child of the
 *                      final node is rejected, the bonus is drawn from the
 *                      last r (from cur when its sum is 0); at a leaf from p~.
 *                      On a chain it decides exactly as TV_TEST_RATIO.
 *                      debug_pq holds (cur(x_c), q~(x_c)) of the tested
 *                      children and zeros for untested nodes.
 * gamma: device fp32 [batch] or NULL (1); a gamma_b that is not a positive
 * finite number gives that sequence TV_ERR_BAD_TREE.  log_clamp: L, 0 => 20. */
typedef enum { TV_TEST_RATIO = 0, TV_TEST_LOG_CLAMP = 1, TV_TEST_MULTI = 2 } tv_accept_test;

typedef struct {
  int32_t test;        /* tv_accept_test                                 */
  float log_clamp;     /* L for TV_TEST_LOG_CLAMP, 0 => 20; at most 88    */
  const float* gamma;  /* device fp32 [batch] calibration factors, or NULL */
} tv_accept_options;   /* host struct */

int tv_accept_ex(const tv_accept_params* params, const tv_accept_options* options,
                 const float* target, const float* draft_probs, const int32_t* draft_tokens,
                 const int32_t* parent, const int32_t* node_offsets, const float* uniforms,
                 const uint32_t* retained_mask, int32_t* accepted_len, int32_t* path,
                 int32_t* bonus_token, int32_t* status, float* debug_pq, void* workspace,
                 size_t workspace_bytes, cudaStream_t stream);

/* ========================================================================
 * Retained set of the draft rows (the step before the accept pass's pruning
 * renormalisation; [LLM] §2.1.2 soft truncation by cumulative probability
 * mass, [LLM] §7.1 the same decision in log space).
 *
 * For every row r of draft_probs, with key_v = q_v if q_v > 0 else 0 (NaN
 * and negatives count as 0) and the fixed-point quantum
 * f_v = floor(min(key_v, 32) * 2^40) used by tv_accept:
 *   order the tokens by key desc, id asc; R_r = the shortest prefix of that
 *   order whose sum of f_v reaches T = floor(mass * 2^40), or every token if
 *   no prefix does (the crossing token is kept; ties go to the lower id).
 * Outputs: retained_mask bit v%32 of word v/32 of row r set iff v in R_r
 * (the layout tv_accept takes), and optionally z_fixed[r] = sum of f_v over
 * R_r (exact, uint64), z[r] = z_fixed[r] * 2^-40 rounded once to fp32 (the
 * Z that tv_accept divides by), kept[r] = |R_r|.  Every sum is an exact
 * integer: the result does not depend on the reduction order.
 * ====================================================================== */
typedef struct {
  int32_t rows;   /* R >= 1                                                */
  int32_t vocab;  /* V, 1 <= V <= 2^18                                     */
  float mass;     /* retained mass, 1 - Prune_Ratio: 2^-40 <= mass <= 32   */
} tv_retain_params; /* host struct */

/* Layouts: draft_probs fp32 [rows][V]; retained_mask uint32 [rows][ceil(V/32)];
 * z_fixed uint64 [rows], z fp32 [rows], kept int32 [rows] (each optional,
 * NULL to skip).  Device pointers 16-byte aligned. */
int tv_retained_set(const tv_retain_params* params, const float* draft_probs,
                    uint32_t* retained_mask, uint64_t* z_fixed, float* z, int32_t* kept,
                    cudaStream_t stream);

/* ========================================================================
 * Commit of the accepted path ([MM] §9.1 item 2: the target KV cache is
 * preallocated and tree-node KV is written into it by a scatter kernel;
 * [LLM] §2.3.2: pool slots only for the unique accepted path; [EC] §5.2:
 * the prefix cache grows incrementally by the accepted path).
 *
 * For every sequence b with accepted_len a = accepted_len[b] >= 0 and
 * prefix length L = prefix_lens[b]: the root (local node 0, the token
 * committed by the previous step, whose K/V this step computed) and the
 * accepted nodes path[b][0..a-1] become committed tokens at positions
 * L, L+1, .., L+a.  For every KV head, the K and V rows of node v
 * (k_nodes/v_nodes row n0 + v) are copied to row pos % 16 of pool page
 * block_table[b][pos / 16] (layouts as for tree attention), and
 * new_prefix_lens[b] = L + a + 1; status[b] = TV_OK.
 * A sequence is left untouched (new_prefix_lens[b] = L, nothing written) with
 *   TV_ERR_BAD_TREE if a < 0 (its accept pass failed), a >= N_b, its tree
 *     extent is malformed, or path[b][d] is not a child of path[b][d-1]
 *     (path[b][-1] = the root);
 *   TV_ERR_NO_PAGE if a position L..L+a has no page (block id < 0 or >=
 *     num_blocks, or past max_blocks_per_seq): the caller's allocator
 *     provides the pages before the call.
 * Every output is written by the call: status and new_prefix_lens need no
 * initialisation.  new_prefix_lens must not alias prefix_lens.  Positions
 * L..L+a of every listed page must not be read by other work in flight.
 * ====================================================================== */
typedef struct {
  int32_t batch;              /* B >= 1                                      */
  int32_t num_kv_heads;       /* Hkv                                         */
  int32_t head_dim;           /* D: 64 or 128                                */
  int32_t block_size;         /* must be TV_BLOCK_SIZE (16)                  */
  int32_t max_blocks_per_seq; /* row stride of block_table                   */
  int32_t num_blocks;         /* pages in the pool                           */
  int32_t max_nodes;          /* row stride of path; >= every N_b            */
  int32_t total_nodes;        /* node_offsets[batch] (host copy)             */
} tv_commit_params;           /* host struct */

/* Layouts: k_nodes, v_nodes bf16 [total_nodes][Hkv][D]; parent, node_offsets,
 * accepted_len, path as produced for / by tv_accept; block_table int32
 * [batch][max_blocks_per_seq]; prefix_lens, new_prefix_lens, status int32
 * [batch]; k_prefix_blocks, v_prefix_blocks bf16 [num_blocks][Hkv][16][D]
 * (written).  All device pointers 16-byte aligned. */
int tv_commit_kv(const tv_commit_params* params, const uint16_t* k_nodes,
                 const uint16_t* v_nodes, const int32_t* parent, const int32_t* node_offsets,
                 const int32_t* accepted_len, const int32_t* path, const int32_t* block_table,
                 const int32_t* prefix_lens, uint16_t* k_prefix_blocks, uint16_t* v_prefix_blocks,
                 int32_t* new_prefix_lens, int32_t* status, cudaStream_t stream);

/* ========================================================================
 * Attention of a chunk of new tokens over the paged cache: the prompt (or a
 * part of it) that fills the cache which tree attention then reads, or one
 * plain decode token per sequence, in one ragged batch.
 *
 * Sequence b has seq_lens[b] cached tokens, of which the last C_b =
 * token_offsets[b+1] - token_offsets[b] (0 <= C_b <= seq_lens[b]) are the
 * chunk: their K/V are in the pool already (tv_append_kv).  Token i of the
 * chunk is row token_offsets[b] + i of q and sits at position
 * p = seq_lens[b] - C_b + i.  For every query head h, with KV head
 * floor(h / (Hq/Hkv)):
 *   out[row][h] = sum_k softmax_k(scale * q.k_k) * v_k   over the keys
 *   k <= p with  window == 0  or  k > p - window  or  k < sinks:
 * causal, optionally with a sliding window of `window` tokens (the token
 * itself included) next to which the first `sinks` tokens stay visible.  Every
 * row sees at least itself.  (The tree attentions have no window: they see the
 * whole prefix, so the trees of a windowed layer can be verified with them only
 * while the prefix and a path together are no longer than the window.)
 *   - Pages that no row of the chunk sees are not read: their block-table
 *     entries may hold anything (a windowed cache frees them).  Cached values
 *     at positions that no row sees do not matter; a non-finite V at a position
 *     that some row sees may also reach rows that do not see it (their weight
 *     of 0 times it is NaN).
 *   - An empty chunk (C_b = 0) writes nothing.  Rows of out past
 *     token_offsets[batch] are left as they were.
 *   - A sequence with a malformed extent (C_b < 0, C_b > seq_lens[b], rows past
 *     total_tokens, seq_lens[b] > max_len) or a bad block id of a page that it
 *     sees gets status TV_ERR_BAD_TREE and all-zero rows (those of [0,
 *     total_tokens)).  So do all sequences after one with C_b < 0 (their rows
 *     would be counted twice): of their rows, those that an earlier sequence has
 *     are that sequence's.
 * Inputs bf16, accumulation and softmax fp32, output bf16 or fp32; P is rounded
 * to bf16 for the P V product, so the fp32 output carries that rounding.
 * Repeated calls agree bit for bit.
 * ====================================================================== */
typedef struct {
  int32_t batch;              /* B >= 1                                        */
  int32_t num_q_heads;        /* Hq                                            */
  int32_t num_kv_heads;       /* Hkv; Hq % Hkv == 0, Hq / Hkv <= 256           */
  int32_t head_dim;           /* D: 64 or 128                                  */
  int32_t block_size;         /* tokens per page: must be TV_BLOCK_SIZE (16)   */
  int32_t max_blocks_per_seq; /* row stride of block_table                     */
  int32_t num_blocks;         /* pages in the pool                             */
  int32_t total_tokens;       /* rows of q and out, >= token_offsets[batch]
                                 (host copy); 0: only status is written        */
  int32_t max_len;            /* upper bound of seq_lens[b]                    */
  int32_t window;             /* 0: every earlier token, else >= 1             */
  int32_t sinks;              /* first tokens that stay visible next to a window */
  int32_t out_dtype;          /* tv_out_dtype of `out`                         */
  float softmax_scale;        /* finite, >= 0; 0 => 1/sqrt(D)                  */
  int64_t q_stride;           /* elements between the rows of q (a slice of a
                                 fused projection), 0 => Hq*D; rows 16-byte aligned */
} tv_chunk_params;            /* host struct */

/* Bytes of device workspace for these parameters on the current device (0 if
 * they are invalid): a ticket counter per CTA (zeroed by every call, on the
 * stream) and two partial-result slots per CTA, at most 40.5 MB at D = 128 on
 * 152 SMs.  Contents need no initialisation; calls that overlap on the GPU
 * (two captured graphs replayed at once among them) need distinct workspaces. */
size_t tv_chunk_attention_workspace_size(const tv_chunk_params* params);

/* Layouts: q bf16 [total_tokens][Hq][D] (rows q_stride apart); k_pool, v_pool
 * bf16 [num_blocks][Hkv][16][D]; block_table int32 [batch][max_blocks_per_seq];
 * seq_lens int32 [batch]; token_offsets int32 [batch+1]; out [total_tokens]
 * [Hq][D]; status int32 [batch].  All device pointers 16-byte aligned.
 * TV_ERR_UNSUPPORTED: a head_dim other than 64 and 128, or Hq / Hkv > 256.
 * TV_ERR_INVALID_ARG also where the work is too long to be counted in 32 bits: a
 * whole prompt of 2^19 tokens with 64/8 heads is taken, one of 2^20 in parts. */
int tv_chunk_attention(const tv_chunk_params* params, const uint16_t* q, const uint16_t* k_pool,
                       const uint16_t* v_pool, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* token_offsets, void* out,
                       int32_t* status, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream);

/* The same over an E4M3 cache (tv_append_kv_fp8), in the formats of
 * tv_tree_attention_fp8 and with its values: S on the tensor cores over the
 * codes, V as the fp32 product code x scale rounded to fp16, P in fp16:
 * q u8 codes [total_tokens][Hq][128] with
 * q_scale fp32 [total_tokens][Hq] (tv_quantize_rows), pools u8 [num_blocks]
 * [Hkv][16][128] with scales fp32 [num_blocks][Hkv][16].  Scales are positive;
 * code x scale of V lies in the fp16 range.  head_dim must be 128
 * (TV_ERR_UNSUPPORTED otherwise). */
int tv_chunk_attention_fp8(const tv_chunk_params* params, const uint8_t* q, const float* q_scale,
                           const uint8_t* k_pool, const float* k_scale, const uint8_t* v_pool,
                           const float* v_scale, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* token_offsets, void* out,
                           int32_t* status, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* ========================================================================
 * Writing new K/V rows into the paged cache, and reading an E4M3 cache back.
 *
 * Token i of sequence b's chunk (rows token_offsets[b] + i, 0 <= i < C_b =
 * token_offsets[b+1] - token_offsets[b]) belongs at position
 * pos = seq_lens[b] - C_b + i: seq_lens counts the chunk in, as for the chunk
 * attention that follows.  Its rows of every KV head go to row pos % 16 of page
 * block_table[b][pos / 16].
 *   tv_append_kv       copies bf16 rows.
 *   tv_append_kv_fp8   quantises each row of D values: scale s = fl32(max|x| /
 *                      448) over its finite entries, at least 2^-126, 1 for a
 *                      row of zeros; code = the E4M3 value nearest to the real
 *                      quotient x / s, ties to even, magnitudes above 448 (an
 *                      infinity) saturating, NaN as 0x7F.  With D = 128, the
 *                      cache that tv_tree_attention_fp8 and
 *                      tv_chunk_attention_fp8 read; they take V in fp16, so rows
 *                      of V beyond 65504 (stored here as they are) become
 *                      infinite there.  With D = 64 tv_read_kv_fp8 alone reads it.
 *   tv_read_kv_fp8     the other way: bf16 rows code x scale (the fp32 product,
 *                      rounded to nearest even).
 * status[b]: TV_OK, also for an empty chunk; TV_ERR_BAD_TREE if seq_lens[b] <
 * C_b, and for every sequence if token_offsets is not non-decreasing within
 * [0, total_tokens]; TV_ERR_NO_PAGE if a position of the chunk has no page
 * (block id < 0 or >= num_blocks, or past max_blocks_per_seq).  Of a failed
 * sequence nothing is written (an append) or its rows read as zeros (a read;
 * with malformed token_offsets nothing is written).  Rows past
 * token_offsets[batch] and pool rows of other positions are left as they were.
 * Two tokens must not share a pool row: the block tables of sequences that
 * append do not overlap at the appended positions.
 * ====================================================================== */
typedef struct {
  int32_t batch;              /* B >= 1                                      */
  int32_t num_kv_heads;       /* Hkv                                         */
  int32_t head_dim;           /* D: 64 or 128                                */
  int32_t block_size;         /* must be TV_BLOCK_SIZE (16)                  */
  int32_t max_blocks_per_seq; /* row stride of block_table                   */
  int32_t num_blocks;         /* pages in the pool                           */
  int32_t total_tokens;       /* rows, >= token_offsets[batch] (host copy);
                                 0: only status is written                   */
  int64_t kv_stride;          /* elements between the rows of k_new and v_new
                                 (k_out, v_out), 0 => Hkv*D; a multiple of 8 */
} tv_cache_params;            /* host struct */

/* Layouts: k_new, v_new, k_out, v_out bf16 [total_tokens][Hkv][D] (rows
 * kv_stride apart: slices of a fused projection); pools bf16 or u8
 * [num_blocks][Hkv][16][D]; scales fp32 [num_blocks][Hkv][16]; block_table
 * int32 [batch][max_blocks_per_seq]; seq_lens int32 [batch]; token_offsets
 * int32 [batch+1]; status int32 [batch].  Device pointers 16-byte aligned. */
int tv_append_kv(const tv_cache_params* params, const uint16_t* k_new, const uint16_t* v_new,
                 const int32_t* block_table, const int32_t* seq_lens,
                 const int32_t* token_offsets, uint16_t* k_pool, uint16_t* v_pool,
                 int32_t* status, cudaStream_t stream);
int tv_append_kv_fp8(const tv_cache_params* params, const uint16_t* k_new, const uint16_t* v_new,
                     const int32_t* block_table, const int32_t* seq_lens,
                     const int32_t* token_offsets, uint8_t* k_pool, float* k_scale,
                     uint8_t* v_pool, float* v_scale, int32_t* status, cudaStream_t stream);
int tv_read_kv_fp8(const tv_cache_params* params, const uint8_t* k_pool, const float* k_scale,
                   const uint8_t* v_pool, const float* v_scale, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* token_offsets, uint16_t* k_out,
                   uint16_t* v_out, int32_t* status, cudaStream_t stream);

/* Plain rows to E4M3 codes and scales, by the same rule: queries and tree K/V
 * for the E4M3 attentions.  x bf16 [tokens][heads][head_dim], tokens `stride`
 * elements apart (0 => heads*head_dim; a multiple of 8); codes u8
 * [tokens][heads][head_dim]; scale fp32 [tokens][heads].  head_dim 64 or 128
 * (TV_ERR_UNSUPPORTED otherwise); tokens 0 enqueues nothing. */
typedef struct {
  int32_t tokens, heads, head_dim;
  int64_t stride;
} tv_quant_params; /* host struct */
int tv_quantize_rows(const tv_quant_params* params, const uint16_t* x, uint8_t* codes,
                     float* scale, cudaStream_t stream);

/* tv_commit_kv of an E4M3 cache: codes and scales of the root and the accepted
 * nodes (as tv_tree_attention_fp8 took them) are copied to the pool.  Same
 * semantics, layouts of the index arrays and status codes. */
int tv_commit_kv_fp8(const tv_commit_params* params, const uint8_t* k_nodes,
                     const float* k_nodes_scale, const uint8_t* v_nodes,
                     const float* v_nodes_scale, const int32_t* parent,
                     const int32_t* node_offsets, const int32_t* accepted_len,
                     const int32_t* path, const int32_t* block_table, const int32_t* prefix_lens,
                     uint8_t* k_prefix_blocks, float* k_prefix_scale, uint8_t* v_prefix_blocks,
                     float* v_prefix_scale, int32_t* new_prefix_lens, int32_t* status,
                     cudaStream_t stream);

/* ========================================================================
 * Penalties for repeated tokens, biases and grammar masks on the target logits
 * of the tree nodes, ahead of tv_accept with TV_INPUT_LOGITS.
 *
 * Row i of tree b holds the logits after node i.  Counted against it are the
 * sequence's history and the drafted tokens on the path root .. i (node i's own
 * included, the root's not: it is the last committed token, part of the
 * history).  With c(v) = the occurrences of v in the history past the first
 * prompt_lens[b] tokens and on the path, and seen(v) = c(v) > 0 or v among the
 * first prompt_lens[b] tokens, in this order and each step rounded to fp32:
 *   seen(v):   x = x > 0 ? x / repetition[b] : x * repetition[b]
 *              x = x - frequency[b] * c(v)
 *   c(v) > 0:  x = x - presence[b]
 *              x = x + bias of v (of an id listed twice the last entry holds)
 *   bit v % 32 of word v / 32 of the row's allowed_mask clear: x = -inf
 * A logit of -inf stays -inf; a row whose mask allows nothing is all -inf.  Ids
 * outside [0, V), in the history, the bias list or the tree, count for nothing.
 * A sequence with a malformed tree, history or bias extent, or a rate that is
 * not finite (a repetition not positive), gets TV_ERR_BAD_TREE and its rows
 * unchanged (as far as they can be addressed).  So do all sequences after one
 * whose node_offsets decrease: of their rows, those that an earlier sequence has
 * are that sequence's.
 * ====================================================================== */
typedef struct {
  int32_t batch;         /* 1 <= B <= 65535                                */
  int32_t vocab;         /* V, 1 <= V < 2^18: as tv_accept, which takes the rows next */
  int32_t max_nodes;     /* >= every N_b, <= TV_MAX_NODES                  */
  int32_t total_nodes;   /* node_offsets[batch] (host copy)                */
  int32_t total_history; /* entries of history, <= 2^30                    */
  int32_t total_bias;    /* entries of bias_ids and bias_values, <= 2^30   */
  int32_t logits_dtype;  /* tv_out_dtype of `logits`: bf16 (0) or fp32 (1) */
} tv_penalty_params;     /* host struct */

/* Layouts: logits bf16 or fp32 [total_nodes][V]; draft_tokens, parent,
 * node_offsets as for tv_accept; history int32 [total_history] with
 * history_offsets int32 [batch+1], or both NULL; prompt_lens int32 [batch] or
 * NULL (0: all history is generated); repetition, presence, frequency fp32
 * [batch] or NULL (1, 0, 0); bias_ids int32 and bias_values fp32 [total_bias]
 * with bias_offsets int32 [batch+1], or NULL (a list without entries may be NULL
 * with its offsets given: they are checked); allowed_mask uint32
 * [total_nodes][ceil(V/32)] or NULL; out fp32 [total_nodes][V], which may be
 * the fp32 logits themselves (in place) and otherwise does not overlap them;
 * status int32 [batch].  Device pointers 16-byte aligned. */
int tv_penalize_logits(const tv_penalty_params* params, const void* logits,
                       const int32_t* draft_tokens, const int32_t* parent,
                       const int32_t* node_offsets, const int32_t* history,
                       const int32_t* history_offsets, const int32_t* prompt_lens,
                       const float* repetition, const float* presence, const float* frequency,
                       const int32_t* bias_ids, const float* bias_values,
                       const int32_t* bias_offsets, const uint32_t* allowed_mask, float* out,
                       int32_t* status, cudaStream_t stream);

/* ========================================================================
 * Norm of every query and key head and its rotation by the token's position,
 * in one pass, ahead of tv_append_kv, tv_quantize_rows and the attentions
 * (which take rotated rows).
 *
 * A head x of D values of token t becomes, with weights w given (q_weight for
 * queries, k_weight for keys; NULL: no norm),
 *   x = x / sqrt(mean(x^2) + eps) * w,
 * and of its first R = rotary_dim values pair i < R/2, (x_i, x_{i+R/2}), or
 * (x_2i, x_2i+1) with `interleaved`, turns by
 *   theta = positions[axis_of_pair[i]][t] * frequencies[i]:
 *   (a, b) -> scale * (a cos theta - b sin theta, a sin theta + b cos theta).
 * The other values stay as they are (normed).  Several axes serve images and
 * video: of a text token all positions are the same, of an image's its time, row
 * and column; a list of sections, or axes taken in turn, is a choice of
 * axis_of_pair.  Tree nodes have the position prefix length + depth.  Frequencies
 * of the other sign turn back.
 * Arithmetic: fp32, one rounding to bf16.  An angle's fraction of a turn is
 * computed in 64-bit fixed point, off by at most |position| 2^-64 turns for
 * |frequency| <= 2 pi: far positions lose nothing.  A frequency that is not
 * finite makes its pairs NaN.  The norm's sum of squares overflows fp32 from
 * values near 2^60 on, and a row of zeros with eps = 0 is NaN.
 * In place: q_out may be q with the same stride, k_out k with its own; other
 * overlaps of an output with an input or with the other output are refused (of the
 * weights, positions and frequencies also between its rows).
 * ====================================================================== */
#define TV_MAX_POSITION_AXES 4
typedef struct {
  int32_t tokens;         /* T rows, <= 2^30; 0 enqueues nothing                */
  int32_t num_q_heads;    /* 1 <= Hq <= 2^20; T * (Hq + Hkv) < 2^40             */
  int32_t num_kv_heads;   /* 0 <= Hkv <= 2^20 (0: queries alone)                */
  int32_t head_dim;       /* D: 64 or 128                                       */
  int32_t rotary_dim;     /* R: even, 0 <= R <= D (0: norms alone)              */
  int32_t interleaved;    /* 0: pairs (i, i + R/2); 1: pairs (2i, 2i + 1)       */
  int32_t num_axes;       /* rows of positions, 1 .. TV_MAX_POSITION_AXES       */
  int32_t weight_dtype;   /* tv_out_dtype of the weights: bf16 (0) or fp32 (1)  */
  float eps;              /* >= 0                                               */
  float scale;            /* of the turned values (a long-context rule's factor), 0 => 1 */
  int64_t q_stride;       /* elements between the rows of q, 0 => Hq*D; multiples of 8 */
  int64_t k_stride;       /* ... of k, 0 => Hkv*D                               */
  int64_t q_out_stride;
  int64_t k_out_stride;
  uint8_t axis_of_pair[64]; /* position axis of pair i < R/2                    */
} tv_rotate_params;       /* host struct */

/* Layouts: q, q_out bf16 [T][Hq][D], k, k_out bf16 [T][Hkv][D] (rows a stride
 * apart: slices of a fused projection); q_weight, k_weight [D] or NULL;
 * positions int32 [num_axes][T]; frequencies fp64 [R/2], radians a position (NULL
 * with R = 0, as positions).  k and k_out may be NULL with num_kv_heads = 0.
 * Device pointers 16-byte aligned. */
int tv_rotate_qk(const tv_rotate_params* params, const uint16_t* q, const uint16_t* k,
                 const void* q_weight, const void* k_weight, const int32_t* positions,
                 const double* frequencies, uint16_t* q_out, uint16_t* k_out,
                 cudaStream_t stream);

/* ========================================================================
 * The next beams of every request: the S best continuations over its K beams
 * and the vocabulary.
 *
 * Request b has rows b*K .. b*K + K-1.  Row r with score s_r (the sum of its
 * tokens' log-probabilities) and logits x offers, for every token v,
 *   score d = s_r + x_v - LSE(x), length lengths[r] + 1;
 * a row with finished[r] != 0 offers itself once: token end_token, score s_r,
 * length lengths[r]; its logits are not read.  Candidates are ordered by
 *   key = d / max(length, 1)^length_penalty, then the lower row, then the lower
 * token, and the first S are written, in order: token, parent row (of all rows,
 * as tv_fork_pages takes it), score, length, and whether the continuation has
 * ended (its parent had, or its token is end_token).  S = 2K candidates hold K
 * that have not ended, whatever ends.
 * A logit of -inf or NaN and a row with score -inf offer nothing; where fewer than
 * S candidates are left the rest is token -1, parent -1, score -inf, length 0,
 * finished 0.  A score that is NaN or +inf, a logit of +inf in a row that is read,
 * or a length below 0 or above 2^24 gives the request TV_ERR_BAD_TREE and such
 * entries throughout.
 * Within a row the order is exact, that of the logits and of equal ones the lower
 * token, also where a large score or logit leaves the keys of a row one value in fp64,
 * in which rows are compared.  LSE is off by less than 2^-15 (fp32 exps and sums; by
 * less than 2^-17 where a row's largest entry is not reached in many small steps, and
 * ordinarily by 1e-7), so candidates of different rows whose scores are closer than
 * that may come in either order, the same in every call; scores are rounded once
 * to fp32.
 * ====================================================================== */
#define TV_MAX_BEAMS 64
#define TV_MAX_BEAM_SELECT 64
typedef struct {
  int32_t batch;         /* 1 <= B <= 65535                                    */
  int32_t beams;         /* K, 1 .. TV_MAX_BEAMS                               */
  int32_t select;        /* S, 1 .. TV_MAX_BEAM_SELECT                         */
  int32_t vocab;         /* V, 1 <= V < 2^18                                   */
  int32_t logits_dtype;  /* tv_out_dtype of the logits: bf16 (0) or fp32 (1)   */
  int32_t end_token;     /* -1: none, else below V                             */
  float length_penalty;  /* -4 .. 4; 0: keys are scores                        */
  int64_t logits_stride; /* entries between the rows of logits, 0 => V         */
} tv_beam_params;        /* host struct */

/* Bytes of device workspace for these parameters on the current device (0 if they
 * are invalid): of each part of a row (at most 32) its maximum, sum and S best, of
 * each row a factor.
 * Contents need no initialisation; calls that overlap on the GPU need distinct
 * workspaces. */
size_t tv_beam_select_workspace_size(const tv_beam_params* params);

/* Layouts: logits bf16 or fp32 [B*K][V] (rows logits_stride apart); scores fp32
 * [B*K]; lengths, finished int32 [B*K] or NULL (lengths may be NULL only with
 * length_penalty 0 and lengths_out NULL); tokens, parents int32 [B][S]; scores_out
 * fp32 [B][S]; lengths_out, finished_out int32 [B][S] or NULL; status int32 [B].
 * Outputs or a workspace that overlap an input or each other are refused.  Device
 * pointers 16-byte aligned. */
int tv_beam_select(const tv_beam_params* params, const void* logits, const float* scores,
                   const int32_t* lengths, const int32_t* finished, int32_t* tokens,
                   int32_t* parents, float* scores_out, int32_t* lengths_out,
                   int32_t* finished_out, int32_t* status, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/* ========================================================================
 * The pages of the paged cache: given to sequences, taken back, passed on to the
 * children of a beam step (or of a shared prompt), compacted, copied.
 *
 * An entry >= 0 of a block-table row is a reference to a page; a negative one is
 * none.  ref_counts[p] counts the references to page p, and the caller's own
 * besides; a page is free where it is 0.  The caller keeps ref_counts[p] at least
 * the number of entries that name p (a table of -1 and counts of 0 to begin with);
 * the calls keep it so.  Where it is not, no call reads or writes out of range, and
 * that is all.  An entry >= num_blocks names nothing.
 * Pages are given lowest number first, to rows in order: the same tables and
 * counts give the same result.  Calls on the same counts must not overlap on the
 * GPU.  Arrays of a call that overlap are refused (TV_ERR_INVALID_ARG) but for the
 * two that tv_compact_pages names.
 * ====================================================================== */
typedef struct {
  int32_t rows;               /* 1 <= R <= 65536 rows of block_table           */
  int32_t new_rows;           /* tv_fork_pages: 1 <= R' <= 65536; else unused  */
  int32_t block_size;         /* must be TV_BLOCK_SIZE (16)                    */
  int32_t max_blocks_per_seq; /* row stride of the block tables, <= 2^27, and
                                 R times it < 2^31                             */
  int32_t num_blocks;         /* pages in the pool, <= 2^30                    */
  int32_t sinks;              /* tv_free_pages: first tokens that are kept     */
} tv_page_params;             /* host struct */

/* Bytes of device workspace of tv_alloc_pages and tv_fork_pages (0 if the
 * parameters are invalid).  Contents need no initialisation; calls that overlap on
 * the GPU need distinct workspaces. */
size_t tv_pages_workspace_size(const tv_page_params* params);

/* Pages for the positions [begin[b], end[b]) of every row: entries that lack one
 * (below 0) get a free page, whose count becomes 1.  status[b]: TV_OK, also where
 * nothing was lacking; TV_ERR_NO_PAGE, and the row unchanged, if its pages do not
 * fit behind those that all rows before it lack (theirs count whether they fit or
 * not); TV_ERR_BAD_TREE, and the row unchanged, if begin < 0, end < 0 or end > 16 *
 * max_blocks_per_seq, or one of these entries is >= num_blocks.
 * block_table int32 [R][max_blocks_per_seq] and ref_counts int32 [num_blocks] are
 * changed in place; begin int32 [R] or NULL (0); end int32 [R]; status int32 [R].
 * Device pointers 16-byte aligned. */
int tv_alloc_pages(const tv_page_params* params, int32_t* block_table, int32_t* ref_counts,
                   const int32_t* begin, const int32_t* end, int32_t* status, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/* Takes back the pages of every row outside its positions [keep_begin[b],
 * keep_end[b]): the entries of whole pages below keep_begin (but for those of the
 * first `sinks` tokens: what a sliding window no longer sees) and of pages from
 * keep_end on (a sequence that has ended: keep_end 0) become -1, and their pages'
 * counts are lowered.  keep_begin int32 [R] or NULL (0), keep_end int32 [R] or NULL
 * (everything from keep_begin on is kept); status[b]: TV_OK; TV_ERR_BAD_TREE if a
 * position is negative (the row unchanged) or such an entry was >= num_blocks (it
 * becomes -1 as well).  In place, layouts as tv_alloc_pages. */
int tv_free_pages(const tv_page_params* params, int32_t* block_table, int32_t* ref_counts,
                  const int32_t* keep_begin, const int32_t* keep_end, int32_t* status,
                  cudaStream_t stream);

/* New rows from old ones: row i of block_table_out continues row parents[i] of
 * block_table (-1: an empty row, length 0), seq_lens_out[i] = its length.  The old
 * rows are used up: their references pass to the new ones, or are given back.
 *   - Pages that the length fills are shared by all children of a row.
 *   - The page that it fills in part, which the children go on to write, stays with
 *     the first child (the lowest i) where nobody else refers to it; every other
 *     child gets a free page for it and an entry of `copies` (source page,
 *     destination page, tokens to copy) for tv_copy_pages; (-1, -1, 0) where there
 *     is nothing to copy.  Free pages are those that were free before the call.
 *     tv_copy_pages has to be enqueued before any call that gives out, moves or writes
 *     pages or reads the new rows: a source may be free from here on (of rows that
 *     share a half-filled page every child gets a copy, and nobody keeps the page).
 *   - Entries past the length (pages given ahead) pass to the first child.
 * status[i]: TV_OK; TV_ERR_BAD_TREE if parents[i] is not a row, or its row's length
 * is negative or longer than the row, or the partly filled page is missing or has
 * no count; TV_ERR_NO_PAGE if no page was left for the copy: row i is empty then,
 * length 0, and refers to nothing.  An entry >= num_blocks becomes -1 in the rows
 * that continue it, which get TV_ERR_BAD_TREE and are otherwise whole.
 * block_table int32 [R][max_blocks_per_seq], seq_lens int32 [R], parents int32
 * [R']; ref_counts int32 [num_blocks], in place; block_table_out int32 [R']
 * [max_blocks_per_seq], seq_lens_out int32 [R'], which are no inputs of the call;
 * copies int32 [R'][3]; status int32 [R'].  Device pointers 16-byte aligned. */
int tv_fork_pages(const tv_page_params* params, const int32_t* block_table,
                  const int32_t* seq_lens, const int32_t* parents, int32_t* ref_counts,
                  int32_t* block_table_out, int32_t* seq_lens_out, int32_t* copies,
                  int32_t* status, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/* Moves the pages in use together: of N pages with a count other than 0, those
 * numbered N and above move to the free numbers below N, in order.  moves[k] =
 * (source, destination, 16) for tv_copy_pages, k < count[1]; count[0] = N;
 * page_map[p] = the new number of page p, -1 of a free one (for references that
 * the caller holds); ref_counts_out and block_table_out are the counts and tables
 * in new numbers.  tv_copy_pages has to be enqueued before any call that gives out,
 * moves, writes or reads pages by them: the sources are free there.  status[b]: TV_OK;
 * TV_ERR_BAD_TREE if an entry of the row names a free page or is >= num_blocks (it
 * becomes -1).
 * ref_counts_out may be ref_counts, and block_table_out block_table.  moves int32
 * [max(1, num_blocks / 2)][3] (entries from count[1] on are left as they were), count
 * int32 [2], page_map int32 [num_blocks].  Device pointers 16-byte aligned. */
int tv_compact_pages(const tv_page_params* params, const int32_t* block_table,
                     const int32_t* ref_counts, int32_t* block_table_out,
                     int32_t* ref_counts_out, int32_t* page_map, int32_t* moves,
                     int32_t* count, int32_t* status, cudaStream_t stream);

/* Copies pages within the pools of K and V, for every layer: entry i of `copies`
 * is (source, destination, tokens): the first `tokens` rows (of 16) of every head.
 * Entries from count[0] on (count NULL: none) are left out.  No destination is
 * another entry's source or destination.  status[i]: TV_OK, also of an entry whose
 * pages are both negative (nothing to copy) or the same; TV_ERR_NO_PAGE, and
 * nothing copied, if one is not in the pool or tokens is not in 0 .. 16. */
typedef struct {
  int32_t entries;      /* of copies; 0 enqueues nothing                      */
  int32_t layers;       /* L >= 1 pools, one behind another                   */
  int32_t num_kv_heads; /* Hkv                                                */
  int32_t head_dim;     /* D: 64 or 128                                       */
  int32_t block_size;   /* must be TV_BLOCK_SIZE (16)                         */
  int32_t num_blocks;   /* pages in a layer's pool                            */
} tv_copy_params;       /* host struct */

/* Layouts: copies int32 [entries][3]; count int32 [1] (4-byte aligned) or NULL;
 * pools bf16 [L][num_blocks][Hkv][16][D]; status int32 [entries] or NULL.  _fp8:
 * pools u8, scales fp32 [L][num_blocks][Hkv][16].  Device pointers 16-byte aligned. */
int tv_copy_pages(const tv_copy_params* params, const int32_t* copies, const int32_t* count,
                  uint16_t* k_pool, uint16_t* v_pool, int32_t* status, cudaStream_t stream);
int tv_copy_pages_fp8(const tv_copy_params* params, const int32_t* copies, const int32_t* count,
                      uint8_t* k_pool, float* k_scale, uint8_t* v_pool, float* v_scale,
                      int32_t* status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TV_H_ */
