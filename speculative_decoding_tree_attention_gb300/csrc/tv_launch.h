// tv_launch.h -- argument blocks and launchers shared by the host API and the
// kernels (internal to libtv; not part of the public ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tv {

struct AcceptArgs {
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parent;
  const int32_t* node_offsets;
  const float* uniforms;
  const uint32_t* mask;
  int32_t* accepted_len;
  int32_t* path;
  int32_t* bonus_token;
  int32_t* status;
  float* debug_pq;
  int32_t vocab;
  int32_t max_nodes;
  int32_t kind;
  int32_t batch;
  int32_t total_nodes;
  int32_t test;          // 0: ratio test, 1: log-space clamped test
  float log_clamp;       // L of the clamped test
  const float* gamma;    // [batch] calibration factors or null (1)
};

// Launches the accept pass; `workspace` holds per-(row, part) statistics (at
// most one part per 8K-entry chunk of the vocabulary) and
// must be accept_workspace_bytes() long when the input is logits or a mask
// is given (it is not touched otherwise).
int launch_accept(const AcceptArgs& a, void* workspace, cudaStream_t stream);

struct RetainArgs {
  const float* draft;          // [rows][vocab]
  uint32_t* mask;              // [rows][ceil(vocab/32)]
  unsigned long long* z_fixed; // [rows] or null
  float* z;                    // [rows] or null
  int32_t* kept;               // [rows] or null
  unsigned long long threshold;// T = floor(mass * 2^40) >= 1
  int32_t rows, vocab;
};

// Retained set of every row (one CTA per row).
int launch_retained_set(const RetainArgs& a, cudaStream_t stream);
size_t accept_workspace_bytes(int vocab, int total_nodes);
int accept_cluster_size(int vocab, int batch, int sms);
int accept_max_nodes();

struct AttnArgs {
  const uint16_t* q;          // [total_nodes][Hq][D]
  const int32_t* block_table; // [batch][max_blocks_per_seq]
  const int32_t* parent;      // [total_nodes]
  const int32_t* prefix_lens; // [batch]
  const int32_t* node_offsets;// [batch+1]
  void* out;                  // [total_nodes][Hq][D], bf16 or fp32 (out_fp32)
  int32_t* status;            // [batch]
  int32_t* counters;          // [ctas][2] ticket and done counters of split units (zeroed per call)
  uint8_t* slots;             // [2 * ctas] partial-result slots of attn_slot_bytes(D)
  int32_t batch, hq, hkv, group, head_dim;
  int32_t max_blocks_per_seq, num_blocks, max_nodes, max_prefix_len, total_nodes;
  int32_t lanes;              // CTAs per virtual CTA: one per m-tile pair of a layer
  int32_t vctas;              // virtual CTAs launched (ctas = vctas * lanes)
  int32_t min_tiles;          // fewest key tiles a virtual CTA is given
  int32_t out_fp32;           // 1: fp32 output, 0: bf16
  float scale_log2;           // softmax scale * log2(e)
  // E4M3 inputs (tv_tree_attention_fp8): q, pools and tree K/V hold codes,
  // each row of D codes with one fp32 scale
  int32_t fp8;
  const float* q_scale;       // [total_nodes][Hq]
  const float* kp_scale;      // [num_blocks][Hkv][16]
  const float* vp_scale;
  const float* kn_scale;      // [total_nodes][Hkv]
  const float* vn_scale;
};

struct AttnMaps {
  CUtensorMap k_pool;   // 5D (64, 8 rows, halves, 2 groups, pages), box = one page, 128B swizzle
  CUtensorMap v_pool;
  CUtensorMap k_nodes;  // 4D (64, nodes, halves, Hkv heads), box = 8 nodes of one head
  CUtensorMap v_nodes;
};

int launch_tree_attention(const AttnArgs& a, const AttnMaps& maps, cudaStream_t stream);
// Bytes of one partial-result slot: 256 rows of fp32 O, (m, l) per row, a flag.
size_t attn_slot_bytes(int head_dim);

// Costs on the chunk attention's line of work: of a key tile of a full unit,
// and of a piece besides its tiles.  (Piece costs of 4, 6, 8 and 10: 1600-token
// prompts 98, 97, 100 and 102 us, window 1024 100, 103, 103 and 108, E4M3 decode
// 93, 91, 92 and 92.)
constexpr int kChunkTileCost = 3;
constexpr int kChunkPieceCost = 6;

struct ChunkArgs {
  const int32_t* block_table; // [batch][max_blocks_per_seq]
  const int32_t* seq_lens;    // [batch] cached tokens, the chunk's included
  const int32_t* token_offsets; // [batch+1]
  void* out;                  // [total_tokens][Hq][D], bf16 or fp32 (out_fp32)
  int32_t* status;            // [batch]
  int32_t* counters;          // [vctas] ticket counters of split units (zeroed per call)
  uint8_t* slots;             // [2 * vctas] partial-result slots of chunk_slot_bytes(D)
  int32_t q_tokens;           // tokens of a Q box: min(unit_tokens, total_tokens)
  int32_t batch, hq, hkv, group, head_dim;
  int32_t max_blocks_per_seq, num_blocks, max_len, total_tokens;
  int32_t unit_tokens;        // tokens of a unit: floor(256 / group)
  int32_t vctas;              // CTAs launched
  int32_t min_range;          // shortest range of the line a CTA is given
  int32_t window, sinks;      // window 0: every earlier key
  int32_t out_fp32;
  int32_t fp8;                // E4M3 codes with one fp32 scale per row
  float scale_log2;           // softmax scale * log2(e)
  const float* q_scale;       // [total_tokens][Hq]
  const float* k_scale;       // [num_blocks][Hkv][16]
  const float* v_scale;
};

struct ChunkMaps {
  CUtensorMap q;        // 3D (row, heads, tokens), box = 128 bytes of the g heads of q_tokens tokens
  CUtensorMap k_pool;   // as AttnMaps
  CUtensorMap v_pool;
};

int launch_chunk_attention(const ChunkArgs& a, const ChunkMaps& maps, int sms, cudaStream_t stream);
size_t chunk_slot_bytes(int head_dim);

struct CommitArgs {
  const void* k_nodes;        // [total_nodes][Hkv][D] bf16, or E4M3 codes (k_scale given)
  const void* v_nodes;
  const float* k_nodes_scale; // E4M3: [total_nodes][Hkv], else null
  const float* v_nodes_scale;
  const int32_t* parent;      // [total_nodes]
  const int32_t* node_offsets;// [batch+1]
  const int32_t* accepted_len;// [batch]
  const int32_t* path;        // [batch][max_nodes]
  const int32_t* block_table; // [batch][max_blocks_per_seq]
  const int32_t* prefix_lens; // [batch]
  void* k_pool;               // [num_blocks][Hkv][16][D]
  void* v_pool;
  float* k_scale;             // E4M3: [num_blocks][Hkv][16], else null
  float* v_scale;
  int32_t* new_prefix_lens;   // [batch]
  int32_t* status;            // [batch]
  int32_t batch, hkv, head_dim, max_blocks_per_seq, num_blocks, max_nodes, total_nodes;
};

int launch_commit(const CommitArgs& a, cudaStream_t stream);

// New K/V rows into the pool (bf16; E4M3 when k_scale is given), or, with
// `read`, an E4M3 pool's rows back into bf16 rows.
struct CacheArgs {
  void* k_new;                // bf16 rows [total_tokens][Hkv][D], kv_stride elements apart
  void* v_new;
  const int32_t* block_table; // [batch][max_blocks_per_seq]
  const int32_t* seq_lens;    // [batch] tokens, the chunk's included
  const int32_t* token_offsets; // [batch+1]
  void* k_pool;               // [num_blocks][Hkv][16][D]
  void* v_pool;
  float* k_scale;             // [num_blocks][Hkv][16] or null
  float* v_scale;
  int32_t* status;            // [batch]
  size_t kv_stride;
  int32_t batch, hkv, head_dim, max_blocks_per_seq, num_blocks, total_tokens;
  int32_t read;
  int32_t tile_shift;         // log2 of the tokens per CTA (set by the launcher)
};
int launch_cache(CacheArgs a, int sms, cudaStream_t stream);

struct QuantArgs {
  const uint16_t* x;          // bf16 [tokens][heads][D], rows `stride` elements apart
  uint8_t* codes;             // [tokens][heads][D]
  float* scale;               // [tokens][heads]
  size_t stride;
  int32_t tokens, heads, head_dim;
};
int launch_quantise_rows(const QuantArgs& a, int sms, cudaStream_t stream);

struct PenaltyArgs {
  const void* logits;         // [total_nodes][vocab], bf16 or fp32
  float* out;                 // [total_nodes][vocab]
  const int32_t* tokens;      // [total_nodes]
  const int32_t* parent;      // [total_nodes]
  const int32_t* node_offsets;// [batch+1]
  const int32_t* history;     // [total_history] or null
  const int32_t* history_offsets; // [batch+1]; null: no history (as bias_offsets)
  const int32_t* prompt_lens; // [batch] or null
  const float* repetition;    // [batch] or null
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;    // [total_bias] or null
  const float* bias_values;
  const int32_t* bias_offsets;// [batch+1]
  const uint32_t* allowed_mask; // [total_nodes][ceil(vocab/32)] or null
  int32_t* status;            // [batch]
  int32_t batch, vocab, max_nodes, total_nodes, total_history, total_bias, bf16;
};
int launch_penalty(const PenaltyArgs& a, int sms, cudaStream_t stream);

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 64;  // of a head of 128

// Norm of every head and rotation by the position.
struct RotateArgs {
  const uint16_t* q;          // bf16 [tokens][Hq][D], rows q_stride elements apart
  const uint16_t* k;          // [tokens][Hkv][D]
  const void* q_weight;       // [D] bf16 or fp32, or null: no norm
  const void* k_weight;
  const int32_t* positions;   // [axes][tokens]
  const double* frequencies;  // [rotary_dim / 2] radians a position
  uint16_t* q_out;
  uint16_t* k_out;
  size_t q_stride, k_stride, q_out_stride, k_out_stride;
  int32_t tokens, hq, hkv, head_dim, rotary_dim, axes;
  int32_t interleaved;        // pairs (2i, 2i + 1), else (i, i + rotary_dim / 2)
  int32_t weight_fp32;
  float eps, scale;
  int32_t items, each;        // warps that share a token, or steps of a warp (set by the launcher)
  uint8_t axis[kMaxPairs];    // position axis of each pair
};
int launch_rotate(RotateArgs a, int sms, cudaStream_t stream);

struct BeamArgs {
  const void* logits;         // [batch * beams][vocab], rows `stride` entries apart
  const float* scores;        // [batch * beams]
  const int32_t* lengths;     // [batch * beams] or null
  const int32_t* finished;    // [batch * beams] or null
  int32_t* tokens;            // [batch][select]
  int32_t* parents;
  float* scores_out;
  int32_t* lengths_out;       // or null
  int32_t* finished_out;      // or null
  int32_t* status;            // [batch]
  float2* stats;              // [batch * beams][parts] maximum and sum (workspace)
  float2* lists;              // [batch][select][beams][parts] logit and token, best first
  double* power;              // [batch * beams] length^length_penalty, where that exponent is not 0
  size_t stride;
  int32_t batch, beams, select, vocab, bf16, end_token, parts, chunk;
  int32_t each, more;         // a row's CTAs take each parts, the first more of them one more
  int32_t turns;              // of a part, most
  float length_penalty;
};
int launch_beam_select(const BeamArgs& a, cudaStream_t stream);
void plan_beam_parts(BeamArgs& a, int sms);  // parts, chunk, each, more
int beam_max_select();
int beam_max_beams();

struct PageArgs {
  int32_t* block_table;       // [rows][width]
  int32_t* ref_counts;        // [num_blocks]
  const int32_t* begin;       // alloc: [rows] first positions that need a page, or null
  const int32_t* end;         // alloc: [rows] their ends
  const int32_t* keep_begin;  // free: [rows] or null
  const int32_t* keep_end;    // free: [rows] or null
  const int32_t* seq_lens;    // fork: [rows]
  const int32_t* parents;     // fork: [new_rows]
  int32_t* table_out;         // fork: [new_rows][width], compact: [rows][width]
  int32_t* lens_out;          // fork: [new_rows]
  int32_t* copies;            // fork: [new_rows][3], compact: [num_blocks / 2][3] (source, destination, tokens)
  int32_t* refs_out;          // compact: [num_blocks]
  int32_t* page_map;          // compact: [num_blocks]
  int32_t* count;             // compact: [2] pages in use, moves
  int32_t* status;            // [rows], fork: [new_rows]
  int32_t* list;              // workspace: free pages in order
  int32_t* first;             // workspace: [rows] fork: first child of a row; alloc of kManyPages: its place in the list
  int32_t* counts;            // workspace: [kPageSegments] free pages of the pool's segments
  int32_t* needs;             // workspace: alloc of kManyPages: [rows][kMaxCuts] entries of a row's pieces that lack a page
  int32_t rows, new_rows, width, num_blocks, sinks;
  int32_t cuts, piece;        // alloc: pieces of a row and their entries (set by the launcher)
};
constexpr int kPageSegments = 4096;
constexpr int kManyPages = 1 << 17;  // of a pool whose allocation takes the whole GPU
constexpr int kMaxCuts = 8;          // pieces of a row, most
int launch_alloc_pages(PageArgs a, cudaStream_t stream);
int launch_free_pages(const PageArgs& a, cudaStream_t stream);
int launch_fork_pages(const PageArgs& a, cudaStream_t stream);
int launch_compact_pages(const PageArgs& a, cudaStream_t stream);

struct CopyArgs {
  const int32_t* copies;      // [entries][3] source, destination, tokens
  const int32_t* count;       // [1] or null: all entries
  void* pool[2];              // K, V: [layers][num_blocks][Hkv][16][D]
  float* scale[2];            // E4M3: [layers][num_blocks][Hkv][16], else null
  int32_t* status;            // [entries] or null
  size_t layer_stride, scale_stride;  // bytes between layers, values between layers of the scales
  int32_t entries, layers, num_blocks, hkv, row_bytes;
  int32_t slices;             // CTAs that share a page (set by the launcher)
};
int launch_copy_pages(CopyArgs a, int sms, cudaStream_t stream);

}  // namespace tv
