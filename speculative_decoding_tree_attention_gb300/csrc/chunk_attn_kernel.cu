// chunk_attn_kernel.cu -- attention of a chunk of new tokens over a paged
// cache on sm_103a (tv_chunk_attention, tv_chunk_attention_fp8).
//
// Mathematics.  Token i of sequence b sits at position p = len_b - C_b + i;
// its K/V are in the cache already.  Row (i, head) is
//   out = sum_k 2^(s_k - m) v_k / sum_k 2^(s_k - m),  s_k = log2(e) scale q.k_k
// over the visible keys: k <= p and (no window, or k > p - window, or
// k < sinks).  A row always sees itself, so the sum is never empty.
//
// Rows.  The packed query rows of one (sequence, KV head) are
// R = token * g + head-in-group, so the query heads of a GQA group share each
// K/V tile.  A unit is floor(256 / g) consecutive tokens of one (sequence, KV
// head): up to 256 rows, two 128-row m-tiles.  Its keys are the 128-key tiles
// that any of its rows sees: the tiles of the sinks, then the tiles from the
// start of the first row's window to the last row's position.
//
// A small kernel runs first (chunk_check_kernel): it checks every sequence and the
// pages that it sees, and malformed ones take no further part.
//
// Work.  Persistent grid, one CTA per SM.  All units lie on one line ordered
// (sequence, unit, KV head), cut into equal contiguous ranges, one per CTA,
// computed on the device from the lengths.  A single decode token of one
// sequence and a long prompt are split the same way.  A unit's length on the
// line is its cost: kWide for each key tile of two m-tiles, kNarrow for one of
// one (about 2.0 and 1.3 us), and kFixed for what a piece costs besides (Q, the
// first S, the last P V, the output: about 4 us).  With the tiles alone, the
// CTAs with the first units of four 1600-token prompts ran 129 us and those with
// the last 55.  A range boundary
// inside a unit splits it into pieces: each leaves its unnormalised O and
// (m, l) in a workspace slot, and the last piece to take a ticket merges all
// slots in piece order, so results do not depend on timing.
//
// One CTA has 384 threads (512 for an E4M3 cache):
//   warps 8, 11 load the K tiles, and the V tiles and Q, by TMA: one box per
//               16-token page through the block table; pages that no row of
//               the unit sees are never read (an out-of-range page index loads
//               zeros).
//   warps 9, 10 issue the tcgen05.mma of m-tile h = 0 and 1: S_h = Q_h K^T
//               into TMEM, O_h += P_h V with P_h from TMEM.  P_h lies over S_h;
//               the MMAs of one thread run in order, so S_h(t+1) follows
//               P_h(t) V.  The two take turns, P_0 V(t), S_0(t+1), P_1 V(t),
//               S_1(t+1): the softmax of one m-tile runs under the MMAs of the
//               other.  Two threads, because a wait that is over already still
//               costs 100 to 200 clocks and a tile has five of them: the thread
//               whose turn is next has done its own before the turn comes.
//               (Without turns the two fall into step, both softmaxes and then
//               both MMAs: period 4540 clocks a tile pair.)
//   warps 0-7   softmax of m-tile 0 and 1, one thread per row.  P is handed
//               over in halves (64 keys), so that the first four P V steps run
//               under the exponentials of the second half, and the row sum is
//               taken after the hand-over, under the MMAs: what stays on the
//               chain S -> P -> S of an m-tile is the TMEM load, the row max
//               and the exponentials.
//   warps 12-15 (E4M3) convert V tiles to fp16 with their row scales.
// TMEM (512 columns): S_0/P_0 at 0, S_1/P_1 at 128, O_0 at 256, O_1 at 256 + D.
// Every wait on an mbarrier is bounded; on expiry the CTA reports
// TV_ERR_DEVICE_TIMEOUT for its sequence, drains its copies and returns.
//
// Bound: the tensor pipe for chunks (a chain S, softmax, P V, S per m-tile keeps
// it 60 % busy), HBM for decode.  Measured, D = 128 (device time, the call
// replayed): 2048 tokens over 32768, 64/8 heads, 1.66 ms (1.36 PFLOP/s); four
// 1600-token prompts, 28/4 heads, 97 us; 16 decode tokens over 512 to 4096, 32/8
// heads, 42 us (3.9 TB/s); 4 over 32768 in E4M3, 64/8 heads, 91 us (3.0 TB/s).
//
// Precision.  S, the softmax and O are fp32.  P is rounded to the 16-bit type
// of V for the P V product (bf16; fp16 for an E4M3 cache) and the row sum adds
// the rounded values, so that O / l weights V exactly as the product did.  V of
// an E4M3 cache is the fp32 product of code and scale rounded to fp16.  (In fp16
// arithmetic, the scale rounded too, four 32768-token decodes took 86 us instead
// of 90, and a cached V had another value here than in the tree attention.)
// P of an E4M3 cache is raised by 2^7 (kRaiseLog2).
#include <climits>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int BM = 128;               // rows of one m-tile
constexpr int BN = 128;               // keys per tile
constexpr int kUnitRows = 2 * BM;
constexpr int kSoftmaxThreads = 256;  // warps 0-7: two groups of four warps
constexpr int kKWarp = 8;             // TMA: K tiles
constexpr int kVWarp = 11;            // TMA: V tiles and Q
constexpr int kMmaWarp = 9;           // warps 9, 10 issue the MMAs of m-tile 0, 1
constexpr int kConvWarp = 12;         // E4M3: warps 12-15 convert V tiles to fp16
constexpr int kConvThreads = 128;
// Threads, and registers a thread after the split: the softmax holds a row of
// 128 scores.  bf16: three warpgroups launched with 168 registers, 256 x 208 +
// 128 x 80 = 63488 <= 384 x 168.  E4M3: four launched with 128, 256 x 184 +
// 256 x 72 = 65536 = 512 x 128.
template <bool F8>
struct Shares {
  static constexpr int kThreads = F8 ? 512 : 384;
  static constexpr int kSoftmaxRegs = F8 ? 184 : 208;
  static constexpr int kOtherRegs = F8 ? 72 : 80;
};
// m_run moves only when a tile's maximum exceeds it by 2^8 more than when it was
// set: P stays below 2^8 and the row sum below 2^8 x keys, well inside fp32.
constexpr float kRescaleLog2 = 8.0f;
// Over E4M3 m_run is set 7 below the maximum, so that the fp16 P of the largest
// weights lies between 2^7 and 2^15: weights keep their 11 bits down to 2^-21 of
// the largest instead of 2^-14, and are lost below 2^-32 instead of 2^-25 (with
// 131072 keys, 2^-8 of the whole).  O and the row sum carry the same factor.
constexpr float kRaiseLog2 = 7.0f;
constexpr int kMaxPieces = 16;        // pieces per scheduling round
constexpr int kCheckThreads = 256;    // of the kernel that checks the sequences
constexpr int kSclSlots = 8;          // E4M3: scale slots (tile tau in slot tau % 8)

// cost of a key tile of a unit with one and with two m-tiles, and of a piece
constexpr int kNarrow = 2;
constexpr int kWide = kChunkTileCost;
constexpr int kFixed = kChunkPieceCost;
// a unit is not cut within this many tiles of its ends
constexpr int kMinCut = 2;

// Named barriers (0 is __syncthreads): softmax group 0 alone, both groups, all.
constexpr int kBarGroup0 = 1;
constexpr int kBarPair = 2;
constexpr int kBarCta = 3;            // every thread, from the roles' own loops

// A piece: the key tiles [t0, t1) of one unit that this CTA computes.
struct Piece {
  int b, kvh;
  int tok0;         // first token of the unit (row of q)
  int pos0;         // its position
  int ntok;         // tokens of the unit
  int t0, t1;
  int cut;          // pieces of the unit << 16 | CTA of its first piece (its ticket counter)
  __device__ __forceinline__ int npieces() const { return cut >> 16; }
  __device__ __forceinline__ int vfirst() const { return cut & 0xffff; }
  __device__ __forceinline__ int hi() const { return pos0 + ntok - 1; }
  // partial-result slot of a split unit's piece: the first piece (it holds
  // tile 0) uses its CTA's slot 1, every later piece (it starts its CTA's
  // range) slot 0
  __device__ __forceinline__ int slot() const { return 2 * static_cast<int>(blockIdx.x) + (t0 > 0 ? 0 : 1); }
};

// Shared memory of one CTA.  bf16: K and V tiles of 128 keys x D in rings.
// E4M3 (D = 128): K and raw V tiles of one-byte codes in rings of 3, two
// converted fp16 V tiles, and 8 slots of per-key scales (K, V).
template <int D, bool F8>
struct Layout {
  static_assert(!F8 || D == 128, "an E4M3 cache needs D = 128");
  static constexpr int kHalves = D / 64;               // 64-column halves of a 16-bit row
  static constexpr int kStages = F8 ? 3 : (D == 128 ? 2 : 4);
  static constexpr int kVStages = F8 ? 3 : (D == 128 ? 3 : 5);
  static constexpr int kGroupBytes = kHalves * 1024;   // 8 rows of a 16-bit tile
  static constexpr int kTileBytes = BN * D * 2;
  static constexpr int kKTileBytes = F8 ? BN * D : kTileBytes;  // a K or raw V tile as loaded
  static constexpr int kQLines = F8 ? 1 : kHalves;     // 128-byte lines of a Q row
  static constexpr int kQLineBytes = kUnitRows * 128;  // Q: [line][256 rows][128 B]
  static constexpr int kQ = 0;
  static constexpr int kKRing = kQ + kQLines * kQLineBytes;
  static constexpr int kVRing = kKRing + kStages * kKTileBytes;
  static constexpr int kV16 = kVRing + kVStages * kKTileBytes;
  static constexpr int kV16Bytes = F8 ? 2 * kTileBytes : 0;
  static constexpr int kScl = kV16 + kV16Bytes;        // F8: K scales [8][128], V scales [VS][128]
  static constexpr int kVScl = kScl + (F8 ? kSclSlots * BN * 4 : 0);
  static constexpr int kSclBytes = F8 ? (kSclSlots + kVStages) * BN * 4 : 0;
  static constexpr int kPieces = kScl + kSclBytes;
  static constexpr int kPiecesBytes = kMaxPieces * static_cast<int>(sizeof(Piece));
  static constexpr int kXch = kPieces + kPiecesBytes;  // [128] (m, l) of group 1, narrow pieces
  static constexpr int kXchBytes = BM * 8;
  static constexpr int kBar = kXch + kXchBytes;
  // kfull, kempty [S], vfull, vempty [VS], s_full, p_a, p_b, o_done, drain,
  // turn [2], q_full, q_empty, hand [2], v16full, v16empty [2], sfull [8]
  static constexpr int kNumBars = 2 * kStages + 2 * kVStages + 16 + (F8 ? 4 + kSclSlots : 0);
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kMiscBytes = 32;
  static constexpr int kTotal = kMisc + kMiscBytes;
  static constexpr int kAlloc = kTotal + 1024;  // slack for 1024-byte alignment
  // the schedule's scratch (a chunk of 256 sequences) lies over Q, which is
  // written only after the piece list is built
  static constexpr int kSeq = kQ;                      // [4][256] ints, then 8 warp sums
  static constexpr int kTmemCols = 512;
  static_assert(4 * 256 * 4 + 32 <= kQLines * kQLineBytes, "schedule scratch fits over Q");
  static_assert(kAlloc <= 232448, "shared memory per CTA");
};

struct Misc {
  uint32_t tmem_base;
  int abort;
  int npieces;                // pieces of this round
  int more;                   // another round follows
  int merge;                  // this CTA merges the current split unit
};
static_assert(sizeof(Misc) <= Layout<128, true>::kMiscBytes, "Misc fits its area");

// Partial-result slot: unnormalised O (fp32) as float4 [D/4][rows of the
// unit], (m, l) per row, a flag.
template <int D>
struct Slot {
  static constexpr size_t kO = 0;
  static constexpr size_t kMl = static_cast<size_t>(kUnitRows) * D * 4;
  static constexpr size_t kFlag = kMl + kUnitRows * 8;
  static constexpr size_t kBytes = kFlag + 256;
};

// max of three (NaN operands are ignored, as in fmaxf)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void named_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

__device__ __forceinline__ void record_status(int32_t* status, int b, int code) {
  atomicMax(status + b, code);
}

// Waits for this thread's TMEM loads; the registers they fill are operands, so
// that nothing that reads them is moved ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 16 consecutive TMEM columns of this thread's lane, with the wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Two values -> fp16 (nearest even; 65504 at most): at scores past 2^24, whose
// differences are off by more than 1, P could pass 2^16 by rounding alone.
__device__ __forceinline__ uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bits 0 .. n-1 of a 32-bit word (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// ---------------------------------------------------------------- schedule
// The keys that a unit whose first token sits at pos0 sees, besides those past
// its last token: keys < sinks and keys >= lo.  Tile t < st of the unit is key
// tile t, later ones key tile t + skip.  When the whole context is visible (no
// window, or one that reaches the sinks), lo = st = skip = 0.
struct Extent {
  int lo, st, skip;
  __device__ __forceinline__ int key_tile(int t) const { return t < st ? t : t + skip; }
};
__device__ __forceinline__ Extent extent_of(const ChunkArgs& a, int pos0) {
  Extent e;
  e.lo = e.st = e.skip = 0;
  if (a.window > 0 && pos0 - a.window + 1 > a.sinks) {
    e.lo = pos0 - a.window + 1;
    e.st = (a.sinks + BN - 1) / BN;
    e.skip = max(0, e.lo / BN - e.st);
  }
  return e;
}

// Unit u of a chunk of C tokens that starts at position ctx: its first
// position, tokens and key tiles.
struct Unit {
  int pos0, ntok, T;
};
__device__ __forceinline__ Unit unit_of(const ChunkArgs& a, int ctx, int C, int u) {
  Unit x;
  const int tok = u * a.unit_tokens;
  x.ntok = min(a.unit_tokens, C - tok);
  x.pos0 = ctx + tok;
  x.T = (x.pos0 + x.ntok - 1) / BN + 1 - extent_of(a, x.pos0).skip;
  return x;
}

struct SeqInfo {
  int n0, C, len;
  int units;        // per KV head; 0 for an empty chunk or a malformed sequence
};

__device__ __forceinline__ SeqInfo seq_info(const ChunkArgs& a, int b) {
  SeqInfo s;
  s.n0 = __ldg(a.token_offsets + b);
  s.len = __ldg(a.seq_lens + b);
  const bool bad = __ldcg(a.status + b) == kBadTree;
  s.C = bad ? 0 : __ldg(a.token_offsets + b + 1) - s.n0;
  s.units = (s.C + a.unit_tokens - 1) / a.unit_tokens;
  return s;
}

// Exclusive scan over the 256 softmax threads; *total = the sum.
__device__ __noinline__ int scan256(int v, int* scratch, int sid, int* total) {
  const int lane = sid & 31, w = sid >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[w] = x;
  named_sync(kBarPair, kSoftmaxThreads);
  int before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int s = scratch[k];
    if (k < w) before += s;
    all += s;
  }
  named_sync(kBarPair, kSoftmaxThreads);  // scratch may be reused
  *total = all;
  return before + x - v;
}

// Range boundaries of V CTAs on a line of W tiles: CTA v takes [start(v),
// start(v+1)) with start(v) = floor(v W / V), computed as v q + floor(v r / V)
// with W = q V + r.  floor(v r / V) (v r <= V^2 < 2^24) comes from the fp32
// product with 1/V, within one of the quotient, and one integer correction.
struct Line {
  int V, q, r;
  float rV;  // 1 / V
  float VW;  // V / W
  __device__ __forceinline__ int start(int v) const {
    const int n = v * r;
    int k = static_cast<int>(static_cast<float>(n) * rV);
    if (k * V > n) {
      --k;
    } else if ((k + 1) * V <= n) {
      ++k;
    }
    return v * q + k;
  }
  // the CTA whose range holds position p (0 <= p < W): the fp32 estimate
  // p V / W is within two of it; exact integer steps finish it
  __device__ __forceinline__ int owner(int p) const {
    int o = min(V - 1, max(0, static_cast<int>(static_cast<float>(p) * VW)));
#pragma unroll 1
    for (int k = 0; k < 4 && o > 0 && start(o) > p; ++k) --o;
#pragma unroll 1
    for (int k = 0; k < 4 && o + 1 < V && start(o + 1) <= p; ++k) ++o;
    return o;
  }
};

// The key tile at which a range boundary at offset x of a unit of T tiles of
// cost w cuts it (0: before it, T: after it).
__device__ __forceinline__ int cut_at(int x, int T, int w) {
  const int t = x < kFixed ? 0 : (w == kWide ? (x - kFixed) / kWide : (x - kFixed) / kNarrow);
  if (t >= T) return T;
  return t < kMinCut ? 0 : (t > T - kMinCut ? T : t);
}

// Builds this CTA's pieces of scheduling round `round` into shared memory
// (the 256 softmax threads).  `line` is filled in round 0.  Sequences are
// taken 256 at a time, and the units of such a chunk 256 at a time, one per
// thread: a unit is hkv consecutive runs of the line, one per KV head.
template <int D, bool F8>
__device__ void build_schedule(const ChunkArgs& a, uint8_t* smem, int round, int sid, Line* line) {
  using Ly = Layout<D, F8>;
  Misc* misc = reinterpret_cast<Misc*>(smem + Ly::kMisc);
  Piece* pieces = reinterpret_cast<Piece*>(smem + Ly::kPieces);
  int* seq_u = reinterpret_cast<int*>(smem + Ly::kSeq);  // first unit of each sequence
  int* seq_n0 = seq_u + 256;
  int* seq_c = seq_n0 + 256;
  int* seq_ctx = seq_c + 256;
  int* scratch = seq_ctx + 256;

  int units = 0;      // units of the current chunk of sequences
  int loaded = -1;    // the chunk in shared memory
  auto load_chunk = [&](int base) {
    if (loaded == base) return;
    const int b = base + sid;
    SeqInfo s;
    s.units = s.n0 = s.C = s.len = 0;
    if (b < a.batch) s = seq_info(a, b);
    seq_u[sid] = scan256(s.units, scratch, sid, &units);
    seq_n0[sid] = s.n0;
    seq_c[sid] = s.C;
    seq_ctx[sid] = s.len - s.C;
    loaded = base;
    named_sync(kBarPair, kSoftmaxThreads);
  };
  // Pass 0 (round 0 only) adds the line up, pass 1 emits the pieces.  One copy
  // of the code serves both: run once, it costs its instructions' way from L2.
  // A batch with at most 256 units is located once.
  const int v = static_cast<int>(blockIdx.x);
  Unit x;
  int xi = 0, xu = 0;
  bool kept = false;
  int count = 0;  // pieces of this CTA so far (all rounds)
#pragma unroll 1
  for (int pass = round == 0 ? 0 : 1; pass < 2; ++pass) {
    int s_v = 0, e_v = INT_MAX;
    if (pass == 1) {
      s_v = v < line->V ? line->start(v) : 0;
      e_v = v < line->V ? line->start(v + 1) : 0;
    }
    int cum = 0;  // line position of the next group of units
#pragma unroll 1
    for (int base = 0; base < a.batch && cum < e_v; base += kSoftmaxThreads) {
      load_chunk(base);
#pragma unroll 1
      for (int ub = 0; ub < units && cum < e_v; ub += kSoftmaxThreads) {
        const bool have = ub + sid < units;
        if (have && !kept) {
          // unit j of the chunk: its sequence (the last whose first unit is
          // <= j: sequences without units share the next one's), its extent
          const int j = ub + sid;
          xi = 0;
#pragma unroll 1
          for (int step = 128; step > 0; step >>= 1)
            if (seq_u[xi + step] <= j) xi += step;
          xu = j - seq_u[xi];
          x = unit_of(a, seq_ctx[xi], seq_c[xi], xu);
        }
        const int w = x.ntok * a.group > BM ? kWide : kNarrow;
        const int run = x.T * w + kFixed;
        const int len = have ? run * a.hkv : 0;
        int tot;
        const int c0 = cum + scan256(len, scratch, sid, &tot);
        cum += tot;
        if (pass == 0) continue;
        // KV heads [h0, h1) of this unit have tiles in [s_v, e_v)
        int h0 = 0, h1 = 0;
        if (have && c0 < e_v && c0 + len > s_v) {
          h0 = max(0, s_v - c0) / run;
          h1 = (min(e_v - c0, len) + run - 1) / run;
          if (cut_at(s_v - c0 - h0 * run, x.T, w) == x.T) ++h0;
          if (h1 > h0 && cut_at(e_v - c0 - (h1 - 1) * run, x.T, w) == 0) --h1;
          // (a range within one unit may have neither)
          if (h1 == h0 + 1 && cut_at(s_v - c0 - h0 * run, x.T, w) >= cut_at(e_v - c0 - h0 * run, x.T, w)) h1 = h0;
        }
        int ptot;
        int k = count + scan256(max(0, h1 - h0), scratch, sid, &ptot) - round * kMaxPieces;
        count += ptot;
#pragma unroll 1
        for (int h = h0; h < h1; ++h, ++k) {
          if (k < 0 || k >= kMaxPieces) continue;
          const int u0 = c0 + h * run;  // line position of the unit
          Piece& pc = pieces[k];
          const int t0 = cut_at(s_v - u0, x.T, w), t1 = cut_at(e_v - u0, x.T, w);
          pc.b = base + xi;
          pc.kvh = h;
          pc.tok0 = seq_n0[xi] + xu * a.unit_tokens;
          pc.pos0 = x.pos0;
          pc.ntok = x.ntok;
          pc.t0 = t0;
          pc.t1 = t1;
          int vf = v, np = 1;
          if (t0 > 0 || t1 < x.T) {
            // the CTAs of the unit's first and last tiles: every one between
            // them has a piece
            vf = line->owner(u0);
            while (cut_at(line->start(vf + 1) - u0, x.T, w) == 0) ++vf;
            int vl = line->owner(u0 + run - 1);
            while (cut_at(line->start(vl) - u0, x.T, w) == x.T) --vl;
            np = vl - vf + 1;
          }
          pc.cut = np << 16 | vf;
        }
      }
      kept = pass == 0 && a.batch <= kSoftmaxThreads && units <= kSoftmaxThreads;
      named_sync(kBarPair, kSoftmaxThreads);  // the sequence arrays are rewritten
    }
    if (pass == 0) {
      line->V = max(1, min(a.vctas, cum / max(1, a.min_range)));
      line->q = cum / line->V;
      line->r = cum % line->V;
      line->rV = 1.0f / static_cast<float>(line->V);
      line->VW = cum > 0 ? static_cast<float>(line->V) / static_cast<float>(cum) : 0.0f;
    }
  }
  if (sid == 0) {
    const int n = count - round * kMaxPieces;
    misc->npieces = max(0, min(kMaxPieces, n));
    misc->more = n > kMaxPieces;
  }
  fence_proxy_async_smem();  // the scratch lies where TMA writes Q
}

// ---------------------------------------------------------------- output
// Where the lanes of a quad write: lane r of a quad stores 16-byte piece r of
// 64 bytes of the rows of all four lanes, one row after the other, so that a
// warp's store covers 64 consecutive bytes of 8 rows.  (A lane storing its own
// row touches 32 lines a store: about 2 clocks each, 4000 clocks for an m-tile.)
struct QuadRows {
  uint8_t* at[4];  // row k of the quad, at byte 16 r; null: not written
};
template <int D>
__device__ __forceinline__ QuadRows quad_rows(const ChunkArgs& a, size_t row, bool live) {
  const int lane = threadIdx.x & 31;
  const unsigned long long mine =
      live ? reinterpret_cast<unsigned long long>(a.out) + row * D * (a.out_fp32 ? 4 : 2) : 0ull;
  QuadRows q;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long p = __shfl_sync(0xffffffffu, mine, (lane & ~3) + k);
    q.at[k] = p ? reinterpret_cast<uint8_t*>(p) + (lane & 3) * 16 : nullptr;
  }
  return q;
}
// Stores piece c = w[c] of each lane's row, c = 0 .. 3, at byte `off` of the
// rows: a 4 x 4 transposition inside the quad (two exchange steps), then a
// store per row.
__device__ __forceinline__ void quad_store(const QuadRows& q, int off, uint4 (&w)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
      uint4& lo = w[i];
      uint4& hi = w[i | bit];
      uint4 x = up ? lo : hi;
      x.x = __shfl_xor_sync(0xffffffffu, x.x, bit);
      x.y = __shfl_xor_sync(0xffffffffu, x.y, bit);
      x.z = __shfl_xor_sync(0xffffffffu, x.z, bit);
      x.w = __shfl_xor_sync(0xffffffffu, x.w, bit);
      if (up) lo = x; else hi = x;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (q.at[k]) *reinterpret_cast<uint4*>(q.at[k] + off) = w[k];
}
// Writes columns c0 .. c0 + 31 of each lane's output row (fp32 or bf16), by
// the whole warp.
__device__ __forceinline__ void store_rows32(const ChunkArgs& a, const QuadRows& q, int c0, const float (&v)[32]) {
  uint4 w[4];
  if (a.out_fp32) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float* x = v + 16 * half + 4 * c;
        w[c] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      }
      quad_store(q, (c0 + 16 * half) * 4, w);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float* x = v + 8 * c;
      w[c] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    quad_store(q, c0 * 2, w);
  }
}

// The slots of a split unit's pieces.
template <int D>
struct Slots {
  const uint8_t *first, *rest;
  __device__ __forceinline__ Slots(const ChunkArgs& a, const Piece& pc)
      : first(a.slots + static_cast<size_t>(2 * pc.vfirst() + 1) * Slot<D>::kBytes),
        rest(a.slots + static_cast<size_t>(2 * pc.vfirst()) * Slot<D>::kBytes) {}
  __device__ __forceinline__ const uint8_t* at(int s) const {
    return s == 0 ? first : rest + static_cast<size_t>(2 * s) * Slot<D>::kBytes;
  }
  __device__ __forceinline__ int flag(int s) const {
    return __ldcg(reinterpret_cast<const int*>(at(s) + Slot<D>::kFlag));
  }
  __device__ __forceinline__ float2 ml(int s, int row) const {
    return __ldcg(reinterpret_cast<const float2*>(at(s) + Slot<D>::kMl) + row);
  }
  __device__ __forceinline__ const float4* o(int s, int row) const {
    return reinterpret_cast<const float4*>(at(s) + Slot<D>::kO) + row;
  }
};

// This thread's row of the piece's O: O_h of its m-tile, or, in a narrow piece
// whose key tiles the two groups took in turn, w0 O_0 + w1 O_1 against the
// larger maximum.
template <int D>
struct OwnO {
  uint32_t tmem;  // O_h
  bool two;
  float w0, w1;
  __device__ __forceinline__ void load(int c0, float (&v)[32]) const {
    uint32_t o[32];
    tmem_ld32(tmem + c0, o);
    tmem_ld_wait32(o);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]);
    if (two) {
      tmem_ld32(tmem + D + c0, o);
      tmem_ld_wait32(o);
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = w0 * v[k] + w1 * __uint_as_float(o[k]);
    }
  }
};

// Merges the pieces of a split unit: O = sum_s 2^(m_s - M) O_s /
// sum_s 2^(m_s - M) l_s in piece order.  Both forms run once or twice in a
// launch, at its end, and stay rolled: what such code costs besides its loads
// is its instructions' way from L2.
//
// A thread per row (more than half as many rows as threads): piece `own` from
// TMEM and registers (bit for bit what its slot would hold), the others from
// their slots, W columns of a piece in flight.  (Writing and reading its own
// slot too, 16 columns at a time, took 28000 clocks of a 250-row unit.  E4M3: W
// = 32; 64 spill, four 32768-token decodes 92 us instead of 86.)
template <int D, int W>
__device__ void merge_rows(const ChunkArgs& a, const Piece& pc, int ur, int own, float m_own, float l_own,
                           int bad, const OwnO<D>& o) {
  const Slots<D> sl(a, pc);
  const int np = pc.npieces(), rows = pc.ntok * a.group;
  const bool live = ur < rows;
  const int row = min(ur, rows - 1);
  float M = m_own;
#pragma unroll 2
  for (int s = 0; s < np; ++s) {
    if (s == own) continue;
    bad |= sl.flag(s);
    M = fmaxf(M, sl.ml(s, row).x);
  }
  const QuadRows quad =
      quad_rows<D>(a, static_cast<size_t>(pc.tok0 + row / a.group) * a.hq + pc.kvh * a.group + row % a.group, live);
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += W) {
    float l = 0.0f;
    float acc[W];
#pragma unroll
    for (int k = 0; k < W; ++k) acc[k] = 0.0f;
#pragma unroll 1
    for (int s = 0; s < np; ++s) {
      float x[W];
      float2 ml = make_float2(m_own, l_own);
      if (s == own) {
#pragma unroll
        for (int c = 0; c < W; c += 32) o.load(c0 + c, *reinterpret_cast<float(*)[32]>(&x[c]));
      } else {
        ml = sl.ml(s, row);
        const float4* o4 = sl.o(s, row) + (c0 / 4) * rows;
#pragma unroll
        for (int k = 0; k < W / 4; ++k) *reinterpret_cast<float4*>(&x[4 * k]) = __ldcg(o4 + k * rows);
      }
      const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
      l += w * ml.y;
#pragma unroll
      for (int k = 0; k < W; ++k) acc[k] += w * x[k];
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) acc[k] = bad ? 0.0f : acc[k] * inv;
#pragma unroll
    for (int c = 0; c < W; c += 32)
      store_rows32(a, quad, c0 + c, *reinterpret_cast<const float(*)[32]>(&acc[c]));
  }
}

// Several threads per row (a few decode rows, split many ways): every piece
// from its slot, thread `sub` of a row taking groups sub, sub + step, .. of 4
// columns.
template <int D>
__device__ void merge_groups(const ChunkArgs& a, const Piece& pc, int ur, int step) {
  const Slots<D> sl(a, pc);
  const int np = pc.npieces(), rows = pc.ntok * a.group;
  const int row = ur % rows, sub = ur / rows;
  if (sub >= step) return;
  int bad = 0;
  float M = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < np; ++s) {
    bad |= sl.flag(s);
    M = fmaxf(M, sl.ml(s, row).x);
  }
  const size_t out_row = static_cast<size_t>(pc.tok0 + row / a.group) * a.hq + pc.kvh * a.group + row % a.group;
#pragma unroll 1
  for (int d4 = sub; d4 < D / 4; d4 += step) {
    float l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < np; ++s) {
      const float2 ml = sl.ml(s, row);
      const float4 o = __ldcg(sl.o(s, row) + d4 * rows);
      const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
      l += w * ml.y;
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const float4 v = bad ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                         : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (a.out_fp32) {
      reinterpret_cast<float4*>(static_cast<float*>(a.out) + out_row * D)[d4] = v;
    } else {
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * D)[d4] =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  }
}

// Runs first: a CTA per sequence checks its extent and every page that some row
// of it sees, writes its status and zeroes the rows of a malformed one, so that
// the attention kernel meets sound sequences only.  The rows of sequences behind a
// chunk of negative length would be counted twice, and the line of work could pass
// 32 bits: they are malformed too, and rows that an earlier sequence has are not
// theirs.  The attention kernel may start while this one runs (programmatic
// dependent launch); it waits for its end before it reads a status.
__global__ void __launch_bounds__(kCheckThreads) chunk_check_kernel(const __grid_constant__ ChunkArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int decrease;
  const int tid = threadIdx.x;
  if (tid == 0) decrease = INT_MAX;
  __syncthreads();
  for (int i = tid; i < a.batch; i += kCheckThreads)
    if (__ldg(a.token_offsets + i + 1) < __ldg(a.token_offsets + i)) atomicMin(&decrease, i);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.vctas; i += kCheckThreads) a.counters[i] = 0;  // tickets
  __syncthreads();
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int n0 = __ldg(a.token_offsets + b), n1 = __ldg(a.token_offsets + b + 1), len = __ldg(a.seq_lens + b);
    const long long c = static_cast<long long>(n1) - n0;
    bool bad = c < 0 || b > decrease || (c > 0 && (n0 < 0 || n1 > a.total_tokens || len < c || len > a.max_len));
    if (!bad && c > 0) {
      // pages [0, s) of the sinks and [w, the last one]
      const int ctx = len - static_cast<int>(c);
      const int lo = extent_of(a, ctx).lo;  // (the first token's: no later row sees more)
      const int w = lo / 16, s = min((a.sinks + 15) / 16, w);
      const int pages = s + (len - 1) / 16 + 1 - w;
      const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_blocks_per_seq;
#pragma unroll 8
      for (int i = tid; i < pages; i += kCheckThreads) {
        const int blk = __ldg(table + (i < s ? i : i - s + w));
        bad |= blk < 0 || blk >= a.num_blocks;
      }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) a.status[b] = bad ? kBadTree : kOk;
    if (!bad) continue;
    const size_t row_bytes = static_cast<size_t>(a.hq) * a.head_dim * (a.out_fp32 ? 4 : 2);
    const long long r0 = max(0, max(n0, b > decrease ? __ldg(a.token_offsets + decrease) : 0));
    const long long r1 = min(n1, a.total_tokens);
    if (r1 <= r0) continue;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + r0 * row_bytes);
    for (size_t k = tid; k < (r1 - r0) * row_bytes / 16; k += kCheckThreads) dst[k] = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- the kernel
template <int D, bool F8>
__global__ void __launch_bounds__(Shares<F8>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkMaps maps) {
  using Ly = Layout<D, F8>;
  using Sl = Slot<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr int kStages = Ly::kStages;
  constexpr int kVStages = Ly::kVStages;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + Ly::kBar);
  uint64_t* kempty = kfull + kStages;
  uint64_t* vfull = kempty + kStages;
  uint64_t* vempty = vfull + kVStages;    // F8: the converters have read the raw V
  uint64_t* s_full = vempty + kVStages;   // [2]: S_h(t) complete (and every MMA before it)
  uint64_t* p_a = s_full + 2;             // [2]: P_h(t) of keys 0 .. 63 in TMEM (128 arrivals)
  uint64_t* p_b = p_a + 2;                // [2]: P_h(t) of keys 64 .. 127
  uint64_t* o_done = p_b + 2;             // [2]: the last P_h V of a piece complete
  uint64_t* drain = o_done + 2;           // [2]: every MMA of m-tile h so far complete (once per round)
  uint64_t* turn = drain + 2;             // [2]: m-tile h may issue (units with both)
  uint64_t* q_full = turn + 2;            // Q of a piece in shared memory
  uint64_t* q_empty = q_full + 1;         // the last S of both m-tiles of a piece complete
  uint64_t* hand = q_empty + 1;           // [2]: S_1, P_1 and O_1 pass to the MMA thread of m-tile h
  uint64_t* v16full = hand + 2;           // F8 [2]: V(t) converted (128 arrivals)
  uint64_t* v16empty = v16full + 2;       // F8 [2]: the P V of tile t complete
  uint64_t* sfull = v16empty + 2;         // F8 [8]: the scales of tile t landed (32 arrivals)
  Misc* misc = reinterpret_cast<Misc*>(smem + Ly::kMisc);
  Piece* pieces = reinterpret_cast<Piece*>(smem + Ly::kPieces);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  if (tid == 0) {
    misc->abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 2);  // one arrival per m-tile
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&vfull[s], F8 ? 33 : 1);  // E4M3: and every lane's scales
      mbar_init(&vempty[s], F8 ? kConvThreads : 2);
    }
    if constexpr (F8) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(&v16full[k], kConvThreads);
        mbar_init(&v16empty[k], 2);
      }
      for (int k = 0; k < kSclSlots; ++k) mbar_init(&sfull[k], 32);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&p_a[h], BM);
      mbar_init(&p_b[h], BM);
      mbar_init(&o_done[h], 1);
      mbar_init(&drain[h], 1);
      mbar_init(&turn[h], 1);
      mbar_init(&hand[h], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&misc->tmem_base, Ly::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // status and counters are zero
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  volatile int* abort_flag = &misc->abort;
  const int g = a.group;

  // Progress kept across pieces and rounds (ring slots and barrier phases):
  // g_tile, g_piece = K/V tiles and pieces of every earlier round; my_tiles =
  // the tiles of this softmax group so far; tiles0, tiles1 = the tiles of
  // groups 0 and 1, my_turns and my_hands = the turns and take-overs of this MMA
  // thread.
  int g_tile = 0, g_piece = 0, my_tiles = 0, tiles0 = 0, tiles1 = 0, my_turns = 0, my_hands = 0;

  // Each role runs the scheduling rounds in a loop of its own (its registers
  // are its own too).  A round: the softmax warps build the piece list, every
  // role works through it, and all meet again once the round's copies have
  // landed and its MMAs are complete.
  auto rounds = [&](auto&& build, auto&& work) {
    for (int round = 0;; ++round) {
      build(round);
      named_sync(kBarCta, Shares<F8>::kThreads);
      const int npieces = misc->npieces;
      const bool more = misc->more != 0;
      if (npieces == 0) break;
      work(round, npieces);
      tc_fence_before();
      named_sync(kBarCta, Shares<F8>::kThreads);
      tc_fence_after();
      for (int p = 0; p < npieces; ++p) g_tile += pieces[p].t1 - pieces[p].t0;
      g_piece += npieces;
      const bool stop = !more || misc->abort;
      named_sync(kBarCta, Shares<F8>::kThreads);  // the piece list is rebuilt next round
      if (stop) break;
    }
  };
  auto nothing = [](int) {};

  if (warp >= kKWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shares<F8>::kOtherRegs));
    if (warp == kKWarp || warp == kVWarp) {
      rounds(nothing, [&](int, int npieces) {
      // ------------------------------------------------------ K producer, V and Q producer
      // A tile: lane 0 arms the slot's barrier, then lane u issues the box of
      // page u.  A K slot is free again once the last S of its tile is done, a
      // V slot once the last P V is.  The next tile's block ids are read ahead.
      // (One warp polling for both took 3300 clocks a tile, more than an E4M3
      // tile has at the HBM rate.)
      constexpr int kPages = BN / 16;
      constexpr int kUnseen = -1;  // no row of the unit sees the page -> zeros
      const bool is_v = warp == kVWarp;
      const int stages = is_v ? kVStages : kStages;
      uint64_t* full = is_v ? vfull : kfull;
      uint64_t* empty = is_v ? vempty : kempty;
      uint8_t* ring = smem + (is_v ? Ly::kVRing : Ly::kKRing);
      const CUtensorMap* map = is_v ? &maps.v_pool : &maps.k_pool;
      const float* scales = is_v ? a.v_scale : a.k_scale;
      float* scl_ring = reinterpret_cast<float*>(smem + (is_v ? Ly::kVScl : Ly::kScl));
      bool ok = true;
      int tau = g_tile;
      int st = g_tile % stages, ph = (g_tile / stages) & 1;  // ring slot and phase of tile tau
      int p = 0;
      for (; p < npieces && ok; ++p) {
        const Piece& pc = pieces[p];
        const Extent ext = extent_of(a, pc.pos0);
        const int t1 = pc.t1, hi = pc.hi(), kvh = pc.kvh;
        const int32_t* table = a.block_table + static_cast<size_t>(pc.b) * a.max_blocks_per_seq;
        auto fetch_block = [&](int t) -> int {
          const int lp = ext.key_tile(t) * kPages + lane;
          const int k0 = lp * 16;
          return lane < kPages && t < t1 && k0 <= hi && (k0 < a.sinks || k0 + 15 >= ext.lo) ? __ldg(table + lp) : kUnseen;
        };
        int blk = fetch_block(pc.t0);
        if (is_v) {
          // Q (q_tokens tokens of g heads, rows past the unit are other tokens'
          // or zeros and unused), once the S of the piece before are complete
          const int n = g_piece + p;
          ok = n == 0 || __all_sync(0xffffffffu, mbar_wait(q_empty, (n - 1) & 1, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full, Ly::kQLines * a.q_tokens * g * 128);
            for (int l = 0; l < Ly::kQLines; ++l)
              tma_load_3d(smem + Ly::kQ + l * Ly::kQLineBytes, &maps.q, q_full, l * 64, kvh * g, pc.tok0);
          }
          __syncwarp();
        }
        for (int t = pc.t0; t < t1; ++t) {
          const int page_id = blk;
          const bool good = page_id >= 0 && page_id < a.num_blocks;
          const int page = good ? page_id * a.hkv + kvh : a.num_blocks * a.hkv;  // out of bounds: zero fill
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], Ly::kKTileBytes);
          __syncwarp();
          if (lane < kPages) {
            uint8_t* dst = ring + st * Ly::kKTileBytes + lane * (Ly::kKTileBytes / kPages);
            if constexpr (F8) {
              tma_load_3d(dst, map, &full[st], 0, 0, page);
            } else {
              tma_load_5d(dst, map, &full[st], 0, 0, 0, 0, page);
            }
          }
          blk = fetch_block(t + 1);
          if constexpr (F8) {
            // the tile's scales: lane u the keys 4u .. 4u+3 (page u / 4); 0
            // where the page is not read.  K: slot tau % 8 with a barrier of its
            // own (the softmax reads them later than the MMA the tile); V: with
            // the tile.
            const int from = __shfl_sync(0xffffffffu, good ? page : -1, lane >> 2);
            const size_t idx = from >= 0 ? static_cast<size_t>(from) * 16 + (lane & 3) * 4 : 0;
            cpa16_zfill(scl_ring + (is_v ? st : tau % kSclSlots) * BN + 4 * lane, scales + idx, from >= 0 ? 16 : 0);
            cpa_arrive_noinc(is_v ? &vfull[st] : &sfull[tau % kSclSlots]);
          }
          ++tau;
          if (++st == stages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        misc->abort = 1;
        if (lane == 0) record_status(a.status, pieces[min(p, npieces - 1)].b, kDeviceTimeout);
      }
      if constexpr (F8) cpa_wait_all();  // this lane's scale copies have landed
      if (lane == 0) {
        // every issued copy has landed before the ring is reused or the CTA
        // exits (at most a ring of them can still be in flight)
        for (int t = max(g_tile, tau - stages); t < tau; ++t)
          mbar_wait(&full[t % stages], (t / stages) & 1);
        if (is_v && ok) mbar_wait(q_full, (g_piece + npieces - 1) & 1);
      }
      __syncwarp();
      });
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      rounds(nothing, [&](int round, int npieces) {
      // ------------------------------------------------------ MMA issuer of m-tile h
      if (lane == 0) {
        const int h = warp - kMmaWarp;
        // bf16: both products on kind::f16 in bf16.  E4M3: S on kind::f8f6f4
        // over the codes, P V on kind::f16 in fp16.
        constexpr uint32_t idesc_s = F8 ? idesc_e4m3(BM, BN) : idesc_bf16(BM, BN, 0);
        constexpr uint32_t idesc_o = F8 ? idesc_f16(BM, D, 1) : idesc_bf16(BM, D, 1);
        // K (K-major): 8-row groups at kGroupBytes (16-bit) or 1024
        // (8-bit), 64-column halves at +1024.  V (MN-major): 8-key groups at
        // kGroupBytes, column halves at +1024.
        // Q (K-major): 8-row groups at 1024, lines at kQLineBytes.
        constexpr uint32_t kKRow8 = F8 ? 1024 : Ly::kGroupBytes;
        const uint64_t dk0 = smem_desc(smem_u32(smem + Ly::kKRing), 16, kKRow8);
        const uint64_t dv0 = smem_desc(smem_u32(smem + (F8 ? Ly::kV16 : Ly::kVRing)), 1024, Ly::kGroupBytes);
        const uint64_t dq0 = smem_desc(smem_u32(smem + Ly::kQ), 16, 1024);
        uint64_t* vready = F8 ? v16full : vfull;  // V(t) as the P V reads it, and its release
        uint64_t* vdone = F8 ? v16empty : vempty;
        constexpr int kVSlots = F8 ? 2 : kVStages;
        auto k_wait = [&](int t) { return mbar_wait(&kfull[t % kStages], (t / kStages) & 1, abort_flag); };
        auto v_wait = [&](int t) { return mbar_wait(&vready[t % kVSlots], (t / kVSlots) & 1, abort_flag); };
        auto issue_s = [&](int x, int m, int t) {  // S_x = Q_m K(t)^T
          const uint64_t dk = dk0 + static_cast<uint64_t>((t % kStages) * (Ly::kKTileBytes >> 4));
          const uint64_t dq = dq0 + static_cast<uint64_t>(m * (BM * 128 >> 4));
          const uint32_t tmem_s = tmem + x * BN;
          if constexpr (F8) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)  // 32 codes of each row per MMA
              mma_f8_ss(tmem_s, dq + kk * 2, dk + kk * 2, idesc_s, kk > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t in = (kk & 3) * 2;  // 32 bytes within the 128-byte line
              mma_bf16_ss(tmem_s, dq + (kk >> 2) * (Ly::kQLineBytes >> 4) + in, dk + (kk >> 2) * 64 + in,
                          idesc_s, kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(&s_full[x]);
        };
        // O_x (+)= P_x V(t) over keys 64 half .. 64 half + 63
        auto issue_pv = [&](int x, int t, int half, bool acc) {
          const uint64_t dv = dv0 + static_cast<uint64_t>((t % kVSlots) * (Ly::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) {
            const int kk = half * (BN / 32) + k;
            mma_bf16_ts(tmem + 256 + x * D, tmem + x * BN + kk * 8, dv + ((kk * 2 * Ly::kGroupBytes) >> 4),
                        idesc_o, (acc || k > 0) ? 1u : 0u);
          }
        };
        // turns are taken in wide pieces, m-tile 0 first
        auto turn_wait = [&]() {
          const int n = my_turns - (h == 0 ? 1 : 0);
          return n < 0 || mbar_wait(&turn[h], n & 1, abort_flag);
        };
        auto turn_pass = [&]() {
          mbar_arrive(&turn[h ^ 1]);
          ++my_turns;
        };
        auto count = [&](int T, bool narrow) {
          tiles0 += narrow ? (T + 1) / 2 : T;
          tiles1 += narrow ? T / 2 : T;
        };
        // S_1, P_1 and O_1 belong to warp 9 in narrow pieces and to warp 10 in
        // wide ones; MMAs of two threads are not ordered, so where the kind
        // changes the next owner waits until the last one's are complete
        auto is_narrow = [&](int p) { return pieces[p].ntok * g <= BM; };
        auto hand_over = [&](int p, bool narrow) {
          if (p + 1 < npieces && is_narrow(p + 1) != narrow && h == (narrow ? 0 : 1)) mma_commit(&hand[h ^ 1]);
        };
        auto take_over = [&](int p, bool narrow) {
          if (p == 0 || is_narrow(p - 1) == narrow || h != (narrow ? 0 : 1)) return true;
          return mbar_wait(&hand[h], my_hands++ & 1, abort_flag);
        };
        bool ok = true;
        int tau = g_tile;
        for (int p = 0; p < npieces && ok; ++p) {
          const int T = pieces[p].t1 - pieces[p].t0;
          const bool narrow = is_narrow(p);
          ok = mbar_wait(q_full, (g_piece + p) & 1, abort_flag) && take_over(p, narrow);
          if (!ok) break;
          if (narrow && h == 1) {
            // warp 9 issues for both groups: these arrivals keep the rings turning
            mbar_arrive(q_empty);
            for (int t = tau; t < tau + T && ok; ++t) {
              ok = k_wait(t);
              if (ok) mbar_arrive(&kempty[t % kStages]);
              ok = ok && v_wait(t);
              if (ok) mbar_arrive(&vdone[t % kVSlots]);
            }
            count(T, true);
            tau += T;
            continue;
          }
          // tile i goes to S_x, P_x and O_x: x = h, or in a narrow piece the
          // tile's parity; the S of a tile is issued `ahead` tiles before its P V
          const int ahead = narrow ? 2 : 1;
          const int m = narrow ? 0 : h;
          for (int i = 0; i < min(ahead, T) && ok; ++i) {
            ok = k_wait(tau + i);
            if (!ok) break;
            tc_fence_after();
            issue_s(narrow ? i : h, m, tau + i);
            mma_commit(&kempty[(tau + i) % kStages]);
          }
          if (ok && T <= ahead) mma_commit(q_empty);
          for (int i = 0; i < T && ok; ++i) {
            const int t = tau + i, x = narrow ? i & 1 : h;
            const bool next = i + ahead < T;
            const int ph = ((x ? tiles1 : tiles0) + (narrow ? i >> 1 : i)) & 1;
            // everything but the second half of P before the turn
            ok = v_wait(t) && (!next || k_wait(t + ahead)) && mbar_wait(&p_a[x], ph, abort_flag) &&
                 (narrow || turn_wait());
            if (!ok) break;
            tc_fence_after();
            issue_pv(x, t, 0, i >= ahead);
            ok = mbar_wait(&p_b[x], ph, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_pv(x, t, 1, true);
            if (next) issue_s(x, m, t + ahead);
            if (!narrow) turn_pass();
            mma_commit(&vdone[t % kVSlots]);
            if (next) mma_commit(&kempty[(t + ahead) % kStages]);
            if (i + 1 + ahead == T) mma_commit(q_empty);
          }
          if (!ok) break;
          mma_commit(&o_done[h]);
          if (narrow) mma_commit(&o_done[1]);
          hand_over(p, narrow);
          count(T, narrow);
          tau += T;
        }
        if (!ok) {
          record_status(a.status, pieces[0].b, kDeviceTimeout);
          misc->abort = 1;
        }
        // every MMA issued so far completes before the next round or the exit
        mma_commit(&drain[h]);
        mbar_wait(&drain[h], round & 1);
      }
      __syncwarp();
      });
      if (warp == kMmaWarp) tmem_dealloc(tmem, Ly::kTmemCols);
    } else {
      rounds(nothing, [&](int, int npieces) {
      // ------------------------------------------------------ V conversion (E4M3)
      // Per tile: each key's row as the fp32 product code x V scale, rounded once
      // to fp16 (the value that the tree attention takes too), into converted slot
      // t % 2, in the MN-major layout the P V MMA reads.  Keys that no row of the
      // unit sees get zero rows (their codes may be stale).
      if (F8 && warp >= kConvWarp) {
        const int ct = tid - kConvWarp * 32;  // 0 .. 127
        const float* scl = reinterpret_cast<const float*>(smem + Ly::kVScl);
        bool ok = true;
        int tau = g_tile;
        for (int p = 0; p < npieces; ++p) {
          const Piece& pc = pieces[p];
          const Extent ext = extent_of(a, pc.pos0);
          const int hi = pc.hi();
          for (int t = pc.t0; t < pc.t1; ++t, ++tau) {
            const int vs = tau % kVStages;
            if (ok) ok = mbar_wait(&vfull[vs], (tau / kVStages) & 1, abort_flag);
            if (ok && tau >= 2) ok = mbar_wait(&v16empty[tau & 1], ((tau - 2) >> 1) & 1, abort_flag);
            if (!ok) {
              misc->abort = 1;
            } else {
              // thread ct: key ct of the tile.  Raw: 128 bytes a key, 16-byte
              // chunk c at chunk c ^ (key % 8); fp16: [8-key group][64-column
              // half][key][128 B], 16-byte chunk q of a line at q ^ (key % 8):
              // eight neighbouring lanes touch all banks once on either side.
              const int key = ext.key_tile(t) * BN + ct;
              const bool seen = key <= hi && (key < a.sinks || key >= ext.lo);
              const float s = seen ? scl[vs * BN + ct] : 0.0f;
              const float2 s2 = make_float2(s, s);
              const uint8_t* raw = smem + Ly::kVRing + vs * Ly::kKTileBytes + ct * 128;
              uint8_t* v16 = smem + Ly::kV16 + (tau & 1) * Ly::kTileBytes + (ct >> 3) * Ly::kGroupBytes + (ct & 7) * 128;
              const int sw = (ct & 7) << 4;
              // rolled: unrolled by 4 four 32768-token decodes take 9 us more (the
              // kernel's loops share one instruction cache)
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t h[8];
                const uint4 w = *reinterpret_cast<const uint4*>(raw + ((c << 4) ^ sw));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t c01, c23;
                  e4m3x4_to_f16x2x2(seen ? ww[k] : 0u, c01, c23);  // exact
                  const float2 v01 = mul2(unpack_f16x2(c01), s2), v23 = mul2(unpack_f16x2(c23), s2);
                  h[2 * k] = pack_f16x2(v01.x, v01.y);
                  h[2 * k + 1] = pack_f16x2(v23.x, v23.y);
                }
                uint8_t* line = v16 + (c >> 2) * 1024;
                *reinterpret_cast<uint4*>(line + ((((2 * c) & 7) << 4) ^ sw)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(line + ((((2 * c + 1) & 7) << 4) ^ sw)) = make_uint4(h[4], h[5], h[6], h[7]);
              }
              fence_proxy_async_smem();  // generic writes, read by the MMA
            }
            mbar_arrive(&v16full[tau & 1]);
            mbar_arrive(&vempty[vs]);
          }
        }
        if (!ok) record_status(a.status, pieces[0].b, kDeviceTimeout);
      }
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shares<F8>::kSoftmaxRegs));
    Line line;
    rounds([&](int round) { build_schedule<D, F8>(a, smem, round, tid, &line); }, [&](int, int npieces) {
      // ------------------------------------------------------ softmax groups
      // Warps 4h .. 4h+3 own m-tile h; warp w's rows are its TMEM lane
      // quarter 32 (w % 4) .. +31.
      const int h = warp >> 2;
      const int r = (warp & 3) * 32 + lane;  // row of the m-tile == TMEM lane
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tmem_s = tmem + h * BN + lane_off;
      const uint32_t tmem_o = tmem + 256 + h * D + lane_off;
      bool ok = true;
      int tau = g_tile;  // global index of the piece's first tile
      for (int p = 0; p < npieces; ++p) {
        const Piece& pc = pieces[p];
        const int T = pc.t1 - pc.t0;
        const int rows = pc.ntok * g;
        // a narrow piece has one m-tile: group h takes every second key tile of
        // its rows, from tile h on, and group 0 joins the two results
        const bool narrow = rows <= BM;
        const int ur = narrow ? r : h * BM + r;    // row of the unit
        const bool live = ur < rows;
        // a warp without live rows only keeps the barriers turning (what its
        // rows of P and O hold is not used): a decode token fills one warp
        const bool idle = ur - lane >= rows;
        const int tok = live ? ur / g : 0;
        const int pos = pc.pos0 + tok;             // position of this row
        const size_t q_row = static_cast<size_t>(pc.tok0 + tok);
        const int head = pc.kvh * g + (live ? ur - tok * g : 0);
        // E4M3: the row's scale is folded into the exponent factor (kept above
        // 0, so that a masked -inf never meets a factor of 0; NaN stays)
        float cq = a.scale_log2;
        if constexpr (F8) {
          if (live) cq = a.scale_log2 * __ldg(a.q_scale + q_row * a.hq + head);
          if (cq < 1e-37f) cq = 1e-37f;
        }

        float m_run = -INFINITY;  // what P is taken against: a running max (log2 units; kRaiseLog2 below it)
        float l_run = 0.0f;       // row sum against m_run
        const Extent ext = extent_of(a, pc.pos0);
        const int t0 = pc.t0, lo = ext.lo, hi = pc.hi(), pos0 = pc.pos0;
        const int first = narrow ? h : 0, every = narrow ? 2 : 1;
        for (int i = first; i < T; i += every) {
          const int k0 = ext.key_tile(t0 + i) * BN;  // first key of the tile
          const int gt = tau + i;                    // global tile (ring slot)
          // some row of the unit does not see some key of the tile
          const bool masked = k0 + BN - 1 > pos0 || (a.window > 0 && hi - a.window >= k0 && k0 + BN > a.sinks);
          if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[h], my_tiles & 1, abort_flag));
            if constexpr (F8) {  // the keys' K scales (landed with the K tile)
              ok = ok && __all_sync(0xffffffffu, mbar_wait(&sfull[gt % kSclSlots], (gt / kSclSlots) & 1, abort_flag));
            }
            if (!ok) misc->abort = 1;
          }
          ++my_tiles;
          // keys that no row of the unit sees: their V rows are cleared
          // (stale data; P is 0 there but 0 * NaN would poison O), a row per
          // thread, by each group before its own P_h(t) V(t).  (After S: only
          // then is every earlier use of the slot known to be over, and the
          // parity waited for unambiguous.)
          if constexpr (!F8) {
            if (ok && (k0 + BN - 1 > hi || (lo > k0 && k0 + BN > a.sinks))) {
              const int vs = gt % kVStages;
              mbar_wait(&vfull[vs], (gt / kVStages) & 1, abort_flag);  // acquire the TMA writes
              const int key = k0 + r;
              if (!(key <= hi && (key < a.sinks || key >= lo))) {
                // (eight neighbouring rows, eight chunks: every bank once)
                uint8_t* row = smem + Ly::kVRing + vs * Ly::kTileBytes + (r >> 3) * Ly::kGroupBytes + (r & 7) * 128;
#pragma unroll
                for (int k = 0; k < 8 * Ly::kHalves; ++k)
                  *reinterpret_cast<uint4*>(row + (k >> 3) * 1024 + ((k ^ r) & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();  // generic writes, read by the MMA
            }
          }
          if (!ok || idle) {
            mbar_arrive(&p_a[h]);
            mbar_arrive(&p_b[h]);
            continue;
          }
          // the scores stay unscaled; the softmax scale is folded into the exponent
          float x[128];
          float mx[4];
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tmem_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait32(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
            float* y = x + 32 * c;
            if constexpr (F8) {
              const float* sk = reinterpret_cast<const float*>(smem + Ly::kScl) + (gt % kSclSlots) * BN + 32 * c;
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 s4 = *reinterpret_cast<const float4*>(sk + k);
                const float2 a2 = mul2(make_float2(y[k], y[k + 1]), make_float2(s4.x, s4.y));
                const float2 b2 = mul2(make_float2(y[k + 2], y[k + 3]), make_float2(s4.z, s4.w));
                y[k] = a2.x;
                y[k + 1] = a2.y;
                y[k + 2] = b2.x;
                y[k + 3] = b2.y;
              }
            }
            if (masked) {
              const int kc = k0 + 32 * c;
              uint32_t bits = bits_below(pos + 1 - kc);
              if (a.window > 0) bits &= ~bits_below(pos + 1 - a.window - kc) | bits_below(a.sinks - kc);
              // (the rows of a warp are a few tokens: most of its words are whole)
              if (__any_sync(0xffffffffu, bits != 0xffffffffu)) {
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = (bits & (1u << k)) ? y[k] : -INFINITY;
              }
            }
            float u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u[j] = fmax3(y[j], y[j + 4], y[j + 8]);
              u[j] = fmax3(u[j], y[j + 12], y[j + 16]);
              u[j] = fmax3(u[j], y[j + 20], y[j + 24]);
              u[j] = fmaxf(u[j], y[j + 28]);
            }
            mx[c] = fmax3(u[0], u[1], fmaxf(u[2], u[3]));
          }
          const float smax = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * cq;
          constexpr float kRaise = F8 ? kRaiseLog2 : 0.0f;
          const bool up = live && smax > m_run + (kRescaleLog2 + kRaise);  // (the first visible score too)
          if (__any_sync(0xffffffffu, up)) {
            const float m_new = smax - kRaise;
            const float alpha = up ? exp2f(m_run - m_new) : 1.0f;
            if (up) m_run = m_new;
            // O holds P(..t-1) V against the old max; P_h(t-1) V is complete
            // (S_h(t), which this thread has seen complete, was issued after it)
            // (the piece's first P V overwrites O)
#pragma unroll 1
            for (int c0 = 0; i > first && c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(tmem_o + c0, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st16(tmem_o + c0, o);
            }
            l_run *= alpha;  // (this tile's sum is added below, against the new max)
          }
          // P = 2^(s * scale * log2(e) - m) as 16-bit pairs (column c holds
          // keys 2c, 2c+1), written over S_h; masked scores are -inf -> 0
          const float mref = m_run == -INFINITY ? 0.0f : m_run;
          const float2 sc2 = make_float2(cq, cq);
          const float2 nm2 = make_float2(-mref, -mref);
          uint32_t pk[4][16];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 e = fma2(make_float2(x[32 * q4 + 2 * k], x[32 * q4 + 2 * k + 1]), sc2, nm2);
              const float e0 = ex2_approx(e.x), e1 = ex2_approx(e.y);
              pk[q4][k] = F8 ? pack_f16x2_sat(e0, e1) : pack_bf16x2(e0, e1);
            }
            tmem_st16(tmem_s + 16 * q4, pk[q4]);
            if (q4 == 1 || q4 == 3) {
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(q4 == 1 ? &p_a[h] : &p_b[h]);
            }
          }
          // the row sum of the rounded values, under the MMAs
          float2 lacc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              if constexpr (F8) {
                acc_f16x2(pk[q4][k], lacc[k & 1]);
              } else {
                acc_bf16x2(pk[q4][k], lacc[k & 1]);
              }
            }
          l_run += (lacc[0].x + lacc[1].x) + (lacc[0].y + lacc[1].y);
        }
        // -------------------------------------------------- piece epilogue
        bool done = false;
        if (ok) {
          done = mbar_wait(&o_done[h], (g_piece + p) & 1, abort_flag);
          if (narrow && h == 0) done = done && mbar_wait(&o_done[1], (g_piece + p) & 1, abort_flag);
          done = __all_sync(0xffffffffu, done);
          if (!done) {
            ok = false;
            misc->abort = 1;
            record_status(a.status, pc.b, kDeviceTimeout);
          }
        }
        tc_fence_after();
        OwnO<D> own_o = {tmem_o, false, 1.0f, 0.0f};
        if (narrow) {
          // join: weights against the larger maximum, as in a merge
          float2* xch = reinterpret_cast<float2*>(smem + Ly::kXch);
          if (h == 1) xch[r] = make_float2(m_run, l_run);
          named_sync(kBarPair, kSoftmaxThreads);
          if (h == 0 && T > 1) {
            const float2 other = xch[r];
            const float M = fmaxf(m_run, other.x);
            own_o.two = true;
            own_o.w0 = m_run == -INFINITY ? 0.0f : exp2f(m_run - M);
            own_o.w1 = other.x == -INFINITY ? 0.0f : exp2f(other.x - M);
            l_run = own_o.w0 * l_run + own_o.w1 * other.y;
            m_run = M;
          }
        }
        if (narrow && h == 1) {
          // (group 0 writes)
        } else if (pc.npieces() == 1) {
          // the whole unit: normalise and write
          // (rolled, as everything that runs once a piece: see merge_rows)
          const float inv_l = l_run > 0.0f ? 1.0f / l_run : 0.0f;
          if (done) {
            const QuadRows quad = quad_rows<D>(a, q_row * a.hq + head, live);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float v[32];
              own_o.load(c0, v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= inv_l;
              store_rows32(a, quad, c0, v);
            }
          }
        } else {
          // a piece of a split unit.  With a thread per row, a piece that
          // finds every other one done merges straight from TMEM.  Otherwise
          // raw O and (m, l) go to its slot and it takes a ticket; the last to
          // take one merges.
          const int nthr = narrow ? BM : kSoftmaxThreads;
          const int bar = narrow ? kBarGroup0 : kBarPair;
          const int step = nthr / rows;
          const int flag = done ? 0 : 1;
          int* ticket = a.counters + pc.vfirst();
          if (ur == 0) misc->merge = step == 1 && *static_cast<volatile int*>(ticket) == pc.npieces() - 1;
          named_sync(bar, nthr);
          bool merge = misc->merge;
          if (!merge) {
            uint8_t* slot = a.slots + static_cast<size_t>(pc.slot()) * Sl::kBytes;
            float4* so4 = reinterpret_cast<float4*>(slot + Sl::kO) + ur;
            if (done) {  // (otherwise the flag voids the slot)
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                float v[32];
                own_o.load(c0, v);
                if (live) {
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    __stcg(so4 + (c0 / 4 + k) * rows, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
                }
              }
            }
            if (live) __stcg(reinterpret_cast<float2*>(slot + Sl::kMl) + ur, make_float2(m_run, l_run));
            if (ur == 0) __stcg(reinterpret_cast<int*>(slot + Sl::kFlag), flag);
            __threadfence();
            named_sync(bar, nthr);
            if (ur == 0) misc->merge = atomicAdd(ticket, 1) == pc.npieces() - 1;
            named_sync(bar, nthr);
            merge = misc->merge;
          }
          if (merge) {
            __threadfence();
            if (step == 1) {
              merge_rows<D, F8 ? 32 : 64>(a, pc, ur, static_cast<int>(blockIdx.x) - pc.vfirst(), m_run, l_run, flag, own_o);
            } else {
              merge_groups<D>(a, pc, ur, step);
            }
          }
          named_sync(bar, nthr);  // misc->merge is rewritten by the next split piece
        }
        if (narrow) named_sync(kBarPair, kSoftmaxThreads);  // O_1 and the exchange area are read
        tc_fence_before();
        tau += T;
      }
    });
  }
}

template <int D, bool F8>
int launch(const ChunkArgs& a, const ChunkMaps& maps, cudaStream_t stream) {
  static thread_local int attr_set_device = -1;  // the attribute is set once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (attr_set_device != dev) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<D, F8>::kAlloc) != cudaSuccess)
      return -1;
    attr_set_device = dev;
  }
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.vctas, 1, 1);
  cfg.blockDim = dim3(Shares<F8>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<D, F8>::kAlloc;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_attn_kernel<D, F8>, a, maps) == cudaSuccess ? 0 : -1;
}

}  // namespace

size_t chunk_slot_bytes(int head_dim) {
  return head_dim == 64 ? Slot<64>::kBytes : Slot<128>::kBytes;
}

int launch_chunk_attention(const ChunkArgs& a, const ChunkMaps& maps, int sms, cudaStream_t stream) {
  chunk_check_kernel<<<a.batch < sms ? a.batch : sms, kCheckThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return -1;
  if (a.total_tokens == 0) return 0;
  if (a.fp8) return launch<128, true>(a, maps, stream);
  return a.head_dim == 128 ? launch<128, false>(a, maps, stream) : launch<64, false>(a, maps, stream);
}

}  // namespace tv
