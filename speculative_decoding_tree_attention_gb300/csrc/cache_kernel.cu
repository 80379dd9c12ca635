// cache_kernel.cu -- writing new K/V rows into the paged cache (bf16, or
// quantised to E4M3 as they are written), reading an E4M3 cache back to bf16,
// and quantising plain rows.
//
// Quantisation of a row x of D values: s = fl32(max |x_i| / 448) over the
// finite entries (at least 2^-126; 1 for a row of zeros), code_i = the E4M3
// value nearest to the real quotient x_i / s, ties to even, saturating at 448;
// NaN gives NaN.
//
// The quotient is rounded once without dividing each value.  The middle of two
// codes is c 2^j with c odd, c < 32, and with m = max |x_i|
//   448 x / m = c 2^j   <=>   7 X 2^k = c A   for the 8-bit integers X, A of x
// and m: either equal, or apart by 1 in c A < 2^13.  So a product q = x fl(1/s),
// within 2^-22 of the quotient, rounds as it does unless 448 x / m is a middle
// itself.  There x / s = (448 x / m) (m / (448 s)) lies on the side on which
// 448 s rounded off m, the same for the whole row: 1/s is moved by 2^-20 to that
// side.  Where s is exact (m a multiple of 7, or a clamped s) the middles have
// to be met exactly: the last 4 of q's 24 bits are rounded off, which takes a q
// within 2 ulp of a middle to it and no other across one.
//
// All of it is one read and one write of each row, bound by HBM for prompts and
// by latency for single tokens.  A row is taken by D / 8 lanes, 16 bytes of
// bf16 and 8 codes each; the rows of a CTA are ordered (K or V, head, token), so
// that neighbouring rows of a page are written together.
//
// Measured (8 KV heads, D = 128; device time, the call replayed): the K/V of 4 x
// 8192 tokens to E4M3 52 us (3.9 TB/s; the same bytes moved without the arithmetic
// 34 us; with a cold L2 56), of 16 tokens 4 us; 4 x 32768 tokens read back to bf16
// 149 us (5.5 TB/s), 1001 tokens 4 us.
#include <climits>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;   // tokens of a CTA: one per lane of the warp that finds their sequences
static_assert(kMaxTile == 32, "place_tokens: a lane per token");
constexpr int kNoPage = 7;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two values -> two E4M3 codes (nearest, ties to even, saturating; the first
// in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row's scale and the factor that takes a value to its code's quotient.
struct Scale {
  float s, inv;
  bool exact;  // 448 s is the row's largest magnitude (or s is the clamp)
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale r;
  r.s = amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-126f);
  r.inv = __fdiv_rn(1.0f, r.s);
  const float off = __fmaf_rn(-r.s, 448.0f, amax);  // (exact)
  r.exact = off == 0.0f || r.s == 0x1p-126f || amax == 0.0f;
  if (!r.exact) r.inv = __fmaf_rn(r.inv, off > 0.0f ? 0x1p-20f : -0x1p-20f, r.inv);
  return r;
}
// Both are the same for the 128 mantissas of a bf16 maximum but for powers of
// two: a table of them (s < 0: exact) saves every lane of every row two
// divisions.
struct Table {
  float2 of[128];
};
__device__ __forceinline__ void fill_table(Table& t) {
  if (threadIdx.x < 128) {
    const Scale r = scale_of(1.0f + threadIdx.x / 128.0f);
    t.of[threadIdx.x] = make_float2(r.exact ? -r.s : r.s, r.inv);
  }
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int LANES>
__device__ __forceinline__ uint32_t across(uint32_t m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m & 0xffffu, m >> 16);
}
// The scale of a row of which this lane holds 8 values (w) and the LANES lanes
// around it the rest.  Every lane of the warp takes part.
template <int LANES>
__device__ __forceinline__ Scale row_scale(const Table& t, const uint4& w) {
  const uint32_t v[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
  uint32_t m = across<LANES>(max_u16x2(max_u16x2(v[0], v[1]), max_u16x2(v[2], v[3])));
  if (__any_sync(0xffffffffu, m >= 0x7f80u)) {  // infinities or NaN: the finite ones
    uint32_t f = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = v[k] & 0xffffu, hi = v[k] >> 16;
      f = max(f, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
    m = across<LANES>(f);
  }
  const uint32_t e = m >> 7;  // biased exponent
  if (e < 16) return scale_of(__uint_as_float(m << 16));  // zero, subnormal, or a scale near the clamp
  const float2 at = t.of[m & 127u];
  Scale r;
  r.exact = at.x < 0.0f;
  r.s = __uint_as_float((__float_as_uint(at.x) & 0x7fffffffu) + ((e - 127u) << 23));
  r.inv = __uint_as_float(__float_as_uint(at.y) - ((e - 127u) << 23));
  return r;
}

__device__ __forceinline__ uint2 row_codes(const uint4& w, const Scale& r) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  float q[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    q[2 * k] = bf16_lo(v[k]) * r.inv;
    q[2 * k + 1] = bf16_hi(v[k]) * r.inv;
  }
  if (r.exact) {
#pragma unroll
    for (int k = 0; k < 8; ++k)  // (infinities and -0 stay)
      if (q[k] == q[k]) q[k] = __uint_as_float((__float_as_uint(q[k]) + 8u) & ~15u);
  }
  return make_uint2(e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16, e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16);
}

// Where each token of a CTA's tile goes.
struct Tile {
  int hist[kMaxTile + 1];     // sequences whose offset falls on a token
  int seq[kMaxTile];          // sequence of each token, -1: none or failed
  int slot[kMaxTile];         // its page and row: block * 16 + position % 16
  int code[kMaxTile];         // of the sequence that starts the run at this token
  int bad_offsets;
};

// Fills the tile's places: the sequence of each token (from a histogram of the
// offsets over the tile, one pass over the batch), the checks of that
// sequence's extent and of the pages of all its tokens (so that every CTA of a
// sequence decides alike), and the token's place.  The CTA of a sequence's
// first token writes its status; CTA 0 those of empty sequences.
__device__ void place_tokens(const CacheArgs& a, Tile& tl, int t0, int n) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i <= kMaxTile; i += kThreads) tl.hist[i] = 0;
  if (tid == 0) tl.bad_offsets = 0;
  __syncthreads();
  for (int i = tid; i < a.batch; i += kThreads) {
    const int o = __ldg(a.token_offsets + i), next = __ldg(a.token_offsets + i + 1);
    if (o < 0 || next < o || next > a.total_tokens) tl.bad_offsets = 1;
    if (o < t0 + n) atomicAdd(&tl.hist[max(o, t0) - t0], 1);  // (o - t0 of a malformed o may wrap)
  }
  __syncthreads();
  const bool bad = tl.bad_offsets != 0;
  if (warp == 0) {
    // sequence of token t0 + lane: offsets at or before it, less one
    int c = tl.hist[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    const int b = c - 1, t = t0 + lane;
    const bool in = lane < n && !bad && b >= 0 && t < __ldg(a.token_offsets + b + 1);
    tl.seq[lane] = in ? b : -1;
  }
  if (blockIdx.x == 0)
    for (int b = tid; b < a.batch; b += kThreads)
      if (bad || a.token_offsets[b + 1] == a.token_offsets[b]) a.status[b] = bad ? kBadTree : kOk;
  __syncthreads();
  // a warp per sequence of the tile (per run of tokens)
  for (int i = warp; i < n; i += kThreads / 32) {
    const int b = tl.seq[i];
    if (b < 0 || (i > 0 && tl.seq[i - 1] == b)) continue;
    const int n0 = __ldg(a.token_offsets + b), c = __ldg(a.token_offsets + b + 1) - n0;
    const int len = __ldg(a.seq_lens + b);
    const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_blocks_per_seq;
    int code = len < c ? kBadTree : kOk;
    if (code == kOk) {
      bool none = false;
      for (int p = (len - c) / 16 + lane; p <= (len - 1) / 16; p += 32) {
        const int blk = p < a.max_blocks_per_seq ? __ldg(table + p) : -1;
        none |= blk < 0 || blk >= a.num_blocks;
      }
      if (__any_sync(0xffffffffu, none)) code = kNoPage;
    }
    if (lane == 0) {
      tl.code[i] = code;
      if (n0 == t0 + i) a.status[b] = code;
    }
  }
  __syncthreads();
  if (tid < n) {
    const int b = tl.seq[tid];
    int place = -1;
    if (b >= 0) {
      int i = tid;  // the first token of its run
      while (i > 0 && tl.seq[i - 1] == b) --i;
      if (tl.code[i] == kOk) {
        const int n0 = __ldg(a.token_offsets + b), c = __ldg(a.token_offsets + b + 1) - n0;
        const int pos = __ldg(a.seq_lens + b) - c + (t0 + tid - n0);
        place = __ldg(a.block_table + static_cast<size_t>(b) * a.max_blocks_per_seq + pos / 16) * 16 + pos % 16;
      }
    }
    tl.slot[tid] = place;
  }
  __syncthreads();
}

enum Op { kCopy, kQuantise, kRead };

// OP kCopy, kQuantise: rows of k_new / v_new into the pool.  kRead: pool rows
// into k_new / v_new.
template <int D, Op OP>
__global__ void __launch_bounds__(kThreads) cache_kernel(const CacheArgs a) {
  constexpr int kLanes = D / 8;
  // rows in flight per lane group (of 1, 2, 4 and 8, reading 4 x 32768 tokens
  // took 166, 149, 159 and 153 us, writing 4 x 8192 was fastest at 2 as well)
  constexpr int kUnroll = 2;
  __shared__ Tile tl;
  __shared__ Table table;
  if (OP == kQuantise) fill_table(table);  // (place_tokens synchronises)
  const int tile = 1 << a.tile_shift;
  const int t0 = blockIdx.x << a.tile_shift;
  const int n = min(tile, a.total_tokens - t0);
  place_tokens(a, tl, t0, n);
  const int sub = threadIdx.x % kLanes;
  const int rows = 2 * a.hkv << a.tile_shift;  // (of a whole tile)
  constexpr int kStep = kThreads / kLanes;
  for (int r0 = threadIdx.x / kLanes; r0 - r0 % kStep < rows; r0 += kStep * kUnroll) {
    uint4 w[kUnroll];
    float s[kUnroll];
    uint8_t* dst[kUnroll];
    float* sdst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kStep;
      dst[u] = nullptr;
      w[u] = make_uint4(0, 0, 0, 0);
      const int tok = r & (tile - 1);
      if (r >= rows || tok >= n) continue;
      const int kv = (r >> a.tile_shift) >= a.hkv;
      const int head = (r >> a.tile_shift) - (kv ? a.hkv : 0);
      const int place = tl.slot[tok];
      uint8_t* row = static_cast<uint8_t*>(kv ? a.v_new : a.k_new) +
                     (static_cast<size_t>(t0 + tok) * a.kv_stride + static_cast<size_t>(head) * D) * 2 + sub * 16;
      if (OP == kRead && place < 0) {
        // a failed sequence reads as zeros; rows of no sequence stay
        if (tl.seq[tok] >= 0) *reinterpret_cast<uint4*>(row) = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (place < 0) continue;
      const size_t at = (static_cast<size_t>(place / 16) * a.hkv + head) * 16 + place % 16;
      uint8_t* pool = static_cast<uint8_t*>(kv ? a.v_pool : a.k_pool) + at * (OP == kCopy ? 2 * D : D) +
                      sub * (OP == kCopy ? 16 : 8);
      sdst[u] = (kv ? a.v_scale : a.k_scale) + at;
      if (OP == kRead) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2*>(pool));
        w[u] = make_uint4(c.x, c.y, 0, 0);
        s[u] = __ldg(sdst[u]);
        dst[u] = row;
      } else {
        w[u] = __ldcs(reinterpret_cast<const uint4*>(row));
        dst[u] = pool;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (OP == kCopy) {
        if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = w[u];
      } else if (OP == kQuantise) {
        const Scale sc = row_scale<kLanes>(table, w[u]);  // (every lane takes part)
        if (dst[u]) {
          *reinterpret_cast<uint2*>(dst[u]) = row_codes(w[u], sc);
          if (sub == 0) *sdst[u] = sc.s;
        }
      } else if (dst[u]) {
        // the fp32 product of code and scale, rounded to bf16
        uint32_t h[4], o[4];
        e4m3x4_to_f16x2x2(w[u].x, h[0], h[1]);
        e4m3x4_to_f16x2x2(w[u].y, h[2], h[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = unpack_f16x2(h[k]);
          o[k] = pack_bf16x2(c.x * s[u], c.y * s[u]);
        }
        *reinterpret_cast<uint4*>(dst[u]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) quantise_rows_kernel(const QuantArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kUnroll = 4;
  __shared__ Table table;
  fill_table(table);
  __syncthreads();
  const int sub = threadIdx.x % kLanes;
  const long long rows = static_cast<long long>(a.tokens) * a.heads;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads / kLanes);
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads / kLanes);
  for (long long b0 = first; b0 < rows; b0 += step * kUnroll) {  // (uniform over the CTA)
    const long long r0 = b0 + threadIdx.x / kLanes;
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long r = r0 + u * step;
      w[u] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        w[u] = __ldcs(reinterpret_cast<const uint4*>(a.x + (r / a.heads) * a.stride + (r % a.heads) * D) + sub);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long r = r0 + u * step;
      const Scale s = row_scale<kLanes>(table, w[u]);
      if (r >= rows) continue;
      reinterpret_cast<uint2*>(a.codes + r * D)[sub] = row_codes(w[u], s);
      if (sub == 0) a.scale[r] = s.s;
    }
  }
}

template <int D>
void launch_cache_d(const CacheArgs& a, int grid, cudaStream_t stream) {
  if (a.read) {
    cache_kernel<D, kRead><<<grid, kThreads, 0, stream>>>(a);
  } else if (a.k_scale) {
    cache_kernel<D, kQuantise><<<grid, kThreads, 0, stream>>>(a);
  } else {
    cache_kernel<D, kCopy><<<grid, kThreads, 0, stream>>>(a);
  }
}

}  // namespace

int launch_cache(CacheArgs a, int sms, cudaStream_t stream) {
  // tokens per CTA (a power of two): as many as keep about 8 CTAs per SM busy,
  // at most a tile; one token per CTA for a decode step
  a.tile_shift = 0;
  while (2 << a.tile_shift <= kMaxTile && (2ll << a.tile_shift) * 8 * sms <= a.total_tokens) ++a.tile_shift;
  const int tile = 1 << a.tile_shift;
  const int grid = a.total_tokens > 0 ? (a.total_tokens + tile - 1) / tile : 1;
  if (a.head_dim == 128) {
    launch_cache_d<128>(a, grid, stream);
  } else {
    launch_cache_d<64>(a, grid, stream);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_quantise_rows(const QuantArgs& a, int sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.tokens) * a.heads;
  const int per = kThreads / (a.head_dim / 8);
  const long long want = (rows + per - 1) / per, most = 16ll * sms;
  const int grid = static_cast<int>(want < most ? want : most);
  if (a.head_dim == 128) {
    quantise_rows_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  } else {
    quantise_rows_kernel<64><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tv
