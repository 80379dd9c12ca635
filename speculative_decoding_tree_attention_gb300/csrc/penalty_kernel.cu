// penalty_kernel.cu -- penalties for repeated tokens, biases and grammar masks
// on the target logits of tree nodes, ahead of the accept pass.
//
// Row i of tree b predicts the token after node i, so what its tokens are
// counted against is the sequence's history and the drafted tokens on the path
// root .. i (the root's own token is the last committed one: history).  With
// c(v) = occurrences of v among the generated tokens (history from the prompt's
// end on, and the path) and seen(v) = c(v) > 0 or v in the prompt:
//   x = logit
//   seen:      x = x > 0 ? x / r : x * r      repetition penalty r
//   x = x - freq c                            frequency penalty
//   c > 0:     x = x - pres                   presence penalty
//   x = x + bias(v)
//   mask bit 0: x = -inf
// each step one fp32 rounding.
//
// One CTA takes a chunk of 2048 vocabulary entries of the rows of one tree (or
// of a share of them).  It counts the sequence's history and bias list into
// shared memory once and lists the touched entries, ascending.  Each warp then
// streams rows through, one read and one write of HBM per entry: a masked copy
// that also passes through shared memory, 512 entries at a time, from where the
// touched ones are rewritten, a lane each.  The few tokens of the row's path,
// which have a count of their own, come last.  With the penalties inside the
// stream every warp step met some touched entry and ran their divisions for 16
// of 32 lanes (82 us, the first case below); gathering the touched entries again
// from L2 took longer than the copy (48 us).
//
// Bound: HBM; per entry 4 (fp32) or 2 (bf16) bytes read, 4 written, a mask bit.
// 16 trees of 26 or 64 nodes, V = 32000, bf16, histories of 512 to 4096: 37 us
// (3.9 TB/s: each tree's history is counted by all of its 16 chunks' CTAs).
// 4 trees of 128 nodes, V = 151936, fp32, histories of 1600: 106 us (5.9 TB/s).
// (Device time, the call replayed; with a cold L2 40 and 108 us.)
#include <math.h>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 2048;
constexpr int kBlock = 512;     // entries that pass through shared memory at a time
constexpr int kMaxNodes = 512;
constexpr uint32_t kPrompt = 0x80000000u;  // count word: in the prompt; low 31 bits: generated

struct Shared {
  uint32_t count[kChunk];
  union {
    int entry[kChunk];   // last bias entry of a token
    float bias[kChunk];
  };
  uint32_t path[kWarps][kChunk / 32];  // a warp's row: tokens of its path
  float block[kWarps][kBlock];         // a warp's row: entries on their way
  uint16_t touched[kChunk];            // entries with a count or a bias, ascending
  uint32_t mark[kChunk / 32];          // a bit for each of them
  int before[kChunk / 32 + 1];         // marks in earlier words
  int token[kMaxNodes];
  int16_t parent[kMaxNodes];
  int bad;
  int decrease;                        // the first tree with fewer than 0 nodes (this one: none before it)
};
static_assert(sizeof(Shared) <= 45 * 1024, "no opt-in, and no fewer CTAs an SM than the registers allow");

struct Rates {
  float rep, pres, freq;
};

__device__ __forceinline__ float apply(float x, uint32_t word, uint32_t more, float bias, const Rates& r) {
  const uint32_t c = (word & ~kPrompt) + more;
  if (c > 0 || word) x = x > 0.0f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (c > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.freq, static_cast<float>(c))), r.pres);
  return __fadd_rn(x, bias);
}

// one logit of a row (with plain loads: the rows may be rewritten in place)
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int v) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[v]) << 16)
              : static_cast<const float*>(row)[v];
}
// four of them, as loaded
template <bool BF16>
struct Raw4 {
  uint2 w;
  __device__ __forceinline__ void load(const void* row, int v) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + v);
  }
  __device__ __forceinline__ float4 value() const {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
};
template <>
struct Raw4<false> {
  float4 w;
  __device__ __forceinline__ void load(const void* row, int v) {
    w = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + v);
  }
  __device__ __forceinline__ float4 value() const { return w; }
};

// BF16: the logits' type (else fp32).  VEC: rows are 4-entry aligned.  Three CTAs
// an SM (single bf16 entries: two): left to itself the compiler took 64 registers
// and spilled, the second case above 114 us instead of 107.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, BF16 && !VEC ? 2 : 3) penalty_kernel(const PenaltyArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  const int c0 = blockIdx.x * kChunk, b = blockIdx.y;
  const int nv = min(kChunk, a.vocab - c0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the tree's rows, of a malformed one those that are there
  const int from = __ldg(a.node_offsets + b), to = __ldg(a.node_offsets + b + 1);
  const int n0 = max(from, 0), N = max(min(to, a.total_nodes), n0) - n0;
  int h0 = 0, h1 = 0;
  if (a.history_offsets) {  // (of an empty list too)
    h0 = __ldg(a.history_offsets + b);
    h1 = __ldg(a.history_offsets + b + 1);
  }
  int e0 = 0, e1 = 0;
  if (a.bias_offsets) {
    e0 = __ldg(a.bias_offsets + b);
    e1 = __ldg(a.bias_offsets + b + 1);
  }
  Rates r;
  r.rep = a.repetition ? __ldg(a.repetition + b) : 1.0f;
  r.pres = a.presence ? __ldg(a.presence + b) : 0.0f;
  r.freq = a.frequency ? __ldg(a.frequency + b) : 0.0f;
  if (tid == 0) {
    s.bad = 0;
    s.decrease = b;
  }
  bool bad = from < 0 || to <= from || to > a.total_nodes || N > a.max_nodes || h0 < 0 || h1 < h0 ||
             h1 > a.total_history || e0 < 0 || e1 < e0 || e1 > a.total_bias || !(r.rep > 0.0f && r.rep < INFINITY) ||
             !(fabsf(r.pres) < INFINITY) || !(fabsf(r.freq) < INFINITY);
  const uint4 zero = make_uint4(0, 0, 0, 0), none = make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll
  for (int i = 4 * tid; i < kChunk; i += 4 * kThreads) {
    *reinterpret_cast<uint4*>(&s.count[i]) = zero;
    if (a.bias_ids) *reinterpret_cast<uint4*>(&s.entry[i]) = none;
  }
  if (tid < kWarps * (kChunk / 32) / 4) *reinterpret_cast<uint4*>(&s.path[0][0] + 4 * tid) = zero;
  __syncthreads();
  // trees behind a decreasing offset may have rows of the trees before it: they
  // are malformed.  (16 and 4 trees: no time; 4096 trees of one node, V = 32000:
  // 772 -> 829 us; the loads of 8 steps in flight, 4 offsets a load took as long)
  bool dec = false;
#pragma unroll 8
  for (int i = tid; i < b; i += kThreads) dec |= __ldg(a.node_offsets + i + 1) < __ldg(a.node_offsets + i);
  if (dec) {
    for (int i = tid; i < b; i += kThreads)
      if (__ldg(a.node_offsets + i + 1) < __ldg(a.node_offsets + i)) atomicMin(&s.decrease, i);
  }
  if (!bad) {
    for (int i = tid; i < N; i += kThreads) {
      const int p = __ldg(a.parent + n0 + i);
      s.parent[i] = static_cast<int16_t>(p);
      s.token[i] = __ldg(a.tokens + n0 + i);
      if (i == 0 ? p != -1 : (p < 0 || p >= i)) s.bad = 1;
    }
    // history: ids outside the chunk (and outside the vocabulary) do not count
    const int prompt = a.prompt_lens ? max(0, __ldg(a.prompt_lens + b)) : 0;
    constexpr int kH = 16;  // entries in flight
    for (int i0 = h0 + tid; i0 < h1; i0 += kThreads * kH) {
      int v[kH];
#pragma unroll
      for (int k = 0; k < kH; ++k) v[k] = i0 + k * kThreads < h1 ? __ldg(a.history + i0 + k * kThreads) - c0 : -1;
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        if (v[k] < 0 || v[k] >= nv) continue;
        if (i0 + k * kThreads - h0 < prompt) {
          atomicOr(&s.count[v[k]], kPrompt);
        } else {
          atomicAdd(&s.count[v[k]], 1u);
        }
      }
    }
    for (int i = e0 + tid; i < e1; i += kThreads) {
      const int v = __ldg(a.bias_ids + i) - c0;
      if (v >= 0 && v < nv) atomicMax(&s.entry[v], i);
    }
  }
  __syncthreads();
  bad = bad || s.bad || s.decrease < b;
  if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) a.status[b] = bad ? kBadTree : kOk;
  if (N == 0) return;
  const bool has_bias = a.bias_ids != nullptr;
  if (!bad) {
    // the marks, their prefix counts, and the list
    constexpr int kWords = kChunk / 32 / kWarps;  // per warp
    int v = (warp * kWords) * 32 + lane;
#pragma unroll
    for (int k = 0; k < kWords; ++k, v += 32) {
      const int e = has_bias ? s.entry[v] : -1;
      if (has_bias) s.bias[v] = e >= 0 ? __ldg(a.bias_values + e) : 0.0f;
      const uint32_t m = __ballot_sync(0xffffffffu, s.count[v] != 0u || e >= 0);
      if (lane == 0) s.mark[warp * kWords + k] = m;
    }
    __syncthreads();
    if (warp == 0) {
      int n = 0;
#pragma unroll
      for (int k = 0; k < kChunk / 1024; ++k) {
        const int c = __popc(s.mark[32 * k + lane]);
        int x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        s.before[32 * k + lane] = n + x - c;
        n += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) s.before[kChunk / 32] = n;
    }
    __syncthreads();
    v = (warp * kWords) * 32 + lane;
#pragma unroll
    for (int k = 0; k < kWords; ++k, v += 32) {
      const uint32_t m = s.mark[v >> 5];
      if (m >> lane & 1u) s.touched[s.before[v >> 5] + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(v);
    }
    __syncthreads();
  }
  const bool any_touched = !bad && s.before[kChunk / 32] > 0;  // (bad: the rows as given)
  const uint32_t* mask = bad ? nullptr : a.allowed_mask;
  const int words = (a.vocab + 31) / 32;
  uint32_t* path = s.path[warp];
  float* block = s.block[warp];
  // (behind a decrease: only rows that no sound tree has)
  int row0 = blockIdx.z * kWarps + warp;
  if (s.decrease < b) {
    const int skip = min(max(__ldg(a.node_offsets + s.decrease), n0) - n0, N), step = gridDim.z * kWarps;
    if (skip > row0) row0 += (skip - row0 + step - 1) / step * step;
  }
  for (int i = row0; i < N; i += gridDim.z * kWarps) {
    const size_t row = static_cast<size_t>(n0 + i);
    const void* in = static_cast<const uint8_t*>(a.logits) + row * a.vocab * (BF16 ? 2 : 4);
    float* out = a.out + row * a.vocab;
    const uint32_t* mrow = mask ? mask + row * words : nullptr;
    // the next entries of the row, in flight as loaded, a mask word a lane.  (fp32
    // with 1024 of them: 100 registers a thread, 112 us for the second case)
    constexpr int kStep = BF16 ? 1024 : 512;
    constexpr int kLoads = kStep / (VEC ? 128 : 32);
    Raw4<BF16> x[VEC ? kLoads : 1];
    float z[VEC ? 1 : kLoads];
    uint32_t mw = ~0u;
    auto fetch = [&](int b0) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int v = b0 + (VEC ? 128 * u + 4 * lane : 32 * u + lane);
        if (v >= nv) continue;
        if constexpr (VEC) {
          x[u].load(in, c0 + v);
        } else {
          z[u] = load_logit<BF16>(in, c0 + v);
        }
      }
      if (mrow && lane < kStep / 32 && b0 + 32 * lane < nv) mw = __ldg(mrow + ((c0 + b0) >> 5) + lane);
    };
    fetch(0);
    // marks the drafted tokens of the path in this chunk: lane k looks at every
    // 32nd ancestor from the node up
    bool any = false;
    if (!bad) {
      int j = i;
      for (int k = 0; k < lane && j > 0; ++k) j = s.parent[j];
      while (__any_sync(0xffffffffu, j > 0)) {
        const int v = j > 0 ? s.token[j] - c0 : -1;
        const bool mine = v >= 0 && v < nv;
        if (mine) atomicOr(&path[v >> 5], 1u << (v & 31));
        any |= __any_sync(0xffffffffu, mine);
        for (int k = 0; k < 32 && j > 0; ++k) j = s.parent[j];
      }
      __syncwarp();
    }
    // the masked copy, and the touched entries that are not on the path
#pragma unroll 1
    for (int b0 = 0; b0 < nv; b0 += kStep) {
      const uint32_t word = mw;
      float4 y[VEC ? kLoads : 1];
      float w[VEC ? 1 : kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        if constexpr (VEC) {
          y[u] = x[u].value();
        } else {
          w[u] = z[u];
        }
      }
      fetch(b0 + kStep);
#pragma unroll
      for (int half = 0; half < kStep / kBlock; ++half) {
        const int h0 = b0 + kBlock * half;
        if (h0 >= nv) break;
#pragma unroll
        for (int q = 0; q < (VEC ? 4 : 16); ++q) {
          if constexpr (VEC) {
            const int u = 4 * half + q, v = b0 + 128 * u + 4 * lane;
            const uint32_t ok = __shfl_sync(0xffffffffu, word, 4 * u + (lane >> 3)) >> (v & 31);
            const float4 t = make_float4(ok & 1u ? y[u].x : -INFINITY, ok & 2u ? y[u].y : -INFINITY,
                                         ok & 4u ? y[u].z : -INFINITY, ok & 8u ? y[u].w : -INFINITY);
            if (v < nv) *reinterpret_cast<float4*>(out + c0 + v) = t;
            if (any_touched) *reinterpret_cast<float4*>(block + 128 * q + 4 * lane) = t;
          } else {
            const int u = 16 * half + q, v = b0 + 32 * u + lane;
            const float t = __shfl_sync(0xffffffffu, word, u) >> lane & 1u ? w[u] : -INFINITY;
            if (v < nv) out[c0 + v] = t;
            if (any_touched) block[32 * q + lane] = t;
          }
        }
        if (!any_touched) continue;
        __syncwarp();
        const int k1 = s.before[(h0 + kBlock) >> 5];
        for (int k = s.before[h0 >> 5] + lane; k < k1; k += 32) {
          const int v = s.touched[k];
          const float t = block[v - h0];
          if (t != -INFINITY && !(any && (path[v >> 5] >> (v & 31) & 1u)))
            out[c0 + v] = apply(t, s.count[v], 0, has_bias ? s.bias[v] : 0.0f, r);
        }
        __syncwarp();
      }
    }
    if (!any) continue;
    // the path's tokens: the node nearest to the row computes a token.  An
    // allowed one still holds its logit in place, a masked one stays -inf.
    __syncwarp();  // other lanes stored the copies that are rewritten (and, in place, read) here
    int j = i;
    for (int k = 0; k < lane && j > 0; ++k) j = s.parent[j];
    while (__any_sync(0xffffffffu, j > 0)) {
      const int v = j > 0 ? s.token[j] - c0 : -1;
      if (v >= 0 && v < nv) {
        uint32_t more = 0;
        for (int m = i; m > 0; m = s.parent[m]) {
          if (s.token[m] != v + c0) continue;
          if (more == 0 && m != j) break;
          ++more;
        }
        if (more > 0 && (!mrow || (__ldg(mrow + ((c0 + v) >> 5)) >> (v & 31) & 1u))) {
          const float t = load_logit<BF16>(in, c0 + v);
          if (t != -INFINITY) out[c0 + v] = apply(t, s.count[v], more, has_bias ? s.bias[v] : 0.0f, r);
        }
      }
      for (int k = 0; k < 32 && j > 0; ++k) j = s.parent[j];
    }
    __syncwarp();
    for (int k = lane; k < kChunk / 32; k += 32) path[k] = 0u;
    __syncwarp();
  }
}

}  // namespace

int launch_penalty(const PenaltyArgs& a, int sms, cudaStream_t stream) {
  const int chunks = (a.vocab + kChunk - 1) / kChunk;
  // shares of a tree's rows: 5 CTAs an SM, two or three of them at a time (2
  // an SM: 44 and 121 us, 8: 37 and 110), at least a row per warp
  const long long base = static_cast<long long>(chunks) * a.batch;
  const int most = (a.max_nodes + kWarps - 1) / kWarps;
  long long shares = (5ll * sms + base - 1) / base;
  shares = shares < 1 ? 1 : (shares > most ? most : shares);
  const dim3 grid(chunks, a.batch, static_cast<unsigned>(shares));
  const bool vec = a.vocab % 4 == 0;  // (row starts are then 16-byte aligned, bf16 rows 8-byte)
  auto* k = a.bf16 ? (vec ? penalty_kernel<true, true> : penalty_kernel<true, false>)
                   : (vec ? penalty_kernel<false, true> : penalty_kernel<false, false>);
  k<<<grid, kThreads, sizeof(Shared), stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tv
