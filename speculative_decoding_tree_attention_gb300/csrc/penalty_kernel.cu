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
// One CTA takes a chunk of 4096 vocabulary entries of the rows of one tree (or
// of a share of them): it counts the sequence's history and bias list into
// shared memory once, then each warp streams rows through it, one read and one
// write of HBM per entry.  Path tokens are few: a row that has any in the chunk
// gets them computed apart, from a bitmap that the stream skips.
#include <math.h>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 4096;
constexpr int kMaxNodes = 512;
constexpr uint32_t kPrompt = 0x80000000u;  // count word: in the prompt; low 31 bits: generated

struct Shared {
  uint32_t count[kChunk];
  union {
    int entry[kChunk];   // last bias entry of a token
    float bias[kChunk];
  };
  uint32_t path[kWarps][kChunk / 32];
  int parent[kMaxNodes];
  int token[kMaxNodes];
  int bad;
};

struct Rates {
  float rep, pres, freq;
};

__device__ __forceinline__ float apply(float x, uint32_t word, uint32_t more, float bias, bool allowed, const Rates& r) {
  const uint32_t c = (word & ~kPrompt) + more;
  if (c > 0 || word) x = x > 0.0f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (c > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.freq, static_cast<float>(c))), r.pres);
  x = __fadd_rn(x, bias);
  return allowed ? x : -INFINITY;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int v) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(__ldcs(static_cast<const uint16_t*>(row) + v)) << 16)
              : __ldcs(static_cast<const float*>(row) + v);
}
template <bool BF16>
__device__ __forceinline__ float4 load_logit4(const void* row, int v) {
  if (BF16) {
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + v));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  return __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(row) + v));
}

// BF16: the logits' type (else fp32).  VEC: rows are 4-entry aligned.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) penalty_kernel(const PenaltyArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  const int c0 = blockIdx.x * kChunk, b = blockIdx.y;
  const int nv = min(kChunk, a.vocab - c0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = __ldg(a.node_offsets + b);
  const long long nodes = static_cast<long long>(__ldg(a.node_offsets + b + 1)) - n0;
  int h0 = 0, h1 = 0;
  if (a.history) {
    h0 = __ldg(a.history_offsets + b);
    h1 = __ldg(a.history_offsets + b + 1);
  }
  int e0 = 0, e1 = 0;
  if (a.bias_ids) {
    e0 = __ldg(a.bias_offsets + b);
    e1 = __ldg(a.bias_offsets + b + 1);
  }
  Rates r;
  r.rep = a.repetition ? __ldg(a.repetition + b) : 1.0f;
  r.pres = a.presence ? __ldg(a.presence + b) : 0.0f;
  r.freq = a.frequency ? __ldg(a.frequency + b) : 0.0f;
  if (tid == 0) s.bad = 0;
  const bool rows_ok = nodes >= 1 && n0 >= 0 && n0 + nodes <= a.total_nodes;
  const int N = rows_ok ? static_cast<int>(nodes) : 0;
  bool bad = !rows_ok || N > a.max_nodes || h0 < 0 || h1 < h0 || h1 > a.total_history || e0 < 0 || e1 < e0 ||
             e1 > a.total_bias || !(r.rep > 0.0f && r.rep < INFINITY) || !(fabsf(r.pres) < INFINITY) ||
             !(fabsf(r.freq) < INFINITY);
  const uint4 zero = make_uint4(0, 0, 0, 0), none = make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll
  for (int i = 4 * tid; i < kChunk; i += 4 * kThreads) {
    *reinterpret_cast<uint4*>(&s.count[i]) = zero;
    if (a.bias_ids) *reinterpret_cast<uint4*>(&s.entry[i]) = none;
  }
  *reinterpret_cast<uint4*>(&s.path[0][0] + 4 * tid) = zero;
  static_assert(kWarps * (kChunk / 32) == 4 * kThreads, "one store per thread clears the bitmaps");
  __syncthreads();
  if (!bad) {
    for (int i = tid; i < N; i += kThreads) {
      const int p = __ldg(a.parent + n0 + i);
      s.parent[i] = p;
      s.token[i] = __ldg(a.tokens + n0 + i);
      if (i == 0 ? p != -1 : (p < 0 || p >= i)) s.bad = 1;
    }
    // history: ids outside the chunk (and outside the vocabulary) do not count
    const int prompt = a.prompt_lens ? max(0, __ldg(a.prompt_lens + b)) : 0;
    constexpr int kH = 8;  // entries in flight
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
  bad = bad || s.bad;
  if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) a.status[b] = bad ? kBadTree : kOk;
  if (!rows_ok) return;
  if (bad) {  // the rows as given
    for (int i = tid; i < kChunk; i += kThreads) s.count[i] = 0u;
    __syncthreads();
  }
  if (a.bias_ids) {
    for (int i = tid; i < kChunk; i += kThreads) {
      const int e = s.entry[i];
      s.bias[i] = e >= 0 ? __ldg(a.bias_values + e) : 0.0f;
    }
    __syncthreads();
  }
  const bool has_bias = a.bias_ids != nullptr && !bad;
  const uint32_t* mask = bad ? nullptr : a.allowed_mask;
  const int words = (a.vocab + 31) / 32;
  uint32_t* path = s.path[warp];
  for (int i = blockIdx.z * kWarps + warp; i < N; i += gridDim.z * kWarps) {
    const size_t row = static_cast<size_t>(n0 + i);
    const void* in = static_cast<const uint8_t*>(a.logits) + row * a.vocab * (BF16 ? 2 : 4);
    float* out = a.out + row * a.vocab;
    const uint32_t* mrow = mask ? mask + row * words : nullptr;
    // the drafted tokens of the path in this chunk: lane k looks at every 32nd
    // ancestor from the node up; the first node with a token computes it
    bool any = false;
    if (!bad) {
      int j = i;
      for (int k = 0; k < lane && j > 0; ++k) j = s.parent[j];
      while (__any_sync(0xffffffffu, j > 0)) {
        const int v = j > 0 ? s.token[j] - c0 : -1;
        bool mine = v >= 0 && v < nv;
        if (mine) {
          uint32_t more = 0;
          for (int m = i; m > 0; m = s.parent[m]) {
            if (s.token[m] != v + c0) continue;
            if (more == 0 && m != j) {  // (a node nearer to i has it)
              mine = false;
              break;
            }
            ++more;
          }
          if (mine) {
            const bool ok = !mrow || (__ldg(mrow + ((c0 + v) >> 5)) >> ((c0 + v) & 31) & 1u);
            const float x = load_logit<BF16>(in, c0 + v);
            out[c0 + v] = apply(x, s.count[v], more, has_bias ? s.bias[v] : 0.0f, ok, r);
            atomicOr(&path[v >> 5], 1u << (v & 31));
          }
        }
        any |= __any_sync(0xffffffffu, mine);
        for (int k = 0; k < 32 && j > 0; ++k) j = s.parent[j];
      }
      __syncwarp();
    }
    if (VEC) {
      constexpr int kU = 4;
#pragma unroll 1
      for (int q0 = 4 * lane; q0 < nv; q0 += 128 * kU) {
        float4 x[kU];
        uint32_t ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int v = q0 + 128 * u;
          if (v >= nv) continue;
          x[u] = load_logit4<BF16>(in, c0 + v);
          ok[u] = mrow ? __ldg(mrow + ((c0 + v) >> 5)) >> (v & 31) : 15u;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int v = q0 + 128 * u;
          if (v >= nv) continue;
          const uint4 c = *reinterpret_cast<const uint4*>(&s.count[v]);
          float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (has_bias) bias = *reinterpret_cast<const float4*>(&s.bias[v]);
          float4 y;
          if ((c.x | c.y | c.z | c.w) == 0u) {
            y = make_float4(x[u].x + bias.x, x[u].y + bias.y, x[u].z + bias.z, x[u].w + bias.w);
            if (!has_bias) y = x[u];  // (keeps a -0)
            y.x = ok[u] & 1u ? y.x : -INFINITY;
            y.y = ok[u] & 2u ? y.y : -INFINITY;
            y.z = ok[u] & 4u ? y.z : -INFINITY;
            y.w = ok[u] & 8u ? y.w : -INFINITY;
          } else {
            y.x = apply(x[u].x, c.x, 0, bias.x, ok[u] & 1u, r);
            y.y = apply(x[u].y, c.y, 0, bias.y, ok[u] & 2u, r);
            y.z = apply(x[u].z, c.z, 0, bias.z, ok[u] & 4u, r);
            y.w = apply(x[u].w, c.w, 0, bias.w, ok[u] & 8u, r);
          }
          const uint32_t skip = any ? path[v >> 5] >> (v & 31) & 15u : 0u;
          if (skip == 0u) {
            __stcs(reinterpret_cast<float4*>(out + c0 + v), y);
          } else {
            if (!(skip & 1u)) out[c0 + v] = y.x;
            if (!(skip & 2u)) out[c0 + v + 1] = y.y;
            if (!(skip & 4u)) out[c0 + v + 2] = y.z;
            if (!(skip & 8u)) out[c0 + v + 3] = y.w;
          }
        }
      }
    } else {
      constexpr int kU = 8;
#pragma unroll 1
      for (int q0 = lane; q0 < nv; q0 += 32 * kU) {
        float x[kU];
        uint32_t ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int v = q0 + 32 * u;
          if (v >= nv) continue;
          x[u] = load_logit<BF16>(in, c0 + v);
          ok[u] = mrow ? __ldg(mrow + ((c0 + v) >> 5)) >> (v & 31) & 1u : 1u;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int v = q0 + 32 * u;
          if (v >= nv || (any && (path[v >> 5] >> (v & 31) & 1u))) continue;
          const float y = s.count[v] || has_bias ? apply(x[u], s.count[v], 0, has_bias ? s.bias[v] : 0.0f, ok[u], r)
                                                 : (ok[u] ? x[u] : -INFINITY);
          __stcs(out + c0 + v, y);
        }
      }
    }
    if (any) {
      __syncwarp();
      for (int k = lane; k < kChunk / 32; k += 32) path[k] = 0u;
      __syncwarp();
    }
  }
}

}  // namespace

int launch_penalty(const PenaltyArgs& a, int sms, cudaStream_t stream) {
  const int chunks = (a.vocab + kChunk - 1) / kChunk;
  // shares of a tree's rows: enough CTAs to fill the SMs (5 fit one), at least
  // a row per warp
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
