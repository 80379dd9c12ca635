// beam_kernel.cu -- the next beams of every request: the best S continuations
// over its K beams and the vocabulary.
//
// Beam r with score s_r (the sum of its tokens' log-probabilities) and logits x
// offers every token v at
//   d = s_r + x_v - LSE(x),     LSE(x) = m + log sum_v exp(x_v - m), m = max x;
// an ended beam offers itself once, at s_r.  Candidates are ordered by
// key = d / max(len, 1)^alpha, then the lower beam, then the lower token.
//
// One pass over the logits.  beam_rows_kernel: a CTA takes a part of a row (at
// most 8184 entries, 32 a thread, which stay in registers), and finds the part's
// maximum, its sum and its S best entries.  Those are found without sorting: if
// of W warps each has c threads whose largest entry is at least t, and W c >= S,
// no entry below t is among the S best.  So t is the least over the warps of
// their c-th largest thread maximum; the entries from t on, a few more than S, go
// to shared memory and are ranked by counting.  Within a row the order is exact:
// it is that of the logits.
//
// beam_merge_kernel: a CTA per request joins the parts of each row to its LSE
// and picks the S best of all rows' lists the same way: in fp32 with an error
// bound that keeps every candidate that may be among them, those few in fp64.
//
// LSE: exps and their sums in fp32 against the part's own maximum (x - m rounded
// once, its product with log2 e in two pieces), joined in fp32 and added to m in
// fp64: off by about 1e-7, less than the rounding of a score near 20 to fp32
// (1e-6).  Candidates of different beams that lie closer than that may come in
// either order, the same in every call.
//
// Bound: HBM, one read of the logits; for few requests the latency of two
// dependent kernels.
#include <limits.h>
#include <math.h>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPart = 8192;          // entries that a CTA's threads hold
constexpr int kMaxSelect = 64;
constexpr int kMaxBeams = 64;
constexpr int kMaxParts = 33;        // of a row of 2^18 - 1 entries
constexpr int kMaxLength = 1 << 24;
constexpr int kFound = 1024;         // candidates that are ranked by counting
constexpr int kHeld = 8;             // candidates that a thread of the merge holds

// A float's place in the order of values (all NaN aside), as a signed integer.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b < 0 ? b ^ 0x7fffffff : b;
}
__device__ __forceinline__ float of_ordered(int k) { return __int_as_float(k < 0 ? k ^ 0x7fffffff : k); }

// The n-th largest of the warp's 32 values (n <= 32), and the largest.
__device__ __forceinline__ float nth_largest(float mine, int n, float& top) {
  int key = ordered(mine);
  const int lane = threadIdx.x & 31;
  int best = __reduce_max_sync(0xffffffffu, key);
  top = of_ordered(best);
  for (int i = 1; i < n; ++i) {
    if (lane == __ffs(__ballot_sync(0xffffffffu, key == best)) - 1) key = INT_MIN;
    best = __reduce_max_sync(0xffffffffu, key);
  }
  return of_ordered(best);
}

struct PartSmem {
  float top[kWarps], nth[kWarps], sum[kWarps];
  float value[kFound];
  int index[kFound];
  unsigned long long best[2];
  int found;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 3) beam_rows_kernel(const BeamArgs a) {
  constexpr int kEach = BF16 ? 8 : 4;            // entries of 16 bytes
  constexpr int kLoads = kPart / kThreads / kEach;
  __shared__ PartSmem s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int part = blockIdx.x % a.parts, row = blockIdx.x / a.parts;
  if (a.finished && a.finished[row] != 0) return;
  if (!(a.scores[row] > -INFINITY)) return;      // (nothing, or NaN: the merge sees it)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = part * a.chunk, c1 = min(c0 + a.chunk, a.vocab);
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + static_cast<size_t>(row) * a.stride * (16 / kEach);
  // whole 16-byte words, from the one that holds entry c0 on
  const int before = static_cast<int>((reinterpret_cast<uintptr_t>(base + static_cast<size_t>(c0) * (16 / kEach)) & 15) / (16 / kEach));
  const int start = c0 - before;
  const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;
  uint4 w[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int e = start + (tid + j * kThreads) * kEach;
    w[j] = make_uint4(none, none, none, none);
    if (e >= c0 && e + kEach <= c1) {
      w[j] = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<size_t>(e) * (16 / kEach)));
    } else if (e + kEach > c0 && e < c1) {
      uint32_t x[4] = {none, none, none, none};
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (e + i < c0 || e + i >= c1) continue;
        if (BF16) {
          const uint32_t v = reinterpret_cast<const uint16_t*>(base)[e + i];
          x[i / 2] = i % 2 ? (x[i / 2] & 0xffffu) | v << 16 : (x[i / 2] & 0xffff0000u) | v;
        } else {
          x[i % 4] = reinterpret_cast<const uint32_t*>(base)[e + i];
        }
      }
      w[j] = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  // entry i of word j; NaN counts as -inf
  const auto entry = [&](int j, int i) {
    const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
    const float v = BF16 ? __uint_as_float(i % 2 ? x[i / 2] & 0xffff0000u : x[i / 2] << 16) : __uint_as_float(x[i % 4]);
    return fmaxf(v, -INFINITY);
  };
  float mine = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
#pragma unroll
    for (int i = 0; i < kEach; ++i) mine = fmaxf(mine, entry(j, i));
  // warps whose threads all hold entries, and how many maxima each gives
  const int full = min(kThreads, (c1 - start + kEach - 1) / kEach) / 32;
  const int give = full > 0 && a.select <= 32 * full ? (a.select + full - 1) / full : 0;
  float top;
  const float nth = nth_largest(mine, give > 0 ? give : 1, top);
  if (lane == 0) {
    s.top[warp] = top;
    s.nth[warp] = nth;
  }
  if (tid == 0) s.found = 0;
  __syncthreads();
  float m = s.top[0], t = INFINITY;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    m = fmaxf(m, s.top[i]);
    if (i < full) t = fminf(t, s.nth[i]);
  }
  if (give == 0) t = -INFINITY;
  const size_t lists = static_cast<size_t>(a.beams) * a.parts;
  float2* list = a.lists + static_cast<size_t>(row / a.beams) * a.select * lists +
                 static_cast<size_t>(row % a.beams) * a.parts + part;
  // exp(x - m), 2^(d hi + d lo) with d = x - m; (lo > 0: -inf stays so)
  const float hi = 1.44269502162933349609f, lo = 1.92596298e-8f;
  const float ref = isinf(m) ? 0.0f : m;  // (nothing, or a +inf that the merge refuses)
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    float some = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float d = entry(j, i) - ref;
      some += ex2_approx(fmaf(d, hi, d * lo));
    }
    sum += some;
  }
  if (mine >= t) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float x = entry(j, i);
        if (x >= t && x > -INFINITY) {
          const int at = atomicAdd(&s.found, 1);
          if (at < kFound) {
            s.value[at] = x;
            s.index[at] = start + (tid + j * kThreads) * kEach + i;
          }
        }
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s.sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    float all = 0.0f;
    for (int i = 0; i < kWarps; ++i) all += s.sum[i];
    a.stats[static_cast<size_t>(row) * a.parts + part] = make_float2(m, all);
  }
  const int found = s.found;
  if (found <= kFound) {
    for (int i = tid; i < found; i += kThreads) {
      const float x = s.value[i];
      const int v = s.index[i];
      int rank = 0;
      for (int j = 0; j < found; ++j) rank += s.value[j] > x || (s.value[j] == x && s.index[j] < v);
      if (rank < a.select) list[rank * lists] = make_float2(x, __int_as_float(v));
    }
    for (int i = found + tid; i < a.select; i += kThreads) list[i * lists] = make_float2(-INFINITY, __int_as_float(-1));
    return;
  }
  // so many equal entries: the best after the last one, S times
  unsigned long long last = ~0ull;
  if (tid < 2) s.best[tid] = 0;
  __syncthreads();
  for (int r = 0; r < a.select; ++r) {
    unsigned long long best = 0;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float x = entry(j, i) + 0.0f;  // (one zero)
        const uint32_t v = start + (tid + j * kThreads) * kEach + i;
        const unsigned long long key =
            static_cast<unsigned long long>(static_cast<uint32_t>(ordered(x)) ^ 0x80000000u) << 32 | (0xffffffffu - v);
        if (x > -INFINITY && key < last && key > best) best = key;
      }
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) atomicMax(&s.best[r & 1], best);
    __syncthreads();
    last = s.best[r & 1];
    __syncthreads();
    if (tid == 0) {
      s.best[r & 1] = 0;  // (used again two rounds on, past the next barrier)
      const float x = of_ordered(static_cast<int>(static_cast<uint32_t>(last >> 32) ^ 0x80000000u));
      list[r * lists] = last ? make_float2(x, __uint_as_float(0xffffffffu - static_cast<uint32_t>(last)))
                             : make_float2(-INFINITY, __int_as_float(-1));
    }
  }
}

enum State { kDead, kLive, kEnded };

struct MergeSmem {
  double base[kMaxBeams];    // score - LSE; of an ended beam the score
  double inverse[kMaxBeams]; // 1 / len^alpha
  unsigned long long key[kFound + kMaxBeams];  // in the order of the keys' values
  float value[kFound + kMaxBeams];             // logit
  int at[kFound + kMaxBeams];                  // beam * 2^18 + token
  float2 approx[kMaxBeams];  // (base, inverse) in fp32
  unsigned long long best_key[kWarps];
  int best_at[kWarps], best_list[kWarps];
  int state[kMaxBeams];
  int live[kMaxBeams];       // the live beams, in order
  float nth[kWarps];
  uint8_t next[kMaxBeams * kMaxParts];  // of each list, the next entry
  int lives, ended, found, bad;
};

// A key's place in the order of values, as an unsigned integer above 0.
__device__ __forceinline__ unsigned long long ordered_key(double x) {
  const long long b = __double_as_longlong(x + 0.0);  // (one zero)
  return static_cast<unsigned long long>(b) ^ (b < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ bool better(unsigned long long k, int i, unsigned long long l, int j) {
  return k > l || (k == l && i < j);
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamArgs a) {
  __shared__ MergeSmem s;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.beams, S = a.select;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  // (what the caller gave; the rows kernel's results only after the wait)
  for (int k = tid; k < K; k += kThreads) {
    const size_t row = static_cast<size_t>(b) * K + k;
    const float score = a.scores[row];
    const bool ended = a.finished && a.finished[row] != 0;
    int len = a.lengths ? a.lengths[row] : 0;
    if (!(score < INFINITY) || len < 0 || len > kMaxLength) s.bad = 1;
    s.state[k] = !(score > -INFINITY) ? kDead : ended ? kEnded : kLive;
    len = max(len + (ended ? 0 : 1), 1);
    s.inverse[k] = a.length_penalty == 0.0f   ? 1.0
                   : a.length_penalty == 1.0f ? 1.0 / len
                                              : pow(static_cast<double>(len), -static_cast<double>(a.length_penalty));
    s.base[k] = score;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  // LSE of each live row, a warp a row
  for (int k = warp; k < K; k += kWarps) {
    if (s.state[k] != kLive) continue;
    const float2* part = a.stats + (static_cast<size_t>(b) * K + k) * a.parts;
    float m = -INFINITY;
    for (int p = lane; p < a.parts; p += 32) m = fmaxf(m, part[p].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.0f;
    if (!isinf(m))
      for (int p = lane; p < a.parts; p += 32) sum += part[p].y * expf(part[p].x - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (lane == 0) {
      if (m == INFINITY) s.bad = 1;
      if (isinf(m)) {
        s.state[k] = kDead;
      } else {
        // log of sum = 2^e f with f in [1, 2)
        const int e = (__float_as_int(sum) >> 23) - 127;
        const float f = __int_as_float(__float_as_int(sum) - (e << 23));
        s.base[k] -= static_cast<double>(m) + e * 0.69314718055994531 + static_cast<double>(logf(f));
      }
      s.approx[k] = make_float2(static_cast<float>(s.base[k]), static_cast<float>(s.inverse[k]));
    }
  }
  __syncthreads();
  const bool bad = s.bad != 0;
  if (tid == 0) {
    int live = 0, ended = 0;
    for (int k = 0; k < K; ++k) {
      if (s.state[k] == kLive) s.live[live++] = k;
      if (s.state[k] == kEnded) {  // its one candidate, at the lowest place of its beam
        s.key[ended] = ordered_key(s.base[k] * s.inverse[k]);
        s.value[ended] = 0.0f;
        s.at[ended++] = k << 18;
      }
    }
    s.lives = bad ? 0 : live;
    s.ended = s.found = bad ? 0 : ended;
    a.status[b] = bad ? kBadTree : kOk;
  }
  __syncthreads();
  const int own = s.lives * a.parts, total = own * S;
  const size_t lists = static_cast<size_t>(K) * a.parts;
  const float2* all = a.lists + static_cast<size_t>(b) * S * lists;
  // entry r of list q of the live beams, and the list's beam
  const auto beam_of = [&](int q) { return s.live[q / a.parts]; };
  const auto entry = [&](int q, int r) {
    return all[r * lists + static_cast<size_t>(beam_of(q)) * a.parts + q % a.parts];
  };
  // a key in fp32, and how far that may be off
  const auto approx = [&](float x, int k, float& off) {
    const float2 p = s.approx[k];
    off = p.y * (0x1p-22f * (fabsf(x) + fabsf(p.x)));
    return (x + p.x) * p.y;
  };
  const auto key_of = [&](float x, int k) { return ordered_key((s.base[k] + static_cast<double>(x)) * s.inverse[k]); };
  const auto keep = [&](float2 e, int k) {
    const int at = atomicAdd(&s.found, 1);
    if (at < kFound + kMaxBeams) {
      s.key[at] = key_of(e.x, k);
      s.value[at] = e.x;
      s.at[at] = k << 18 | __float_as_int(e.y);
    }
  };
  // A bound: S candidates at least are no worse.  From a few entries of each
  // thread, rank by rank over the lists.
  float2 held[kHeld];
  float top = -INFINITY, unused;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = tid + j * kThreads, r = own ? c / own : 0, q = c - r * own;
    held[j] = make_float2(-INFINITY, 0.0f);
    if (c < total) {
      float off;
      held[j] = entry(q, r);
      const float v = approx(held[j].x, beam_of(q), off);
      top = fmaxf(top, v - off);  // (NaN: none)
    }
  }
  for (int q = kThreads * kHeld + tid; q < own; q += kThreads) {  // (more lists than that)
    float off;
    const float v = approx(entry(q, 0).x, beam_of(q), off);
    top = fmaxf(top, v - off);
  }
  const int full = min(total, kThreads) / 32;
  const int give = full > 0 && S <= 32 * full ? (S + full - 1) / full : 0;
  const float nth = nth_largest(top, give > 0 ? give : 1, unused);
  if (lane == 0) s.nth[warp] = nth;
  __syncthreads();
  float t = INFINITY;
#pragma unroll
  for (int i = 0; i < kWarps; ++i)
    if (i < full) t = fminf(t, s.nth[i]);
  if (give == 0) t = -INFINITY;
  if (total <= kThreads * kHeld) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int c = tid + j * kThreads;
      if (!(held[j].x > -INFINITY)) continue;
      const int k = beam_of(c % own);
      float off;
      const float v = approx(held[j].x, k, off);
      if (!(v + off < t)) keep(held[j], k);
    }
  } else {
    // a list is in order: its entries until one is worse
    for (int q = tid; q < own; q += kThreads) {
      const int k = beam_of(q);
      bool more = true;
      for (int r0 = 0; more && r0 < S; r0 += 4) {
        float2 e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = r0 + j < S ? entry(q, r0 + j) : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float off;
          const float v = approx(e[j].x, k, off);
          more = more && e[j].x > -INFINITY && !(v + off < t);
          if (more) keep(e[j], k);
        }
      }
    }
  }
  __syncthreads();
  const auto put = [&](int rank, float x, int at) {
    const int k = at >> 18;
    const size_t row = static_cast<size_t>(b) * K + k, o = static_cast<size_t>(b) * S + rank;
    const bool ended = s.state[k] == kEnded;
    const int token = ended ? a.end_token : at & ((1 << 18) - 1);
    a.tokens[o] = token;
    a.parents[o] = static_cast<int>(row);
    a.scores_out[o] = static_cast<float>(ended ? s.base[k] : s.base[k] + static_cast<double>(x));
    if (a.lengths_out) a.lengths_out[o] = a.lengths[row] + (ended ? 0 : 1);
    if (a.finished_out) a.finished_out[o] = ended || (a.end_token >= 0 && token == a.end_token);
  };
  const auto put_none = [&](int rank) {
    const size_t o = static_cast<size_t>(b) * S + rank;
    a.tokens[o] = a.parents[o] = -1;
    a.scores_out[o] = -INFINITY;
    if (a.lengths_out) a.lengths_out[o] = 0;
    if (a.finished_out) a.finished_out[o] = 0;
  };
  const int found = s.found;
  if (found <= kFound + kMaxBeams) {
    for (int i = tid; i < found; i += kThreads) {
      const unsigned long long key = s.key[i];
      const int at = s.at[i];
      int rank = 0;
      for (int j = 0; j < found; ++j) rank += better(s.key[j], s.at[j], key, at);
      if (rank < S) put(rank, s.value[i], at);
    }
    for (int i = found + tid; i < S; i += kThreads) put_none(i);
    return;
  }
  // so many alike: the best of the lists' next entries, S times
  for (int q = tid; q < own; q += kThreads) s.next[q] = 0;
  __syncthreads();
  unsigned ended_left = 0;  // of the ended beams' candidates, a thread's (two at most) that are not taken
  for (int i = tid, j = 0; i < s.ended; i += kThreads, ++j) ended_left |= 1u << j;
  for (int rank = 0; rank < S; ++rank) {
    unsigned long long key = 0;
    int at = INT_MAX, list = -1;
    for (int q = tid; q < own; q += kThreads) {
      const int r = s.next[q];
      if (r >= S) continue;
      const float2 e = entry(q, r);
      const int k = beam_of(q), place = k << 18 | __float_as_int(e.y);
      if (!(e.x > -INFINITY)) continue;
      const unsigned long long v = key_of(e.x, k);
      if (better(v, place, key, at)) key = v, at = place, list = q;
    }
    for (int i = tid, j = 0; i < s.ended; i += kThreads, ++j)
      if ((ended_left >> j & 1u) && better(s.key[i], s.at[i], key, at)) key = s.key[i], at = s.at[i], list = -2 - i;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, key, o);
      const int a2 = __shfl_xor_sync(0xffffffffu, at, o), l2 = __shfl_xor_sync(0xffffffffu, list, o);
      if (better(k2, a2, key, at)) key = k2, at = a2, list = l2;
    }
    if (lane == 0) s.best_key[warp] = key, s.best_at[warp] = at, s.best_list[warp] = list;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i)
      if (better(s.best_key[i], s.best_at[i], key, at)) key = s.best_key[i], at = s.best_at[i], list = s.best_list[i];
    if (list == -1) {
      if (tid == 0) put_none(rank);
    } else if (list >= 0) {
      if (tid == list % kThreads) {
        put(rank, entry(list, s.next[list]).x, at);
        s.next[list] += 1;
      }
    } else if (tid == (-2 - list) % kThreads) {
      put(rank, 0.0f, at);
      ended_left &= ~(1u << ((-2 - list) / kThreads));
    }
    __syncthreads();
  }
}

}  // namespace

int beam_parts(int vocab) { return (vocab + kPart - 8 - 1) / (kPart - 8); }
int beam_max_select() { return kMaxSelect; }
int beam_max_beams() { return kMaxBeams; }
int beam_part_entries() { return kPart - 8; }

int launch_beam_select(const BeamArgs& a, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(a.batch) * a.beams * a.parts;
  if (a.bf16) {
    beam_rows_kernel<true><<<rows, kThreads, 0, stream>>>(a);
  } else {
    beam_rows_kernel<false><<<rows, kThreads, 0, stream>>>(a);
  }
  if (cudaGetLastError() != cudaSuccess) return -1;
  // the merge's CTAs may start while the last rows are read; they wait for them
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge_kernel, a) == cudaSuccess ? 0 : -1;
}

}  // namespace tv
