// beam_kernel.cu -- the next beams of every request: the best S continuations
// over its K beams and the vocabulary.
//
// Beam r with score s_r (the sum of its tokens' log-probabilities) and logits x
// offers every token v at
//   d = s_r + x_v - LSE(x),     LSE(x) = m + log sum_v exp(x_v - m), m = max x;
// an ended beam offers itself once, at s_r.  Candidates are ordered by
// key = d / max(len, 1)^alpha, then the lower beam, then the lower token.
//
// beam_rows_kernel: a warp takes a part of a row, four 16-byte words a lane at a time,
// the next ones on their way to shared memory.  Each lane keeps a running maximum and
// the sum of exps against it, and notes the largest entry of its words of every turn.
// After its part each warp tells a bound: if warp w has c_w lanes whose largest entry is
// at least t, and the c_w add up to S, S entries of the row are no worse than t; the 8
// warps of a CTA, which work on one row, take the least of their c_w-th largest, c_w
// about S / 8.  Few noted entries pass it (3 to 6 of 512 of a warp; where many do, as
// with a mask over some warps' parts, the warps tell bounds of their own notes and take
// the best: 64 x 8 of V = 128256 with the upper half masked 63 us, without 151); their
// words are read again, an entry a lane, and ranked into the warp's list.  Within a row
// the order is exact: it is that of the logits, and of equal ones the lower token.
//
// beam_merge_kernel: a CTA per request joins the parts of each row to its LSE
// and picks the S best of all rows' lists the same way: in fp32 with an error
// bound that keeps every candidate that may be among them, those few in fp64; equal keys
// there by beam, logit and token.
//
// LSE: exps and their sums in fp32 against the lane's own maximum, lanes and parts joined
// in fp32, the logarithm and the maximum added in fp64: off by less than 2^-15, the sum of
// its operations' bounds, of which 2^-15.7 are the factors of up to 64 turns that each
// raise the maximum a little; without those 2^-17.  Measured: 2e-7 at most on random rows,
// 4e-6 on rows made for it (a peak of every lane, then equal entries).  Candidates of
// different beams that lie closer than that may come in either order, the same in every
// call.
//
// Bound: HBM for large calls (18 us of the first one here are the pass over the logits,
// near 7 TB/s; then the bound and the lists, 3 to 4, up to 4 more where 4 instead of 3 of
// the 512 CTAs are on an SM, and the merge's 5); for few requests the latency of two
// dependent kernels.  Measured (device time, the call
// replayed): 64 requests of 8 beams, V = 128256, bf16, S = 16: 35 us; 32 of 8, V = 32000,
// fp32: 15.4; 1 of 4: 9.2.  On the way, the first case: a CTA per 8192 entries, entries
// in registers and ranks of the CTA's threads' maxima 153 us; a warp a part with its own
// bound that rises as it reads 71; bounds shared by a CTA's warps while they read 53;
// words from shared memory, looked at by all lanes 36, the second 18.8 (a quarter of the
// instructions was a look at words that had an entry from the bound on, in most turns).
// The barrier that such a late bound asks for, ranks by a list's scan and noted entries
// of every turn in the bound: 40.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSelect = 64;
constexpr int kMaxBeams = 64;
constexpr int kMaxParts = 32;        // of a row
constexpr int kMaxLength = 1 << 24;
constexpr int kWords = 4;            // 16-byte words that a lane has in flight
constexpr int kStages = 2;           // of them
constexpr int kList = 2 * kMaxSelect + 16;  // entries of a warp's list
constexpr int kFound = 1024;         // candidates that the merge ranks by counting
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

// A warp's words on their way, and its list: entries from its bound on.
struct List {
  uint4 ring[kStages][32 * kWords];
  float value[kList];   // -inf: taken
  int index[kList];
  float2 best[kMaxSelect];
};

// Keeps the best n of the list's `count` entries, in order, in l.best and at the
// list's front; returns how many there are.
__device__ int keep_best(List& l, int count, int n) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (count <= 64) {  // each entry's rank by counting
    for (int j = lane; j < count; j += 32) {
      const float x = l.value[j];
      const int k = l.index[j];
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < count; ++o) rank += l.value[o] > x || (l.value[o] == x && l.index[o] < k);
      if (rank < n) l.best[rank] = make_float2(x, __int_as_float(k));
    }
    const int kept = min(count, n);
    __syncwarp();
    for (int j = lane; j < kept; j += 32) {
      l.value[j] = l.best[j].x;
      l.index[j] = __float_as_int(l.best[j].y);
    }
    __syncwarp();
    return kept;
  }
  float v = -INFINITY;
  int i = INT_MAX, slot = 0;
  const auto scan = [&] {
    v = -INFINITY, i = INT_MAX;
    for (int j = lane; j < count; j += 32) {
      const float x = l.value[j];
      const int k = l.index[j];
      if (x > v || (x == v && k < i)) v = x, i = k, slot = j;
    }
  };
  scan();
  int kept = 0;
  for (; kept < n; ++kept) {
    const int key = ordered(v), top = __reduce_max_sync(0xffffffffu, key);
    if (top == ordered(-INFINITY)) break;
    const int first = __reduce_min_sync(0xffffffffu, key == top ? i : INT_MAX);
    if (key == top && i == first) {
      l.best[kept] = make_float2(v, __int_as_float(i));
      l.value[slot] = -INFINITY;
      scan();
    }
  }
  __syncwarp();
  for (int j = lane; j < kept; j += 32) {
    l.value[j] = l.best[j].x;
    l.index[j] = __float_as_int(l.best[j].y);
  }
  __syncwarp();
  return kept;
}

// A part of a row: entries [c0, c1) from `base` on, in 16-byte words, the first of
// which holds entry c0.
template <bool BF16>
struct Part {
  static constexpr int kEach = BF16 ? 8 : 4;  // entries of a word
  const uint8_t* base;
  int c0, c1, start;
  __device__ __forceinline__ int entry_of(int word) const { return start + word * kEach; }
  // a word; entries outside of the part -inf
  __device__ __forceinline__ uint4 load(int word) const {
    const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;
    const int e = entry_of(word);
    if (e >= c0 && e + kEach <= c1) return __ldcs(reinterpret_cast<const uint4*>(base + static_cast<long long>(e) * (16 / kEach)));
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
    return make_uint4(x[0], x[1], x[2], x[3]);
  }
};
// A word's values, two by two.
template <bool BF16>
__device__ __forceinline__ void values_of(const uint4& w, float2 (&v)[BF16 ? 4 : 2]) {
  if constexpr (BF16) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
  } else {
    v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}
// NaN as -inf
template <bool BF16>
__device__ __forceinline__ uint4 without_nan(uint4 w) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      if ((x[i] & 0x7fffu) > 0x7f80u) x[i] = (x[i] & 0xffff0000u) | 0xff80u;
      if ((x[i] & 0x7fff0000u) > 0x7f800000u) x[i] = (x[i] & 0xffffu) | 0xff800000u;
    } else if ((x[i] & 0x7fffffffu) > 0x7f800000u) {
      x[i] = 0xff800000u;
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// exp(d) for d = x - m <= 0 as 2^(d hi + d lo)   (lo > 0: -inf stays so)
constexpr float kLog2eHi = 1.44269502162933349609f, kLog2eLo = 1.92596298e-8f;
__device__ __forceinline__ float exp_of(float d) { return ex2_approx(fmaf(d, kLog2eHi, d * kLog2eLo)); }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two words' larger values, place by place (a number rather than NaN).
template <bool BF16>
__device__ __forceinline__ uint4 most_of(const uint4& a, const uint4& b) {
  if constexpr (BF16) {
    return make_uint4(max_bf16x2(a.x, b.x), max_bf16x2(a.y, b.y), max_bf16x2(a.z, b.z), max_bf16x2(a.w, b.w));
  } else {
    const auto most = [](uint32_t x, uint32_t y) { return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y))); };
    return make_uint4(most(a.x, b.x), most(a.y, b.y), most(a.z, b.z), most(a.w, b.w));
  }
}
// The largest value of a word (of numbers and NaN, that of the numbers).
template <bool BF16>
__device__ __forceinline__ float top_of(const uint4& w) {
  if constexpr (BF16) {
    const uint32_t m = max_bf16x2(max_bf16x2(w.x, w.y), max_bf16x2(w.z, w.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
}

// Where word i of a stage is: lane l's are 4 l .. 4 l + 3, and eight lanes' j-th ones lie
// in different banks.
__device__ __forceinline__ int place_of(int i) { return (i & ~3) | ((i ^ i >> 3) & 3); }

// The four words of each lane from word w0 on, on their way into a stage.
template <bool BF16>
__device__ __forceinline__ void fetch_words(const Part<BF16>& p, int w0, uint4* stage) {
  const int lane = threadIdx.x & 31;
  if (p.entry_of(w0) >= p.c0 && p.entry_of(w0 + 32 * kWords) <= p.c1) {
    const uint8_t* at = p.base + static_cast<long long>(p.entry_of(w0 + lane)) * (16 / p.kEach);
#pragma unroll
    for (int j = 0; j < kWords; ++j) cpa16(stage + place_of(j * 32 + lane), at + j * 512);
  } else {
#pragma unroll 1
    for (int j = 0; j < kWords; ++j) {
      const int w = w0 + j * 32 + lane, e = p.entry_of(w);
      if (e >= p.c0 && e + p.kEach <= p.c1) {
        cpa16(stage + place_of(j * 32 + lane), p.base + static_cast<long long>(e) * (16 / p.kEach));
      } else {
        stage[place_of(j * 32 + lane)] = p.load(w);
      }
    }
  }
}
__device__ __forceinline__ void commit_words() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_words() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }

// What the warps of a CTA tell each other: the c_w-th largest of their lanes' maxima
// (+inf of warps without a part) and, where that leaves many, a bound of their own (-inf:
// none).  NaN: not known yet.
struct Bounds {
  float nth[kWarps], own[kWarps];
};
// All warps' (every warp tells its own whatever the others do): that of warp `lane`.
__device__ __forceinline__ float told(const float* of, float others) {
  const int lane = threadIdx.x & 31;
  float t = NAN;
  for (int i = 0; i < 1 << 20 && __any_sync(0xffffffffu, t != t); ++i)
    t = lane < kWarps ? reinterpret_cast<const volatile float*>(of)[lane] : others;
  return t == t ? t : -INFINITY;
}

// One pass over a part by a warp: the maximum m and sum of exp(x - m), and of every
// lane's words of every turn the largest entry, as the upper half of its place in the
// order (of fp32 rounded down, as the bound's is), in tops.  Returns whether it is done.
//
// The sums are of 2^(x hi + c), hi = fl(log2 e), c = -fl(m hi) with m the lane's
// maximum so far: rounded once, near 0 where it counts.  (hi is log2 e but for 1.3e-8
// of it: an entry 10 below the maximum counts 1.3e-7 too much or too little, below
// the approximate power's own error.)  Where a sum is NaN (a NaN among the entries)
// or the maximum beyond 2^20 (a part that is masked by the lowest value), the pass
// is done again (SAFE), without NaN and from x - m.
template <bool BF16, bool SAFE>
__device__ bool part_pass(const Part<BF16>& p, List& l, int16_t* tops, Bounds* bounds, int give, float& m, float& sum) {
  constexpr int kPairs = BF16 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int words = (p.c1 - p.start + p.kEach - 1) / p.kEach;
  m = SAFE ? -FLT_MAX : -0x1p126f;  // (not -inf: nothing minus nothing)
  float high = -INFINITY;
  float c = -m * kLog2eHi;
  float2 acc = make_float2(0.0f, 0.0f);
  // (the first stages are the caller's)
  for (int w0 = 0, turn = 0; w0 < words; w0 += 32 * kWords, ++turn) {
    wait_words();
    __syncwarp();
    uint4* stage = l.ring[turn % kStages];
    uint4 w[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      w[j] = stage[place_of(lane * kWords + j)];
      if (SAFE) w[j] = without_nan<BF16>(w[j]);
    }
    __syncwarp();
    const int ahead = w0 + kStages * 32 * kWords;
    if (ahead < words) fetch_words<BF16>(p, ahead, stage);
    commit_words();
    const float top = fmaxf(top_of<BF16>(most_of<BF16>(most_of<BF16>(w[0], w[1]), most_of<BF16>(w[2], w[3]))), -INFINITY);
    if (!SAFE) tops[turn * 32 + lane] = static_cast<int16_t>(ordered(top + 0.0f) >> 16);
    high = fmaxf(high, top);
    if (!SAFE && w0 + 32 * kWords >= words) {  // (the last turn)
      float unused;
      const float nth = give <= 32 ? nth_largest(high, give, unused) : -INFINITY;
      if (lane == 0) reinterpret_cast<volatile float*>(bounds->nth)[threadIdx.x >> 5] = nth;
    }
    if (top > m) {
      if (SAFE) {
        const float f = exp_of(m - top);
        acc.x *= f, acc.y *= f;
      } else {
        const float to = -top * kLog2eHi, f = ex2_approx(to - c);
        acc.x *= f, acc.y *= f;
        c = to;
      }
      m = top;
    }
    float2 part = make_float2(0.0f, 0.0f);  // (a turn's by itself: few roundings of each term)
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      float2 v[kPairs];
      values_of<BF16>(w[j], v);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        float2 e;
        if (SAFE) {
          const float2 d = add2(v[i], make_float2(-m, -m));
          e = fma2(d, make_float2(kLog2eHi, kLog2eHi), mul2(d, make_float2(kLog2eLo, kLog2eLo)));
        } else {
          e = fma2(v[i], make_float2(kLog2eHi, kLog2eHi), make_float2(c, c));
        }
        part = add2(part, make_float2(ex2_approx(e.x), ex2_approx(e.y)));
      }
    }
    acc = add2(acc, part);
  }
  sum = acc.x + acc.y;
  const float all = of_ordered(__reduce_max_sync(0xffffffffu, ordered(m)));
  const bool fails = __any_sync(0xffffffffu, sum != sum) || (!SAFE && !(fabsf(all) <= 0x1p20f));
  if (!SAFE) {
    // as of 2^((x - m) hi): by 2^(-c - m hi), next to 1
    const float y = -0.69314718f * fmaf(m, kLog2eHi, c);
    sum = fabsf(y) < 0x1p-8f ? fmaf(sum, fmaf(y * y, 0.5f, y), sum) : sum * expf(y);
  }
  // the lanes' sums against the warp's maximum
  sum = m < all - 256.0f ? 0.0f : sum * exp_of(m - all);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  m = of_ordered(__reduce_max_sync(0xffffffffu, ordered(high)));
  if (m == -INFINITY) {  // nothing (but NaN)
    sum = 0.0f;
    return true;
  }
  return !fails;
}

// The first stages of a part's words on their way.
template <bool BF16>
__device__ __forceinline__ void start_words(const Part<BF16>& p, List& l) {
  const int words = (p.c1 - p.start + p.kEach - 1) / p.kEach;
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    if (i == 0 || i * 32 * kWords < words) fetch_words<BF16>(p, i * 32 * kWords, l.ring[i]);
    commit_words();
  }
}

// The part's entries from the CTA's bound on into the warp's list; returns how many
// there are.  For all warps of the CTA that have parts.
template <bool BF16>
__device__ int collect(const Part<BF16>& p, List& l, const int16_t* tops, Bounds* bounds, int select) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (p.c1 - p.start + p.kEach - 1) / p.kEach, turns = (words + 32 * kWords - 1) / (32 * kWords);
  float t = of_ordered(__reduce_min_sync(0xffffffffu, ordered(told(bounds->nth, INFINITY))));
  t = fmaxf(t, -FLT_MAX);  // (-inf is no candidate)
  uint16_t* codes = reinterpret_cast<uint16_t*>(l.ring);
  constexpr int kCodes = sizeof(l.ring) / 2, kOf = kWords * p.kEach, kAtOnce = 32 / kOf, kFly = 8 / kAtOnce;
  int n = 0, count = 0;
  bool raised = false;
  const auto look = [&] {
    __syncwarp();
    for (int q = 0; q < n; q += kFly * kAtOnce) {
      if (raised) {  // (by now none of these may pass)
        const int k = q + lane;
        if (!__any_sync(0xffffffffu, lane < kFly * kAtOnce && k < n && tops[codes[min(k, n - 1)]] >= ordered(t) >> 16)) continue;
      }
      float x[kFly];
      int at[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const int k = q + u * kAtOnce + lane / kOf, code = k < n ? codes[k] : 0;
        at[u] = p.entry_of(((code >> 5) * 32 + (code & 31)) * kWords) + lane % kOf;
        x[u] = -INFINITY;
        if (k < n && at[u] >= p.c0 && at[u] < p.c1)
          x[u] = BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.base)[at[u]]) << 16)
                      : reinterpret_cast<const float*>(p.base)[at[u]];
        x[u] += 0.0f;  // (one zero)
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const unsigned hit = __ballot_sync(0xffffffffu, x[u] >= t);
        if (hit == 0) continue;
        if (count + 32 > kList) {
          count = keep_best(l, count, select);
          // (of equal ones the later token does not count: from the type's next value on)
          if (count == select) t = fmaxf(t, of_ordered((ordered(l.value[select - 1]) | (BF16 ? 0xffff : 0)) + 1));
          raised = true;
        }
        const unsigned still = __ballot_sync(0xffffffffu, x[u] >= t);
        if (x[u] >= t) {
          const int to = count + __popc(still & ((1u << lane) - 1));
          l.value[to] = x[u];
          l.index[to] = at[u];
        }
        count += __popc(still);
      }
    }
    n = 0;
    __syncwarp();
  };
  // the lanes' words of turns that pass
  const auto gather = [&](bool all) {
    const int key = ordered(t) >> 16;
#pragma unroll 4
    for (int i = 0; i < turns; ++i) {
      const bool is = tops[i * 32 + lane] >= key;
      const unsigned has = __ballot_sync(0xffffffffu, is);
      if (is) codes[n + __popc(has & ((1u << lane) - 1))] = static_cast<uint16_t>(i * 32 + lane);
      n += __popc(has);
      if (n + 32 > kCodes) {
        if (!all) return;
        look();
      }
    }
  };
  gather(false);
  volatile float* own = reinterpret_cast<volatile float*>(bounds->own);
  if (n <= 32 + 4 * (select / kWarps)) {
    if (lane == 0) own[warp] = -INFINITY;
  } else {
    // The warps' words are not alike (a mask over some, a row that rises): the best of
    // the bounds of single warps' words, the largest that `select` of them are at or above.
    int low = ordered(t) >> 16, high = SHRT_MAX;
    while (low < high) {
      const int middle = (low + high + 1) >> 1;
      int some = 0;
#pragma unroll 4
      for (int i = 0; i < turns; ++i) some += tops[i * 32 + lane] >= middle;
      if (static_cast<int>(__reduce_add_sync(0xffffffffu, some)) >= select) {
        low = middle;
      } else {
        high = middle - 1;
      }
    }
    if (lane == 0) own[warp] = of_ordered(low << 16);
    t = fmaxf(t, of_ordered(__reduce_max_sync(0xffffffffu, ordered(told(bounds->own, -INFINITY)))));
    n = 0;
    __syncwarp();
    gather(true);
  }
  look();
  return count;
}

// CTAs behind those of the parts: len^alpha of a row per thread (its fp64 power would
// stand in the merge's way).
__device__ void row_powers(const BeamArgs& a, int row) {
  if (row >= a.batch * a.beams) return;
  const bool ended = a.finished && a.finished[row] != 0;
  const int len = max(min(a.lengths[row], kMaxLength) + (ended ? 0 : 1), 1);
  a.power[row] = a.length_penalty == 1.0f ? len : pow(static_cast<double>(len), static_cast<double>(a.length_penalty));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  List* lists = reinterpret_cast<List*>(raw);
  int16_t* tops = reinterpret_cast<int16_t*>(raw + kWarps * sizeof(List)) + (threadIdx.x >> 5) * a.turns * 32;
  __shared__ Bounds bounds;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = (a.parts + kWarps - 1) / kWarps;  // of a row
  const int row = blockIdx.x / ctas, cta = blockIdx.x - row * ctas;
  const int first = cta * a.each + min(cta, a.more), warps = a.each + (cta < a.more), part = first + warp;
  if (threadIdx.x < kWarps) {
    const bool here = static_cast<int>(threadIdx.x) < warps;
    bounds.nth[threadIdx.x] = here ? NAN : INFINITY;
    bounds.own[threadIdx.x] = here ? NAN : -INFINITY;
  }
  __syncthreads();
  if (row >= a.batch * a.beams) {
    row_powers(a, (blockIdx.x - a.batch * a.beams * ctas) * kThreads + threadIdx.x);
    return;
  }
  if (warp >= warps) return;
  const int ended = a.finished ? a.finished[row] : 0;
  const float score = a.scores[row];
  Part<BF16> p;
  p.base = static_cast<const uint8_t*>(a.logits) + static_cast<size_t>(row) * a.stride * (16 / p.kEach);
  p.c0 = min(part * a.chunk, a.vocab), p.c1 = min(p.c0 + a.chunk, a.vocab);
  p.start = p.c0 - static_cast<int>((reinterpret_cast<uintptr_t>(p.base + static_cast<size_t>(p.c0) * (16 / p.kEach)) & 15) / (16 / p.kEach));
  List& l = lists[warp];
  start_words<BF16>(p, l);  // (on their way while the row's state arrives)
  if (ended != 0 || !(score > -INFINITY)) {  // (nothing, or NaN: the merge sees it)
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const int give = max(1, a.select / warps + (warp < a.select % warps));
  float m, sum;
  if (!part_pass<BF16, false>(p, l, tops, &bounds, give, m, sum)) {
    start_words<BF16>(p, l);
    part_pass<BF16, true>(p, l, tops, &bounds, give, m, sum);
  }
  if (lane == 0) a.stats[static_cast<size_t>(row) * a.parts + part] = make_float2(m, sum);
  int count = collect<BF16>(p, l, tops, &bounds, a.select);
  const size_t all = static_cast<size_t>(a.beams) * a.parts;
  float2* list = a.lists + static_cast<size_t>(row / a.beams) * a.select * all + static_cast<size_t>(row % a.beams) * a.parts + part;
  if (count <= 32) {  // each entry's rank, a lane an entry
    const float x = lane < count ? l.value[lane] : -INFINITY;
    const int k = lane < count ? l.index[lane] : -1;
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < count; ++o) {
      const float y = __shfl_sync(0xffffffffu, x, o);
      rank += y > x || (y == x && o < lane && lane < count);
    }
    if (lane >= count) rank = lane;
    if (rank < a.select) list[rank * all] = make_float2(x, __int_as_float(k));
    if (32 + lane < a.select) list[(32 + lane) * all] = make_float2(-INFINITY, __int_as_float(-1));
    return;
  }
  count = keep_best(l, count, a.select);
  for (int i = lane; i < a.select; i += 32)
    list[i * all] = i < count ? make_float2(l.value[i], __int_as_float(l.index[i])) : make_float2(-INFINITY, __int_as_float(-1));
}

enum State { kDead, kLive, kEnded };

struct MergeSmem {
  double base[kMaxBeams];    // score - log sum; of an ended beam the score
  float top[kMaxBeams];      // the row's maximum
  double2 power[kMaxBeams];  // len^alpha and its inverse
  unsigned long long key[kFound + kMaxBeams];  // in the order of the keys' values
  float logit[kFound + kMaxBeams];
  float score[kFound + kMaxBeams];
  int at[kFound + kMaxBeams];                  // beam * 2^18 + token
  float2 approx[kMaxBeams];  // (base, 1 / power) in fp32
  unsigned long long best_key[kWarps];
  unsigned long long best_place[kWarps];
  int best_list[kWarps];
  int state[kMaxBeams], length[kMaxBeams];
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
// Among equal keys: beam, then the logit downwards, then the token.  (Where a score or a
// row's maximum is so large that the keys of different logits round to one value, the
// order within the row is still that of the logits.)
__device__ __forceinline__ unsigned long long place_in_order(int at, float logit) {
  const uint32_t down = 0x7fffffffu - static_cast<uint32_t>(ordered(logit));
  return static_cast<unsigned long long>(at >> 18) << 50 | static_cast<unsigned long long>(down) << 18 | static_cast<unsigned>(at & ((1 << 18) - 1));
}
__device__ __forceinline__ int at_of(unsigned long long place) {
  return static_cast<int>(place >> 50) << 18 | (static_cast<int>(place) & ((1 << 18) - 1));
}
template <typename T>
__device__ __forceinline__ bool better(unsigned long long k, T i, unsigned long long l, T j) {
  return k > l || (k == l && i < j);
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamArgs a) {
  __shared__ MergeSmem s;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.beams, S = a.select;
  // what the caller gave, by warp 0 (the rows kernel's results only after the wait)
  if (warp == 0) {
    bool bad = false;
    int live = 0, ended = 0;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int k = k0 + lane;
      int state = kDead;
      if (k < K) {
        const size_t row = static_cast<size_t>(b) * K + k;
        const float score = a.scores[row];
        const int len = a.lengths ? a.lengths[row] : 0;
        bad |= !(score < INFINITY) || len < 0 || len > kMaxLength;
        if (score > -INFINITY) state = a.finished && a.finished[row] != 0 ? kEnded : kLive;
        s.state[k] = state;
        s.length[k] = len;
        s.base[k] = score;
        s.power[k] = make_double2(1.0, 1.0);
      }
      const unsigned lives = __ballot_sync(0xffffffffu, state == kLive), ends = __ballot_sync(0xffffffffu, state == kEnded);
      const unsigned below = (1u << lane) - 1;
      if (state == kLive) s.live[live + __popc(lives & below)] = k;
      if (state == kEnded) s.at[ended + __popc(ends & below)] = k << 18;  // (its one candidate)
      live += __popc(lives);
      ended += __popc(ends);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s.lives = live;
      s.ended = s.found = ended;
      s.bad = bad;
    }
  }
  __syncthreads();
  const int own = s.lives * a.parts, total = own * S;
  const size_t lists = static_cast<size_t>(K) * a.parts;
  const float2* all = a.lists + static_cast<size_t>(b) * S * lists;
  // exact quotients of numbers below 2^18 by ones below 2^13
  const uint32_t by_own = own > 1 ? 0xffffffffu / own + 1 : 0, by_parts = a.parts > 1 ? 0xffffffffu / a.parts + 1 : 0;
  const auto over = [](int c, uint32_t by) { return by ? static_cast<int>(__umulhi(c, by)) : c; };
  // entry r of list q of the live beams, and the list's beam
  const auto beam_of = [&](int q) { return s.live[over(q, by_parts)]; };
  const auto entry = [&](int q, int r) {
    const int n = over(q, by_parts);
    return all[r * lists + static_cast<size_t>(s.live[n]) * a.parts + (q - n * a.parts)];
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // A few candidates of each thread, rank by rank over the lists; the lists of a beam
  // over all warps, whose bounds count alike below (in order, the warps with the
  // worst beams' lists let 10 times as many candidates pass).
  const int place = lane * kWarps + warp;
  static_assert(kMaxBeams * kMaxParts <= kThreads * kHeld, "every list's first entry");
  float2 held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = place + j * kThreads, r = over(c, by_own);
    held[j] = c < total ? entry(c - r * own, r) : make_float2(-INFINITY, 0.0f);
  }
  // len^alpha of each beam, a lane a beam, and its inverse (to 2^-46: keys add what their
  // product by it leaves)
  const int own_beam = tid - (kThreads - kMaxBeams);
  const bool powers = a.length_penalty != 0.0f && own_beam >= 0 && own_beam < K;
  const double power = powers ? a.power[static_cast<size_t>(b) * K + own_beam] : 1.0;
  // LSE of each live row, a warp a row
  for (int n = warp; n < s.lives; n += kWarps) {
    const int k = s.live[n];
    const size_t row = static_cast<size_t>(b) * K + k;
    const float2* part = a.stats + row * a.parts;
    const float2 x = lane < a.parts ? part[lane] : make_float2(-INFINITY, 0.0f);
    const float divisor = a.length_penalty != 0.0f ? static_cast<float>(a.power[row]) : 1.0f;
    const float m = of_ordered(__reduce_max_sync(0xffffffffu, ordered(x.x)));
    float sum = isinf(m) ? 0.0f : x.y * expf(x.x - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      if (m == INFINITY) s.bad = 1;
      if (!isinf(m)) {  // (else all its candidates are -inf)
        // log of sum = 2^e f with f in [1, 2)
        const int e = (__float_as_int(sum) >> 23) - 127;
        const float f = __int_as_float(__float_as_int(sum) - (e << 23));
        s.base[k] -= e * 0.69314718055994531 + static_cast<double>(logf(f));
      }
      s.top[k] = m;
      s.approx[k] = make_float2(static_cast<float>(s.base[k]), 1.0f / divisor);
    }
  }
  if (powers) {
    const double first = 1.0f / static_cast<float>(power);
    s.power[own_beam] = make_double2(power, fma(fma(-power, first, 1.0), first, first));
  }
  __syncthreads();
  if (tid == 0) a.status[b] = s.bad ? kBadTree : kOk;
  if (s.bad) {
    for (int i = tid; i < S; i += kThreads) {
      const size_t o = static_cast<size_t>(b) * S + i;
      a.tokens[o] = a.parents[o] = -1;
      a.scores_out[o] = -INFINITY;
      if (a.lengths_out) a.lengths_out[o] = 0;
      if (a.finished_out) a.finished_out[o] = 0;
    }
    return;
  }
  // a key in fp32, and how far that may be off: half a step each of d, the base, their
  // sum, the power, its inverse, their product, and of the key with `off` added
  const auto approx = [&](float x, int k, float& off) {
    const float2 p = s.approx[k];
    const float d = x - s.top[k];
    off = p.y * (0x1p-21f * (fabsf(d) + fabsf(p.x)));
    return (d + p.x) * p.y;
  };
  // (the maximum off first: rows of the type's lowest value have scores too)
  const auto score_of = [&](float x, int k) {
    return s.state[k] == kEnded ? s.base[k] : s.base[k] + (static_cast<double>(x) - static_cast<double>(s.top[k]));
  };
  // (the quotient, a product by the inverse with what that leaves added: equal means of
  // different lengths have one key)
  const auto key_of = [&](double score, int k) {
    const double2 p = s.power[k];
    const double q = score * p.y;
    return ordered_key(fma(fma(-q, p.x, score), p.y, q));
  };
  const auto keep = [&](float2 e, int k) {
    const int at = atomicAdd(&s.found, 1);
    if (at < kFound + kMaxBeams) {
      s.logit[at] = e.x;
      s.at[at] = k << 18 | __float_as_int(e.y);
    }
  };
  // a bound: S candidates at least are no worse
  float top = -INFINITY, unused;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = place + j * kThreads;
    if (!(held[j].x > -INFINITY)) continue;
    float off;
    const float v = approx(held[j].x, beam_of(c - over(c, by_own) * own), off);
    top = fmaxf(top, v - off);  // (NaN: none)
  }
  const int give = (S + kWarps - 1) / kWarps;
  const float nth = nth_largest(top, give, unused);  // (-inf where a warp has not that many)
  if (lane == 0) s.nth[warp] = nth;
  __syncthreads();
  float t = s.nth[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) t = fminf(t, s.nth[i]);
  if (total <= kThreads * kHeld) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int c = place + j * kThreads;
      if (!(held[j].x > -INFINITY)) continue;
      const int k = beam_of(c - over(c, by_own) * own);
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
  const auto put = [&](int rank, float score, int at) {
    const int k = at >> 18;
    const size_t o = static_cast<size_t>(b) * S + rank;
    const bool ended = s.state[k] == kEnded;
    const int token = ended ? a.end_token : at & ((1 << 18) - 1);
    a.tokens[o] = token;
    a.parents[o] = b * K + k;
    a.scores_out[o] = score;
    if (a.lengths_out) a.lengths_out[o] = s.length[k] + (ended ? 0 : 1);
    if (a.finished_out) a.finished_out[o] = ended || (a.end_token >= 0 && token == a.end_token);
  };
  const auto put_none = [&](int rank) {
    const size_t o = static_cast<size_t>(b) * S + rank;
    a.tokens[o] = a.parents[o] = -1;
    a.scores_out[o] = -INFINITY;
    if (a.lengths_out) a.lengths_out[o] = 0;
    if (a.finished_out) a.finished_out[o] = 0;
  };
  // scores and keys of the few (of all ended beams, the first), in fp64
  const int found = s.found;
  // Whether a smaller logit of a row may have the same key: the next one is at least
  // 2^-24 |x| below, and the roundings of a score and its key add up to less than 2^-50 of
  // its terms.
  bool alike = false;
  for (int i = tid; i < min(found, kFound + kMaxBeams); i += kThreads) {
    const int k = s.at[i] >> 18;
    const float x = s.logit[i];
    const double score = score_of(x, k);
    alike |= i >= s.ended && !(fabsf(x) > 0x1p-25f * (fabsf(s.approx[k].x) + fabsf(x - s.top[k])));
    s.score[i] = static_cast<float>(score);
    s.key[i] = key_of(score, k);
  }
  alike = __syncthreads_or(alike);
  if (found <= kFound + kMaxBeams) {
    for (int i = tid; i < found; i += kThreads) {
      const unsigned long long key = s.key[i];
      const int at = s.at[i];
      int rank = 0;
      if (alike) {
        const unsigned long long place = place_in_order(at, s.logit[i]);
        for (int j = 0; j < found; ++j) rank += better(s.key[j], place_in_order(s.at[j], s.logit[j]), key, place);
      } else {  // (equal keys of a row are equal logits: beam and token decide)
#pragma unroll 4
        for (int j = 0; j < found; ++j) rank += better(s.key[j], s.at[j], key, at);
      }
      if (rank < S) put(rank, s.score[i], at);
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
    unsigned long long key = 0, place = ~0ull;
    int list = -1;
    for (int q = tid; q < own; q += kThreads) {
      const int r = s.next[q];
      if (r >= S) continue;
      const float2 e = entry(q, r);
      if (!(e.x > -INFINITY)) continue;
      const int k = beam_of(q);
      const unsigned long long v = key_of(score_of(e.x, k), k), p = place_in_order(k << 18 | __float_as_int(e.y), e.x);
      if (better(v, p, key, place)) key = v, place = p, list = q;
    }
    for (int i = tid, j = 0; i < s.ended; i += kThreads, ++j) {
      const unsigned long long p = place_in_order(s.at[i], 0.0f);
      if ((ended_left >> j & 1u) && better(s.key[i], p, key, place)) key = s.key[i], place = p, list = -2 - i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, key, o), p2 = __shfl_xor_sync(0xffffffffu, place, o);
      const int l2 = __shfl_xor_sync(0xffffffffu, list, o);
      if (better(k2, p2, key, place)) key = k2, place = p2, list = l2;
    }
    if (lane == 0) s.best_key[warp] = key, s.best_place[warp] = place, s.best_list[warp] = list;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i)
      if (better(s.best_key[i], s.best_place[i], key, place)) key = s.best_key[i], place = s.best_place[i], list = s.best_list[i];
    if (list == -1) {
      if (tid == 0) put_none(rank);
    } else if (list >= 0) {
      if (tid == list % kThreads) {
        const int at = at_of(place);
        put(rank, static_cast<float>(score_of(entry(list, s.next[list]).x, at >> 18)), at);
        s.next[list] += 1;
      }
    } else if (tid == (-2 - list) % kThreads) {
      put(rank, s.score[-2 - list], at_of(place));
      ended_left &= ~(1u << ((-2 - list) / kThreads));
    }
    __syncthreads();
  }
}

}  // namespace

int beam_max_select() { return kMaxSelect; }
int beam_max_beams() { return kMaxBeams; }

namespace {

// Turns of a part of `entries` entries, which may begin inside a word, and the shared
// memory of a CTA whose parts have that many.
int turns_of(int entries, bool bf16) {
  const int each = 32 * kWords * (bf16 ? 8 : 4);
  return (entries + 7 + each - 1) / each;
}
int smem_of(int turns) { return kWarps * (static_cast<int>(sizeof(List)) + turns * 64); }

}  // namespace

// Parts of a row, of whole 512 entries: as many whole CTAs a row as leave no more than 4
// an SM, but 32 parts at most, whose lists the merge reads (V = 151936, 1 request of 32
// beams, S = 64: 22.6 us, of 64 parts 30.8, of 16 24.8; 4 of 16, S = 32: 18.5, 24.7 and
// 19.6).  4 are resident where a part's notes leave them the shared memory: up to 21 turns,
// with 8 parts 81920 fp32 or 167936 bf16 entries a row.  Beyond, 3 are, and more than 456
// CTAs take a second, short wave (64 x 8, V = 128256, fp32: 64 us, 38.8 at the copy rate).
// A row's CTAs share them evenly: one that is left with few warps has a worse bound.
void plan_beam_parts(BeamArgs& a, int sms) {
  const long long rows = static_cast<long long>(a.batch) * a.beams, fit = 4ll * sms / rows;
  const long long most = min((a.vocab + 511) / 512, kMaxParts), want = (fit > 1 ? fit : 1) * kWarps;
  const int parts = static_cast<int>(want < most ? want : most);
  a.chunk = ((a.vocab + parts - 1) / parts + 511) / 512 * 512;
  a.parts = (a.vocab + a.chunk - 1) / a.chunk;
  const int ctas = (a.parts + kWarps - 1) / kWarps;
  a.turns = turns_of(a.chunk, a.bf16);
  a.each = a.parts / ctas, a.more = a.parts % ctas;
}

int launch_beam_select(const BeamArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.batch) * a.beams;
  const long long ctas = rows * ((a.parts + kWarps - 1) / kWarps) + (a.length_penalty != 0.0f ? (rows + kThreads - 1) / kThreads : 0);
  const unsigned grid = static_cast<unsigned>(ctas);
  const int smem = smem_of(a.turns);
  static_assert(sizeof(List) % 16 == 0, "words");
  const auto kernel = a.bf16 ? beam_rows_kernel<true> : beam_rows_kernel<false>;
  // (the kernel's limit is all host threads': always that of the longest part)
  const int limit = smem_of(turns_of((1 << 18) / kWarps, a.bf16));
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess)
    return -1;
  kernel<<<grid, kThreads, smem, stream>>>(a);
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
