// rotate_kernel.cu -- the norm of every query and key head and its rotation by
// the token's position, in one pass ahead of the cache writes and attentions.
//
// A head x of D values, with weights w given, first becomes
//   y = x / sqrt(mean(x^2) + eps) * w,
// then its pair i < R/2, values (a, b), turns by theta = pos f_i, pos the token's
// position on the pair's axis (time, height, width: images and video have
// several):
//   (a, b) -> scale (a cos theta - b sin theta, a sin theta + b cos theta).
// All in fp32, rounded once to bf16.
//
// Angles: of a far position the angle itself does not fit 24 bits, but only its
// fraction of a turn matters.  f_i / 2 pi is held as a 64-bit fraction of a turn
// (fp64 product with the product's own rounding error added), so that pos times
// it modulo 2^64 is the fraction, off by at most |pos| 2^-64 turns, in two integer
// products; its upper 32 bits, as half-turns in [-1, 1), go to sincospif.
//
// A row is taken by D / 8 lanes that hold four pairs each, so that both values of
// a pair are in one lane: pairs (i, i + R/2) as 8 bytes of each half, pairs
// (2i, 2i+1) as 16 bytes; halves that are not 8 bytes aligned (R / 2 no multiple
// of 4) value by value.  Sine and cosine of a token's pairs are computed once per warp,
// a lane a pair, and joined with the weights: with A = w_a cos, B = w_b sin, C = w_a
// sin, D = w_b cos a pair costs two products, two fused ones and two products by the
// root, two values an instruction.
//
// Two kernels.  Few rows: a warp takes a token's heads or a share of them, three rows a
// lane in flight, the first while the angles are computed.  Many rows: a warp takes a
// stretch of rows over several tokens, which come to shared memory two batches of eight
// rows ahead (cp.async: no registers).
//
// Bound: HBM, one read and one write of each row; latency for single tokens.
// Measured (device time, the call replayed, norms): 8192 tokens of 64/8 heads of 128
// 49.7 us (6.1 TB/s, 0.90 of the copy rate), 4 x 1600 of 28/4 on three axes 20.5, 16
// tokens of 32/8 heads 4.2.  Before: with sines by every lane for its own pairs and
// norm, weights and rotation one after the other 80 us for the first; the kernel of few
// rows 57, with two or four rows in flight 60 and 57; stretches in batches of 6 rows 4
// CTAs an SM 50.3, of 2 rows and 8 stages 70.  Other forms of the first: neighbours 49.6,
// half of each head turned 53.8 (neighbours 51.2), 124 of 128 values, whose halves are not
// 8 bytes aligned, 72.9.  Held to 64 and 80 registers, ten of the twenty instances spill 4 to
// 24 bytes (of the kernel of many rows only those by value, 8).
#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum Layout { kHalves, kNeighbours, kHalvesByValue };

struct Shared {
  uint64_t turn[kMaxPairs];  // f / 2 pi, a fraction of 2^64
  float scale[kMaxPairs];    // of sine and cosine; NaN where f is not finite
  uint8_t axis[kMaxPairs];
  float weight[2][2 * kMaxPairs];          // of queries and keys
  float2 angle[kWarps][kMaxPairs];         // of a warp's token: cosine and sine
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_of(uint16_t w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }

__device__ void fill_shared(const RotateArgs& a, Shared& s) {
  const int i = threadIdx.x;
  if (i >= kThreads - 2 * kMaxPairs) {  // (the other half of the threads)
    const int d = i - (kThreads - 2 * kMaxPairs);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const void* w = k ? a.k_weight : a.q_weight;
      float v = 1.0f;
      if (w && d < a.head_dim)
        v = a.weight_fp32 ? static_cast<const float*>(w)[d] : bf16_of(static_cast<const uint16_t*>(w)[d]);
      s.weight[k][d] = v;
    }
  }
  if (i < a.rotary_dim / 2) {
    const double f = a.frequencies[i];
    const double inverse = 0.15915494309189535, rest = -9.839338337591243e-18;  // 1 / 2 pi
    const double p = f * inverse;
    const double e = fma(f, inverse, -p) + f * rest;
    // both parts as whole multiples of 2^-64 turns; whole turns drop out
    const double whole = rint(p);
    s.turn[i] = static_cast<uint64_t>(__double2ll_rn((p - whole) * 0x1p64)) +
                static_cast<uint64_t>(__double2ll_rn((e - rint(e)) * 0x1p64));
    s.scale[i] = isfinite(f) ? a.scale : __int_as_float(0x7fc00000);
    s.axis[i] = a.axis[i];
  }
}

// The four pairs of a lane: a pair's number, and where its values are.
template <int D, Layout L>
__device__ __forceinline__ int pair_of(int sub, int j) {
  return L == kHalvesByValue ? sub + D / 8 * j : 4 * sub + j;
}
// (by value, and past the turned ones: neighbours)
template <int D, Layout L>
__device__ __forceinline__ int first_of(int pair, int rot) {
  return L == kNeighbours || 2 * pair >= rot ? 2 * pair : pair;
}
template <int D, Layout L>
__device__ __forceinline__ int second_of(int pair, int rot) {
  return L == kNeighbours || 2 * pair >= rot ? 2 * pair + 1 : pair + rot / 2;
}

template <int D, Layout L>
struct Row {
  uint32_t w[4];
  // kHalves: two pairs of values of the first half, two of the second (of a lane
  // past the turned ones: 8 values in a row)
  __device__ __forceinline__ void load(const uint16_t* row, int sub, int rot) {
    if (L == kHalves) {
      const bool turned = 8 * sub < rot;
      const uint2 x = *reinterpret_cast<const uint2*>(row + (turned ? 4 * sub : 8 * sub));
      const uint2 y = *reinterpret_cast<const uint2*>(row + (turned ? 4 * sub + rot / 2 : 8 * sub + 4));
      w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
    } else if (L == kNeighbours) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + 8 * sub);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = pair_of<D, L>(sub, j);
        w[j] = row[first_of<D, L>(p, rot)] | static_cast<uint32_t>(row[second_of<D, L>(p, rot)]) << 16;
      }
    }
  }
  __device__ __forceinline__ void store(uint16_t* row, int sub, int rot) const {
    if (L == kHalves) {
      const bool turned = 8 * sub < rot;
      *reinterpret_cast<uint2*>(row + (turned ? 4 * sub : 8 * sub)) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + (turned ? 4 * sub + rot / 2 : 8 * sub + 4)) = make_uint2(w[2], w[3]);
    } else if (L == kNeighbours) {
      *reinterpret_cast<uint4*>(row + 8 * sub) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = pair_of<D, L>(sub, j);
        row[first_of<D, L>(p, rot)] = static_cast<uint16_t>(w[j]);
        row[second_of<D, L>(p, rot)] = static_cast<uint16_t>(w[j] >> 16);
      }
    }
  }
  // the pairs' first and second values, two by two
  __device__ __forceinline__ void values(float2 (&x)[2], float2 (&y)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (L == kHalves) {
        x[j] = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
        y[j] = make_float2(bf16_lo(w[2 + j]), bf16_hi(w[2 + j]));
      } else {
        x[j] = make_float2(bf16_lo(w[2 * j]), bf16_lo(w[2 * j + 1]));
        y[j] = make_float2(bf16_hi(w[2 * j]), bf16_hi(w[2 * j + 1]));
      }
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[2], const float2 (&y)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (L == kHalves) {
        w[j] = pack_bf16x2(x[j].x, x[j].y);
        w[2 + j] = pack_bf16x2(y[j].x, y[j].y);
      } else {
        w[2 * j] = pack_bf16x2(x[j].x, y[j].x);
        w[2 * j + 1] = pack_bf16x2(x[j].y, y[j].y);
      }
    }
  }
};

// Cosine and sine of the pairs of a warp's token, a lane a pair.
__device__ __forceinline__ void fill_angles(Shared& s, const int (&pos)[kMaxAxes], int rot) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = lane + 32 * i;
    if (2 * p < rot) {
      const int axis = s.axis[p];
      const int at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
      const uint64_t phase = s.turn[p] * static_cast<uint64_t>(static_cast<long long>(at));
      float c, n;
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &n, &c);
      s.angle[warp][p] = make_float2(c * s.scale[p], n * s.scale[p]);
    }
  }
  __syncwarp();
}

// What a lane turns its pairs by (a pair that is not turned: its weights alone).
struct Turn {
  float2 a[2], b[2], c[2], d[2];  // (b: with the other sign)
};
template <int D, Layout L, bool ALL>
__device__ __forceinline__ void fill_turn(const Shared& s, int key, int sub, int rot, Turn& r) {
  const float2* angle = s.angle[threadIdx.x >> 5];
  const float* weight = s.weight[key];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = pair_of<D, L>(sub, j);
    const bool turned = ALL || 2 * p < rot;
    const bool run = L == kHalves && !turned;  // (eight values in a row)
    const float wx = weight[run ? 8 * sub + j : first_of<D, L>(p, rot)];
    const float wy = weight[run ? 8 * sub + 4 + j : second_of<D, L>(p, rot)];
    const float2 cs = turned ? angle[p] : make_float2(1.0f, 0.0f);
    (j % 2 ? r.a[j / 2].y : r.a[j / 2].x) = wx * cs.x;
    (j % 2 ? r.b[j / 2].y : r.b[j / 2].x) = -wy * cs.y;
    (j % 2 ? r.c[j / 2].y : r.c[j / 2].x) = wx * cs.y;
    (j % 2 ? r.d[j / 2].y : r.d[j / 2].x) = wy * cs.x;
  }
}

// A row normalised and turned.
template <int D, Layout L, bool ALL>
__device__ __forceinline__ void turn_row(Row<D, L>& r, const Turn& turn, bool norm, float eps, int sub, int rot) {
  constexpr int kLanes = D / 8;
  float2 x[2], y[2];
  r.values(x, y);
  float inv = 1.0f;
  if (norm) {
    const float2 two = fma2(x[0], x[0], fma2(x[1], x[1], fma2(y[0], y[0], mul2(y[1], y[1]))));
    float sum = two.x + two.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = rsqrtf(fmaf(sum, 1.0f / D, eps));
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 n = make_float2(inv, inv);
    const float2 b = mul2(n, fma2(x[j], turn.a[j], mul2(y[j], turn.b[j])));
    const float2 d = mul2(n, fma2(y[j], turn.d[j], mul2(x[j], turn.c[j])));
    if (ALL) {
      x[j] = b, y[j] = d;
    } else {  // (a value that is not turned is none of its neighbour's business, infinite or not)
      const int p = pair_of<D, L>(sub, 2 * j), q = pair_of<D, L>(sub, 2 * j + 1);
      x[j].x = 2 * p < rot ? b.x : x[j].x * turn.a[j].x * inv;
      y[j].x = 2 * p < rot ? d.x : y[j].x * turn.d[j].x * inv;
      x[j].y = 2 * q < rot ? b.y : x[j].y * turn.a[j].y * inv;
      y[j].y = 2 * q < rot ? d.y : y[j].y * turn.d[j].y * inv;
    }
  }
  r.set(x, y);
}

// ALL: every value of a head is turned.
template <int D, Layout L, bool ALL>
__global__ void __launch_bounds__(kThreads, 4) rotate_kernel(const RotateArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows that a warp takes at once
  constexpr int kUnroll = 3;  // rows of a lane in flight
  __shared__ Shared s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
  const int rot = a.rotary_dim;
  const long long it = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(it / a.items);
  const bool here = t < a.tokens;
  // steps of kRows heads, of the queries and then of the keys; this warp's share
  const int q_steps = (a.hq + kRows - 1) / kRows, steps = q_steps + (a.hkv + kRows - 1) / kRows;
  const int each = (steps + a.items - 1) / a.items;
  const int g0 = static_cast<int>(it - static_cast<long long>(t) * a.items) * each, g1 = here ? min(g0 + each, steps) : g0;
  Row<D, L> r[kUnroll];
  // rows of step g on, of queries or keys
  const auto load = [&](int g, int end, bool key) {
    const int heads = key ? a.hkv : a.hq, h0 = (key ? g - q_steps : g) * kRows + lane / kLanes;
    const uint16_t* in = (key ? a.k + t * a.k_stride : a.q + t * a.q_stride) + static_cast<size_t>(h0) * D;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (g + u < end && h0 + u * kRows < heads) {
        r[u].load(in + u * kRows * D, sub, rot);
      } else {
        r[u].w[0] = r[u].w[1] = r[u].w[2] = r[u].w[3] = 0;
      }
    }
  };
  int pos[kMaxAxes];  // the token's position on every axis
#pragma unroll
  for (int i = 0; i < kMaxAxes; ++i)
    pos[i] = here && rot > 0 && i < a.axes ? a.positions[static_cast<size_t>(i) * a.tokens + t] : 0;
  if (g0 < g1) load(g0, g0 < q_steps ? min(g1, q_steps) : g1, g0 >= q_steps);
  fill_shared(a, s);
  __syncthreads();
  if (g0 >= g1) return;
  fill_angles(s, pos, rot);
#pragma unroll 1
  for (int key = 0; key < 2; ++key) {
    const int from = key ? max(g0, q_steps) : g0, to = key ? g1 : min(g1, q_steps);
    if (from >= to) continue;
    const bool norm = (key ? a.k_weight : a.q_weight) != nullptr;
    const int heads = key ? a.hkv : a.hq;
    Turn turn;
    fill_turn<D, L, ALL>(s, key, sub, rot, turn);
    for (int g = from; g < to; g += kUnroll) {
      if (g != g0) load(g, to, key);
      const int h0 = (key ? g - q_steps : g) * kRows + lane / kLanes;
      uint16_t* out = (key ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride) + static_cast<size_t>(h0) * D;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (g + u >= to) break;  // (uniform over the warp)
        turn_row<D, L, ALL>(r[u], turn, norm, a.eps, sub, rot);
        if (h0 + u * kRows < heads) r[u].store(out + u * kRows * D, sub, rot);
      }
    }
  }
}

// The same of many rows: a warp takes a stretch of all tokens' steps, in batches of one
// token's queries or keys, which come to shared memory while the ones before are turned.
constexpr int kBatch = 4, kStages = 3, kResident = 3;
constexpr int kRing = kWarps * kStages * kBatch * 512;  // bytes
template <int D, Layout L, bool ALL>
__global__ void __launch_bounds__(kThreads, kResident) rotate_stream_kernel(const RotateArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  __shared__ Shared s;
  extern __shared__ __align__(16) uint4 ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
  const int rot = a.rotary_dim;
  uint4* mine = ring + warp * (kStages * kBatch * 32);
  const int q_steps = (a.hq + kRows - 1) / kRows, steps = q_steps + (a.hkv + kRows - 1) / kRows;
  const long long begin = (static_cast<long long>(blockIdx.x) * kWarps + warp) * a.each;
  const long long rest = static_cast<long long>(a.tokens) * steps - begin;
  int left = rest > a.each ? a.each : rest > 0 ? static_cast<int>(rest) : 0;  // steps of the stretch
  int t = static_cast<int>(begin / steps), g = static_cast<int>(begin % steps);  // the next one's token and place
  // steps of the next batch
  const auto batch = [&](int g, int left) { return min(kBatch, min(left, (g < q_steps ? q_steps : steps) - g)); };
  int l_left = left, l_t = t, l_g = g;  // of the loads
  const auto fetch = [&](int stage) {
    if (l_left > 0) {
      const bool key = l_g >= q_steps;
      const int heads = key ? a.hkv : a.hq, h0 = (key ? l_g - q_steps : l_g) * kRows + lane / kLanes;
      const int n = batch(l_g, l_left);
      const uint16_t* in = (key ? a.k + l_t * a.k_stride : a.q + l_t * a.q_stride) + static_cast<size_t>(h0) * D + 8 * sub;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u < n && h0 + u * kRows < heads) cpa16(mine + (stage * kBatch + u) * 32 + lane, in + u * kRows * D);
      l_left -= n;
      l_g += n;
      if (l_g == steps) l_g = 0, ++l_t;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  int pos[kMaxAxes];  // the next token's position on every axis
  const auto place = [&](int token) {
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i)
      pos[i] = token < a.tokens && rot > 0 && i < a.axes ? a.positions[static_cast<size_t>(i) * a.tokens + token] : 0;
  };
  place(left > 0 ? t : a.tokens);
  fill_shared(a, s);
  __syncthreads();
  Turn turn;
  int stage = 0, ahead = kStages - 1;
  for (bool first = true; left > 0; first = false) {
    fetch(ahead);
    ahead = ahead + 1 == kStages ? 0 : ahead + 1;
    const bool key = g >= q_steps;
    if (first || g == 0) {
      fill_angles(s, pos, rot);
      place(t + 1);
    }
    if (first || g == 0 || g == q_steps) fill_turn<D, L, ALL>(s, key, sub, rot, turn);
    const bool norm = (key ? a.k_weight : a.q_weight) != nullptr;
    const int heads = key ? a.hkv : a.hq, h0 = (key ? g - q_steps : g) * kRows + lane / kLanes;
    const int n = batch(g, left);
    uint16_t* out = (key ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride) + static_cast<size_t>(h0) * D;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint16_t* row = reinterpret_cast<const uint16_t*>(mine + stage * kBatch * 32 + (lane - sub));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= n) break;  // (uniform over the warp)
      Row<D, L> r;
      r.load(row + u * 256, sub, rot);
      turn_row<D, L, ALL>(r, turn, norm, a.eps, sub, rot);
      if (h0 + u * kRows < heads) r.store(out + u * kRows * D, sub, rot);
    }
    __syncwarp();
    stage = stage + 1 == kStages ? 0 : stage + 1;
    left -= n;
    g += n;
    if (g == steps) g = 0, ++t;
  }
}

template <int D, Layout L, bool ALL>
int start(const RotateArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.each == 0) {
    rotate_kernel<D, L, ALL><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (cudaFuncSetAttribute(rotate_stream_kernel<D, L, ALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing) != cudaSuccess)
      return -1;
    rotate_stream_kernel<D, L, ALL><<<grid, kThreads, kRing, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int D, Layout L>
int launch_rotate_l(const RotateArgs& a, unsigned grid, cudaStream_t stream) {
  return a.rotary_dim == D ? start<D, L, true>(a, grid, stream) : start<D, L, false>(a, grid, stream);
}

template <int D>
int launch_rotate_d(const RotateArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.interleaved) return launch_rotate_l<D, kNeighbours>(a, grid, stream);
  if (a.rotary_dim % 8 == 0) return launch_rotate_l<D, kHalves>(a, grid, stream);
  return start<D, kHalvesByValue, false>(a, grid, stream);
}

}  // namespace

int launch_rotate(RotateArgs a, int sms, cudaStream_t stream) {
  const int rows = 256 / a.head_dim, steps = (a.hq + rows - 1) / rows + (a.hkv + rows - 1) / rows;
  const long long all = static_cast<long long>(a.tokens) * steps, resident = static_cast<long long>(sms) * kResident * kWarps;
  long long ctas;
  if (all < 8 * resident) {
    // Few rows (up to some 900 tokens of 64/8 heads), where the first loads count most:
    // warps that share a token, enough for about eight CTAs on every SM, of four steps
    // of heads each at least, which are on their way together; with few tokens of one.
    // (1000 tokens of 28/4: 7.2 us, as a stretch for each warp 8.2; 1024 of 64/8, 10
    // steps a warp: 11.4 and 10.3.)
    const long long share = (8ll * kWarps * sms + a.tokens - 1) / a.tokens;
    const int most = (steps + 3) / 4;
    a.items = static_cast<int>(share < most ? share : static_cast<long long>(a.tokens) * most < 4ll * sms ? steps : most);
    ctas = (static_cast<long long>(a.tokens) * a.items + kWarps - 1) / kWarps;
  } else if (all < 48 * resident) {
    // One wave of CTAs, a stretch each: angles of as few tokens as can be (2048 tokens of
    // 64/8 heads 14.4 us, in stretches of 18 steps 17.5; 6400 of 28/4 20.5 and 22.6).
    a.each = static_cast<int>((all + resident - 1) / resident);
    ctas = (all + static_cast<long long>(a.each) * kWarps - 1) / (static_cast<long long>(a.each) * kWarps);
  } else {
    // More than L2 holds: CTAs of short stretches, about 18 steps and whole parts or
    // whole numbers of tokens, handed out in order, so that what is read and written at
    // a time lies together (8192 tokens of 64/8 heads 50.2 us, in one wave 57.6; 16384
    // 93.1 and 112.7; 25600 of 28/4 72.8 and 81.0).
    const int parts = (steps + 9) / 18;
    a.each = parts > 1 ? (steps + parts - 1) / parts : steps >= 18 ? steps : 18 / steps * steps;
    ctas = (all + static_cast<long long>(a.each) * kWarps - 1) / (static_cast<long long>(a.each) * kWarps);
  }
  if (ctas > 0x7fffffffll) return -1;
  const unsigned grid = static_cast<unsigned>(ctas);
  return a.head_dim == 128 ? launch_rotate_d<128>(a, grid, stream) : launch_rotate_d<64>(a, grid, stream);
}

}  // namespace tv
