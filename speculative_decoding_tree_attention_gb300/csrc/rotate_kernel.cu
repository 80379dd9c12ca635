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
// of 4) value by value.  Sine and cosine of a lane's pairs are computed once for
// all heads that a warp takes of a token.  Bound: HBM, one read and one write of
// each row; latency for single tokens.
#include "tv_device.cuh"
#include "tv_launch.h"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum Layout { kHalves, kNeighbours, kHalvesByValue };

struct Angles {
  uint64_t turn[kMaxPairs];  // f / 2 pi, a fraction of 2^64
  float scale[kMaxPairs];    // of sine and cosine; NaN where f is not finite
  uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_of(uint16_t w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }

__device__ void fill_angles(const RotateArgs& a, Angles& s) {
  const int i = threadIdx.x;
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
  // value j of the first and of the second of the pairs
  __device__ __forceinline__ void values(float (&x)[4], float (&y)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (L == kHalves) {
        x[j] = j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        y[j] = j % 2 ? bf16_hi(w[2 + j / 2]) : bf16_lo(w[2 + j / 2]);
      } else {
        x[j] = bf16_lo(w[j]);
        y[j] = bf16_hi(w[j]);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[4], const float (&y)[4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (L == kHalves) {
        w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
        w[2 + j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
      } else {
        w[2 * j] = pack_bf16x2(x[2 * j], y[2 * j]);
        w[2 * j + 1] = pack_bf16x2(x[2 * j + 1], y[2 * j + 1]);
      }
    }
  }
};

// A lane's weights of its values.
template <int D, Layout L>
__device__ __forceinline__ void load_weights(const void* w, bool fp32, int sub, int rot, float (&x)[4], float (&y)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = y[j] = 1.0f;
    if (!w) continue;
    const int p = pair_of<D, L>(sub, j);
    int i = first_of<D, L>(p, rot), k = second_of<D, L>(p, rot);
    if (L == kHalves && 8 * sub >= rot) i = 8 * sub + j, k = 8 * sub + 4 + j;
    x[j] = fp32 ? static_cast<const float*>(w)[i] : bf16_of(static_cast<const uint16_t*>(w)[i]);
    y[j] = fp32 ? static_cast<const float*>(w)[k] : bf16_of(static_cast<const uint16_t*>(w)[k]);
  }
}

template <int D, Layout L>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  constexpr int kUnroll = 4;
  __shared__ Angles s;
  fill_angles(a, s);
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const int rot = a.rotary_dim;
  float qx[4], qy[4], kx[4], ky[4];
  load_weights<D, L>(a.q_weight, a.weight_fp32, sub, rot, qx, qy);
  load_weights<D, L>(a.k_weight, a.weight_fp32, sub, rot, kx, ky);
  __syncthreads();
  const int heads = a.hq + a.hkv;
  const int each = ((heads + kRows - 1) / kRows + a.items - 1) / a.items * kRows;  // heads of an item
  const long long all = static_cast<long long>(a.tokens) * a.items;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < all;
       it += static_cast<long long>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(it / a.items);
    const int h0 = static_cast<int>(it - static_cast<long long>(t) * a.items) * each;
    const int h1 = min(h0 + each, heads);
    float c[4], n[4];
    bool turned[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = pair_of<D, L>(sub, j);
      turned[j] = 2 * p < rot;
      c[j] = n[j] = 0.0f;
      if (turned[j]) {
        const long long pos = a.positions[static_cast<size_t>(s.axis[p]) * a.tokens + t];
        const uint64_t phase = s.turn[p] * static_cast<uint64_t>(pos);
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &n[j], &c[j]);
        c[j] *= s.scale[p];
        n[j] *= s.scale[p];
      }
    }
    for (int g = h0; g < h1; g += kRows * kUnroll) {  // (uniform over the warp)
      Row<D, L> r[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = g + u * kRows + lane / kLanes;
        if (h < h1) {
          r[u].load(h < a.hq ? a.q + t * a.q_stride + static_cast<size_t>(h) * D
                             : a.k + t * a.k_stride + static_cast<size_t>(h - a.hq) * D, sub, rot);
        } else {
          r[u].w[0] = r[u].w[1] = r[u].w[2] = r[u].w[3] = 0;
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = g + u * kRows + lane / kLanes;
        const bool q = h < a.hq;
        float x[4], y[4];
        r[u].values(x, y);
        if (a.q_weight || a.k_weight) {
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) sum = fmaf(x[j], x[j], fmaf(y[j], y[j], sum));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (q ? a.q_weight : a.k_weight) {
            const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[j] = x[j] * inv * (q ? qx[j] : kx[j]);
              y[j] = y[j] * inv * (q ? qy[j] : ky[j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float b = x[j] * c[j] - y[j] * n[j], d = x[j] * n[j] + y[j] * c[j];
          if (turned[j]) x[j] = b, y[j] = d;
        }
        r[u].set(x, y);
        if (h < h1)
          r[u].store(q ? a.q_out + t * a.q_out_stride + static_cast<size_t>(h) * D
                       : a.k_out + t * a.k_out_stride + static_cast<size_t>(h - a.hq) * D, sub, rot);
      }
    }
  }
}

template <int D>
void launch_rotate_d(const RotateArgs& a, int grid, cudaStream_t stream) {
  if (a.interleaved) {
    rotate_kernel<D, kNeighbours><<<grid, kThreads, 0, stream>>>(a);
  } else if (a.rotary_dim % 8 == 0) {
    rotate_kernel<D, kHalves><<<grid, kThreads, 0, stream>>>(a);
  } else {
    rotate_kernel<D, kHalvesByValue><<<grid, kThreads, 0, stream>>>(a);
  }
}

}  // namespace

int launch_rotate(RotateArgs a, int sms, cudaStream_t stream) {
  // Warps that share a token: enough that every SM has 32 of them four times
  // over, at most one for each group of heads that a warp takes at once.
  const long long want = 128ll * sms;
  const int rows = 256 / a.head_dim, groups = (a.hq + a.hkv + rows - 1) / rows;
  const long long share = (want + a.tokens - 1) / a.tokens;
  a.items = static_cast<int>(share < groups ? share : groups);
  const long long ctas = (static_cast<long long>(a.tokens) * a.items + kWarps - 1) / kWarps, most = 4ll * sms;
  const int grid = static_cast<int>(ctas < most ? ctas : most);
  if (a.head_dim == 128) {
    launch_rotate_d<128>(a, grid, stream);
  } else {
    launch_rotate_d<64>(a, grid, stream);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tv
