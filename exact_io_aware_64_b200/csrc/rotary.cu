// rotary.cu -- rotary positions of query and key heads, and their gradient.
//
// Pair k of a head's first R elements is turned by the angle t = position * inv_freq[k]:
//   y1 = m (x1 cos t - x2 sin t),  y2 = m (x2 cos t + x1 sin t),
// (x1, x2) = (x[k], x[k + R/2]) or, interleaved, (x[2k], x[2k + 1]); elements from R on are
// copied.  The map is m times a rotation, so its gradient is the same map with -t.
//
// Bound: HBM, each element read and written once.  A float32 product position * inv_freq
// is off by 2^-24 of the angle, 0.006 rad at 10^5 rad, so the angle is formed in float64,
// reduced to a fraction of a turn there, and only the fraction goes to float32 (error of
// the angle 1e-7 rad at any position).  That costs a few float64 operations and one sincospi
// per (token, pair), so it must not be repeated for every head.
//
// Vector form (R, strides and pointers allow 16-byte pieces): a thread owns one piece of a
// head row at one token, forms its 2 to 8 angles once, in registers, and turns that piece of
// every head of Q and K, four heads' loads in flight at a time (the first four while the
// angles are formed; angles shared by the block through shared memory took 32.6 us where
// these take 30.9, B=2 H=16+4 N=8192 d=128 R=64 bf16 interleaved, 168 MB at 83 % of the copy
// rate: the barrier kept the first loads back); neighbouring threads hold
// neighbouring pieces, then neighbouring tokens.  With few tokens, threads (then blocks)
// share a token's heads.  Calls that move more than kStreamBytes load and store past the L2
// (B=2 H=16+16 N=4096 d=64 float32, 134 MB: 20.7 us with, 23.8 without; N=2048 H=16+4 d=128
// bf16, 42 MB, whose output the attention can still find in the L2: 13.4 with, 12.7
// without).  Scalar form (anything else): one pair at a time, 2- or 4-byte accesses, for widths
// such as R = 60 (B=2 H=16+16 N=4096 d=64 float32: 92 us where R = 64 takes 18).
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of one block
constexpr int kUnroll = 4;      // heads whose loads a thread has in flight
constexpr long long kStreamBytes = 96ll << 20;  // in and out: about the L2's size

// cos and sin (times m) of pair k at position pos.  Both products' roundings are carried along
// (fma): at 2^40 that of the position's alone is up to 1e-4 rad.
__device__ __forceinline__ float2 angle(const RotaryArgs& a, double pos, int k) {
  constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591243e-18;  // 1 / (2 pi)
  const double inv = static_cast<double>(a.inv_freq[k]);
  const double per = inv * kTurn;
  const double per_low = fma(inv, kTurn, -per) + inv * kTurnLow;
  const double turns = pos * per;
  const double low = fma(pos, per_low, fma(pos, per, -turns));
  const float f = static_cast<float>(2.0 * (turns - rint(turns) + low));
  float s, c;
  sincospif(f, &s, &c);
  return make_float2(c * a.mscale, s * a.mscale * a.sign);
}

__device__ __forceinline__ double position(const RotaryArgs& a, int tok) {
  return a.positions != nullptr ? static_cast<double>(a.positions[tok])
                                : static_cast<double>(a.first + tok % a.N);
}

// The block's angles, [n][R/2], from flat token t0 on.
__device__ __forceinline__ void fill_angles(float2* cs, const RotaryArgs& a, long long t0, int n) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half;
    cs[i] = angle(a, position(a, static_cast<int>(t0) + t), i - t * half);
  }
  __syncthreads();
}

template <typename T>
struct Vec;  // 16 bytes of elements
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void unpack(uint4 v, float* x) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static uint4 pack(const float* x) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    return v;
  }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  __device__ static void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// One pair turned.  The roundings are spelled out so that every form of the kernel gives
// the same bits.
__device__ __forceinline__ void turn(float x1, float x2, float2 w, float& y1, float& y2) {
  y1 = fmaf(x1, w.x, -__fmul_rn(x2, w.y));
  y2 = fmaf(x2, w.x, __fmul_rn(x1, w.y));
}

template <bool kStream>
__device__ __forceinline__ uint4 get16(const void* p) {
  const uint4* q = static_cast<const uint4*>(p);
  return kStream ? __ldcs(q) : *q;
}
template <bool kStream>
__device__ __forceinline__ void put16(void* p, uint4 v) {
  uint4* q = static_cast<uint4*>(p);
  if (kStream) __stcs(q, v);
  else *q = v;
}

template <typename T, bool kInterleaved, bool kStream>
__global__ void __launch_bounds__(kThreads) rotary_vector_kernel(const RotaryArgs a) {
  grid_dependency_wait();
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  constexpr int kV = Vec<T>::n;
  constexpr int kAngles = kInterleaved ? kV / 2 : kV;
  const int half = a.R / 2;
  const int turned = kInterleaved ? a.R / kV : half / kV;  // pieces of a row: turned, copied
  const int pieces = turned + (a.copy_rest ? (a.d - a.R) / kV : 0);
  // thread = (head group, token, piece), all powers of two but the last group
  const int q = threadIdx.x & (a.lanes - 1);
  const int t = (threadIdx.x / a.lanes) & (a.tokens - 1);
  const int group = threadIdx.x / (a.lanes * a.tokens);
  const int groups = kThreads / (a.lanes * a.tokens);
  if (q >= pieces || t0 + t >= a.total) return;
  const int tok = static_cast<int>(t0) + t;
  const bool turns = q < turned;
  const int e1 = turns ? q * kV : a.R + (q - turned) * kV;
  const long long b = tok / a.N, n = tok - b * a.N;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int h1 = min(h0 + a.heads_per_block, a.x[0].heads + a.x[1].heads);
  const int nq = a.x[0].heads;
  const T* src0 = static_cast<const T*>(a.x[0].in) + (b * a.x[0].in_b + n * a.x[0].in_n + e1);
  const T* src1 = static_cast<const T*>(a.x[1].in) + (b * a.x[1].in_b + n * a.x[1].in_n + e1);
  T* dst0 = static_cast<T*>(a.x[0].out) + (b * a.x[0].out_b + n * a.x[0].out_n + e1);
  T* dst1 = static_cast<T*>(a.x[1].out) + (b * a.x[1].out_b + n * a.x[1].out_n + e1);
  uint4 r1[kUnroll], r2[kUnroll];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * groups;
      if (h >= h1) break;
      const T* p = h < nq ? src0 + h * a.x[0].in_h : src1 + (h - nq) * a.x[1].in_h;
      r1[u] = get16<kStream>(p);
      if (!kInterleaved && turns) r2[u] = get16<kStream>(p + half);
    }
  };
  // the first heads' loads are on their way while the angles are formed
  load(h0 + group);
  float2 w[kAngles];
  if (turns) {
    const double pos = position(a, tok);
#pragma unroll
    for (int k = 0; k < kAngles; ++k) w[k] = angle(a, pos, q * kAngles + k);
  }
  for (int hb = h0 + group; hb < h1; hb += groups * kUnroll) {
    if (hb != h0 + group) load(hb);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * groups;
      if (h >= h1) break;
      T* p = h < nq ? dst0 + h * a.x[0].out_h : dst1 + (h - nq) * a.x[1].out_h;
      if (turns) {
        float x1[kV];
        Vec<T>::unpack(r1[u], x1);
        if constexpr (kInterleaved) {
#pragma unroll
          for (int k = 0; k < kAngles; ++k)
            turn(x1[2 * k], x1[2 * k + 1], w[k], x1[2 * k], x1[2 * k + 1]);
        } else {
          float x2[kV];
          Vec<T>::unpack(r2[u], x2);
#pragma unroll
          for (int k = 0; k < kAngles; ++k) turn(x1[k], x2[k], w[k], x1[k], x2[k]);
          put16<kStream>(p + half, Vec<T>::pack(x2));
        }
        r1[u] = Vec<T>::pack(x1);
      }
      put16<kStream>(p, r1[u]);
    }
  }
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_scalar_kernel(const RotaryArgs a) {
  extern __shared__ __align__(16) float2 cs[];
  grid_dependency_wait();
  const int half = a.R / 2;
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int n = static_cast<int>(min(static_cast<long long>(a.tokens), a.total - t0));
  fill_angles(cs, a, t0, n);
  const int h0 = blockIdx.y * a.heads_per_block;
  const int hn = min(a.heads_per_block, a.x[0].heads + a.x[1].heads - h0);
  const int per_row = half + (a.copy_rest ? a.d - a.R : 0);  // pairs, then copied elements
  const int work = n * hn * per_row;
  for (int i = threadIdx.x; i < work; i += kThreads) {
    const int row = i / per_row, q = i - row * per_row;
    const int hh = row / n, t = row - hh * n;  // tokens of one head follow one another
    int h = h0 + hh;
    const int which = h >= a.x[0].heads;
    const RotaryTensor& x = a.x[which];
    if (which) h -= a.x[0].heads;
    const int tok = static_cast<int>(t0) + t;
    const long long b = tok / a.N, nn = tok - b * a.N;
    const T* src = static_cast<const T*>(x.in) + (b * x.in_b + h * x.in_h + nn * x.in_n);
    T* dst = static_cast<T*>(x.out) + (b * x.out_b + h * x.out_h + nn * x.out_n);
    if (q >= half) {
      dst[a.R + q - half] = src[a.R + q - half];
    } else {
      const int e1 = kInterleaved ? 2 * q : q, e2 = kInterleaved ? 2 * q + 1 : q + half;
      float y1, y2;
      turn(to_f(src[e1]), to_f(src[e2]), cs[t * half + q], y1, y2);
      put(dst + e1, y1);
      put(dst + e2, y2);
    }
  }
}

template <typename T>
cudaError_t launch_t(const RotaryArgs& args, bool vector, int num_sms, cudaStream_t stream) {
  RotaryArgs a = args;
  const int heads = a.x[0].heads + a.x[1].heads;
  int tokens = kMaxTokens;
  if (vector) {
    constexpr int kV = Vec<T>::n;
    const int pieces = (a.interleaved ? a.R / kV : a.R / 2 / kV) +
                       (a.copy_rest ? (a.d - a.R) / kV : 0);
    a.lanes = 1;  // at most 128: d <= 512 float32 elements
    while (a.lanes < pieces) a.lanes *= 2;
    while (tokens * a.lanes > kThreads) tokens /= 2;
  }
  // with few tokens a block takes fewer of them, so that more blocks share the work
  while (tokens > 1 && a.total / tokens < 4ll * num_sms) tokens /= 2;
  a.tokens = tokens;
  const long long bx = (a.total + tokens - 1) / tokens;
  // blocks that share a token's heads, while a block still has a head for each group
  const int groups = vector ? kThreads / (a.lanes * tokens) : 1;
  int split = 1;
  while (split * groups < heads && bx * split < 2ll * num_sms) ++split;
  a.heads_per_block = (heads + split - 1) / split;
  split = (heads + a.heads_per_block - 1) / a.heads_per_block;
  if (split > 65535) {
    a.heads_per_block = (heads + 65534) / 65535;
    split = (heads + a.heads_per_block - 1) / a.heads_per_block;
  }
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(split));
  const size_t smem = vector ? 0 : static_cast<size_t>(tokens) * (a.R / 2) * sizeof(float2);
  const bool stream_out = 2 * a.total * heads * a.d * static_cast<long long>(sizeof(T)) > kStreamBytes;
  void (*kernel)(RotaryArgs) =
      !vector ? (a.interleaved ? rotary_scalar_kernel<T, true> : rotary_scalar_kernel<T, false>)
      : stream_out ? (a.interleaved ? rotary_vector_kernel<T, true, true> : rotary_vector_kernel<T, false, true>)
                   : (a.interleaved ? rotary_vector_kernel<T, true, false> : rotary_vector_kernel<T, false, false>);
  return launch_early(kernel, grid, kThreads, smem, stream, true, a);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int elem_bytes, int num_sms, cudaStream_t stream) {
  // 16-byte pieces: the turned part (each half of it), the row starts and the pointers
  const int v = 16 / elem_bytes;
  const int unit = a.interleaved ? v : 2 * v;
  bool vector = a.R % unit == 0 && a.d % v == 0;
  for (const RotaryTensor& x : a.x) {
    if (x.heads == 0) continue;
    const long long strides[6] = {x.in_b, x.in_h, x.in_n, x.out_b, x.out_h, x.out_n};
    for (const long long s : strides) vector = vector && s % v == 0;
    vector = vector && ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15u) == 0;
  }
  return elem_bytes == 2 ? launch_t<__nv_bfloat16>(a, vector, num_sms, stream)
                         : launch_t<float>(a, vector, num_sms, stream);
}

}  // namespace fa
