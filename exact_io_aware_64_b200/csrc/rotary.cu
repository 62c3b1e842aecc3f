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
// the angle 4e-7 rad).  That costs a few float64 operations and one sincospi per (token,
// pair), so it is done once per block for kTokens tokens, kept in shared memory, and used
// by every head of Q and K that the block turns; heads are dealt to the grid's y extent
// when there are too few tokens to fill the GPU.
//
// A thread turns 16 bytes of elements at a time (both halves: two 16-byte loads) where
// R and every stride and pointer allow it, and one pair at a time otherwise.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;

// cos and sin (times m) of every pair of `n` tokens from token t0 of the flat [B*N] list
__device__ __forceinline__ void fill_angles(float2* cs, const RotaryArgs& a, long long t0, int n) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, k = i - t * half;
    const long long tok = t0 + t;
    const double pos = a.positions != nullptr ? static_cast<double>(a.positions[tok])
                                              : static_cast<double>(a.first + tok % a.N);
    const double turns = pos * (static_cast<double>(a.inv_freq[k]) * 0.15915494309189533577);
    const float f = static_cast<float>(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(f, &s, &c);
    cs[i] = make_float2(c * a.mscale, s * a.mscale * a.sign);
  }
}

template <typename T>
struct Vec;  // 16 bytes of elements as floats
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void load(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float* x) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = v;
  }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  __device__ static void load(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  __device__ static void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
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

// Element offset of (token, head) in a tensor of the given strides.
__device__ __forceinline__ long long row_at(const RotaryTensor& x, long long b, long long n,
                                            int h, bool out) {
  return out ? b * x.out_b + h * x.out_h + n * x.out_n : b * x.in_b + h * x.in_h + n * x.in_n;
}

template <typename T, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  extern __shared__ float2 cs[];
  const int half = a.R / 2;
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int n = static_cast<int>(min(static_cast<long long>(a.tokens), a.total - t0));
  fill_angles(cs, a, t0, n);
  __syncthreads();
  const int heads = a.x[0].heads + a.x[1].heads;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int hn = min(a.heads_per_block, heads - h0);
  // pieces of one row: the turned part, then the copied part
  constexpr int kV = kVector ? Vec<T>::n : 1;
  const int turned = kVector ? (kInterleaved ? a.R / kV : half / kV) : half;
  const int copied = a.copy_rest ? (a.d - a.R) / kV : 0;
  const int per_row = turned + copied;
  const int work = n * hn * per_row;
  for (int i = threadIdx.x; i < work; i += kThreads) {
    const int row = i / per_row, q = i - row * per_row;
    const int hh = row / n, t = row - hh * n;  // tokens of one head follow one another
    int h = h0 + hh;
    const int which = h >= a.x[0].heads;
    const RotaryTensor& x = a.x[which];
    if (which) h -= a.x[0].heads;
    const long long tok = t0 + t, b = tok / a.N, nn = tok - b * a.N;
    const T* src = static_cast<const T*>(x.in) + row_at(x, b, nn, h, false);
    T* dst = static_cast<T*>(x.out) + row_at(x, b, nn, h, true);
    const float2* ang = cs + t * half;
    if (q >= turned) {
      const int e = a.R + (q - turned) * kV;
      if constexpr (kVector) {
        *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(src + e);
      } else {
        dst[e] = src[e];
      }
    } else if constexpr (!kVector) {
      const int e1 = kInterleaved ? 2 * q : q, e2 = kInterleaved ? 2 * q + 1 : q + half;
      const float x1 = to_f(src[e1]), x2 = to_f(src[e2]);
      float y1, y2;
      turn(x1, x2, ang[q], y1, y2);
      put(dst + e1, y1);
      put(dst + e2, y2);
    } else if constexpr (kInterleaved) {
      float v[kV];
      Vec<T>::load(src + q * kV, v);
#pragma unroll
      for (int k = 0; k < kV; k += 2) {
        turn(v[k], v[k + 1], ang[(q * kV + k) / 2], v[k], v[k + 1]);
      }
      Vec<T>::store(dst + q * kV, v);
    } else {
      float v1[kV], v2[kV];
      Vec<T>::load(src + q * kV, v1);
      Vec<T>::load(src + half + q * kV, v2);
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        turn(v1[k], v2[k], ang[q * kV + k], v1[k], v2[k]);
      }
      Vec<T>::store(dst + q * kV, v1);
      Vec<T>::store(dst + half + q * kV, v2);
    }
  }
}

template <typename T>
cudaError_t launch_t(const RotaryArgs& args, bool vector, int num_sms, cudaStream_t stream) {
  RotaryArgs a = args;
  const int heads = a.x[0].heads + a.x[1].heads;
  // tokens of a block: few enough that the grid fills the GPU (two blocks per SM), at
  // most 16 (the angles then take at most 16 KB and one block's rows are still long runs)
  int tokens = 16;
  while (tokens > 1 && a.total / tokens < 4ll * num_sms) tokens /= 2;
  a.tokens = tokens;
  const long long bx = (a.total + tokens - 1) / tokens;
  int split = 1;  // blocks that share a token's heads, when there are few tokens
  while (split < heads && bx * split < 2ll * num_sms) ++split;
  if (split > 65535) split = 65535;
  a.heads_per_block = (heads + split - 1) / split;
  split = (heads + a.heads_per_block - 1) / a.heads_per_block;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(split));
  const size_t smem = static_cast<size_t>(tokens) * (a.R / 2) * sizeof(float2);
  if (a.interleaved) {
    if (vector)
      rotary_kernel<T, true, true><<<grid, kThreads, smem, stream>>>(a);
    else
      rotary_kernel<T, true, false><<<grid, kThreads, smem, stream>>>(a);
  } else {
    if (vector)
      rotary_kernel<T, false, true><<<grid, kThreads, smem, stream>>>(a);
    else
      rotary_kernel<T, false, false><<<grid, kThreads, smem, stream>>>(a);
  }
  return cudaGetLastError();
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
