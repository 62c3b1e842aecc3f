// doc_ranges.cu -- document ids into the ranges that the modified-score calls read.
//
//   start[j] = first token of the run of equal ids that token j lies in,
//   end[j]   = one past its last token;  start[j] = end[j] = j for padding (id < 0).
//
// start is a running maximum of (j where a run begins) from the left, end a running
// minimum of (j + 1 where a run ends) from the right.  One CTA per sequence walks chunks
// of 8192 tokens, 8 to a thread: a scan over the thread's own tokens, one over the
// threads (shuffles inside a warp, then over the 32 warps), and a carry from chunk to
// chunk.  12 bytes per token in all; a call is bound by the latency of its two passes
// (a few microseconds), is made once per batch, and serves every layer's forward and
// backward calls.
#include <climits>

#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = 8;  // tokens per thread and chunk
constexpr int kChunk = kThreads * kPer;

struct Max {
  static constexpr int identity = -1;
  __device__ static int op(int a, int b) { return max(a, b); }
};
struct Min {
  static constexpr int identity = INT_MAX;
  __device__ static int op(int a, int b) { return min(a, b); }
};

// Exclusive scan of one value per thread over the block, in thread order (or, reversed,
// from the last thread down); `total` becomes the scan over all threads.
template <class Op, bool kReverse>
__device__ int block_scan(int v, int* warp_val, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const unsigned all = 0xffffffffu;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = kReverse ? __shfl_down_sync(all, x, o) : __shfl_up_sync(all, x, o);
    if (kReverse ? lane + o < 32 : lane >= o) x = Op::op(x, y);
  }
  __syncthreads();  // the previous scan's readers are done with warp_val
  if (lane == (kReverse ? 0 : 31)) warp_val[warp] = x;
  __syncthreads();
  int w = warp_val[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = kReverse ? __shfl_down_sync(all, w, o) : __shfl_up_sync(all, w, o);
    if (kReverse ? lane + o < 32 : lane >= o) w = Op::op(w, y);
  }
  total = __shfl_sync(all, w, kReverse ? 0 : 31);
  const int before = __shfl_sync(all, w, kReverse ? min(warp + 1, 31) : max(warp - 1, 0));
  int ex = kReverse ? __shfl_down_sync(all, x, 1) : __shfl_up_sync(all, x, 1);
  if (lane == (kReverse ? 31 : 0)) ex = Op::identity;
  if (warp != (kReverse ? 31 : 0)) ex = Op::op(ex, before);
  return ex;
}

__global__ void __launch_bounds__(kThreads)
    doc_ranges_kernel(const int* __restrict__ ids, int* __restrict__ start,
                      int* __restrict__ end, int N) {
  __shared__ int warp_val[32];
  const size_t row = static_cast<size_t>(blockIdx.x) * N;
  ids += row;
  start += row;
  end += row;
  auto id_at = [&](int j) { return j >= 0 && j < N ? max(ids[j], -1) : -2; };
  int carry = Max::identity;
  for (int c = 0; c < N; c += kChunk) {
    const int j0 = c + static_cast<int>(threadIdx.x) * kPer;
    int id[kPer + 1];
#pragma unroll
    for (int k = 0; k <= kPer; ++k) id[k] = id_at(j0 + k - 1);
    int v[kPer];
    int run = Max::identity;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (id[k + 1] != id[k]) run = j0 + k;
      v[k] = run;
    }
    int total;
    const int before = max(block_scan<Max, false>(run, warp_val, total), carry);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (j0 + k < N) start[j0 + k] = id[k + 1] < 0 ? j0 + k : max(v[k], before);
    carry = max(carry, total);
  }
  carry = Min::identity;
  for (int c = (N - 1) / kChunk * kChunk; c >= 0; c -= kChunk) {
    const int j0 = c + static_cast<int>(threadIdx.x) * kPer;
    int id[kPer + 1];
#pragma unroll
    for (int k = 0; k <= kPer; ++k) id[k] = id_at(j0 + k);
    int v[kPer];
    int run = Min::identity;
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k) {
      if (j0 + k < N && id[k] != id[k + 1]) run = j0 + k + 1;
      v[k] = run;
    }
    int total;
    const int after = min(block_scan<Min, true>(run, warp_val, total), carry);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (j0 + k < N) end[j0 + k] = id[k] < 0 ? j0 + k : min(v[k], after);
    carry = min(carry, total);
  }
}

}  // namespace

cudaError_t launch_doc_ranges(const int* ids, int* start, int* end, int B, int N,
                              cudaStream_t stream) {
  doc_ranges_kernel<<<B, kThreads, 0, stream>>>(ids, start, end, N);
  return cudaGetLastError();
}

}  // namespace fa
