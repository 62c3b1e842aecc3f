// doc_ranges.cu -- document ids into the ranges that the modified-score calls read.
//
//   start[j] = first token of the run of equal ids that token j lies in,
//   end[j]   = one past its last token;  start[j] = end[j] = j for padding (id < 0).
//
// start is a running maximum of (j where a run begins) from the left, end a running
// minimum of (j + 1 where a run ends) from the right.  A CTA takes a span of chunks of 2048
// tokens, 4 to a thread: a scan over the thread's own, one over the threads (shuffles inside a
// warp, then over the warps), with what the span's other chunks leave to the next; for the
// runs that cross the span's ends a search outwards, 4096 tokens a step by the whole block, up
// to the run's own end.  A span is one chunk in rows of up to kMaxSpans chunks and longer
// beyond, so that a row's time stays linear in its length whatever its runs: at most N / 4096
// steps of 2.5 us (one run of 2^20 tokens 0.66 ms, of 2^24 tokens 10.5 ms; spans of one chunk
// took 158 ms for the latter).  12 bytes a token: a call is bound by the latency of a few
// dependent loads (2 x 8192 tokens 5.7 us), is made once per batch, and serves every layer's
// forward and backward calls.
#include <climits>

#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;  // tokens per thread
constexpr int kChunk = kThreads * kPer;
constexpr int kSearch = 8;  // tokens per thread and search step
constexpr int kMaxSpans = 512;  // CTAs of one row: about one wave

struct Max {
  static constexpr int identity = -1;
  __device__ static int op(int a, int b) { return max(a, b); }
};
struct Min {
  static constexpr int identity = INT_MAX;
  __device__ static int op(int a, int b) { return min(a, b); }
};

// Exclusive scan of one value per thread over the block, in thread order (or, reversed,
// from the last thread down).
template <class Op, bool kReverse>
__device__ int block_scan(int v, int* warp_val) {
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
  int w = lane < kWarps ? warp_val[lane] : Op::identity;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = kReverse ? __shfl_down_sync(all, w, o) : __shfl_up_sync(all, w, o);
    if (kReverse ? lane + o < 32 : lane >= o) w = Op::op(w, y);
  }
  const int before = __shfl_sync(all, w, kReverse ? min(warp + 1, 31) : max(warp - 1, 0));
  int ex = kReverse ? __shfl_down_sync(all, x, 1) : __shfl_up_sync(all, x, 1);
  if (lane == (kReverse ? 31 : 0)) ex = Op::identity;
  if (warp != (kReverse ? kWarps - 1 : 0)) ex = Op::op(ex, before);
  return ex;
}

// The scan of every thread's v over the whole block.
template <class Op>
__device__ int block_all(int v, int* warp_val) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (threadIdx.x % 32 == 0) warp_val[threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_val[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = Op::op(v, warp_val[w]);
  return v;
}

// (kMany: spans of several chunks.  Four blocks to an SM: with three, 512 of them are two waves
// and one run of 2^20 tokens took 1008 us)
template <bool kMany>
__global__ void __launch_bounds__(kThreads, 4)
    doc_ranges_kernel(const int* ids, int* start, int* end, int N, int long_span) {
  // (ids is not __restrict__: loads of what a kernel may never see written could be moved in
  // front of the wait below, while an earlier kernel still writes the ids)
  __shared__ int warp_val[kWarps];
  // (no early launch of what follows: a forward kernel's CTAs waiting on the SMs took 7 us
  // more than starting after this one)
  grid_dependency_wait();
  const size_t row = static_cast<size_t>(blockIdx.y) * N;
  ids += row;
  start += row;
  end += row;
  auto id_at = [&](int j) { return j >= 0 && j < N ? max(ids[j], -1) : -2; };
  // the CTA's span [s0, s1), a multiple of kChunk long but for the row's end
  const int span = kMany ? long_span : kChunk;
  const int s0 = static_cast<int>(blockIdx.x) * span, s1 = min(s0 + span, N);
  int c0 = s0, j0 = 0, c1 = 0;
  int id[kPer + 2];  // tokens j0 - 1 .. j0 + kPer
  auto load_chunk = [&]() {
    c1 = min(c0 + kChunk, s1);
    j0 = c0 + static_cast<int>(threadIdx.x) * kPer;
#pragma unroll
    for (int k = 0; k < kPer + 2; ++k) id[k] = id_at(j0 + k - 1);
  };
  load_chunk();
  // first token of the run that enters the span, one past the last of the one that leaves
  int left = s0, right = s1;
  const int first = id_at(s0), last = id_at(s1 - 1);
  if (first >= 0 && id_at(s0 - 1) == first) {
    left = Max::identity;
    for (int top = s0 - 1; left < 0; top -= kThreads * kSearch) {
      int found = Max::identity;  // (token 0 begins a run: the search ends there)
#pragma unroll
      for (int k = 0; k < kSearch; ++k) {
        const int j = top - k * kThreads - static_cast<int>(threadIdx.x);
        if (j >= 0 && (j == 0 || ids[j - 1] != ids[j])) found = max(found, j);
      }
      left = block_all<Max>(found, warp_val);
    }
  }
  if (last >= 0 && id_at(s1) == last) {
    right = Min::identity;
    for (int low = s1; right == Min::identity; low += kThreads * kSearch) {
      int found = Min::identity;
#pragma unroll
      for (int k = 0; k < kSearch; ++k) {
        const int j = low + k * kThreads + static_cast<int>(threadIdx.x);
        if (j < N && (j == N - 1 || ids[j + 1] != ids[j])) found = min(found, j + 1);
      }
      right = block_all<Min>(found, warp_val);
    }
  }
  int v[kPer], run;
  while (true) {  // the first chunk to the last
    run = Max::identity;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (j0 + k < c1 && id[k + 1] != id[k]) run = j0 + k;
      v[k] = run;
    }
    const int before = max(block_scan<Max, false>(run, warp_val), left);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (j0 + k < c1) start[j0 + k] = id[k + 1] < 0 ? j0 + k : max(v[k], before);
    if (!kMany || c1 == s1) break;
    left = max(left, block_all<Max>(run, warp_val));
    c0 += kChunk;
    load_chunk();
  }
  while (true) {  // and back
    run = Min::identity;
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k) {
      if (j0 + k < c1 && id[k + 1] != id[k + 2]) run = j0 + k + 1;
      v[k] = run;
    }
    const int after = min(block_scan<Min, true>(run, warp_val), right);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (j0 + k < c1) end[j0 + k] = id[k + 1] < 0 ? j0 + k : min(v[k], after);
    if (!kMany || c0 == s0) break;
    right = min(right, block_all<Min>(run, warp_val));
    c0 -= kChunk;
    load_chunk();
  }
}

}  // namespace

cudaError_t launch_doc_ranges(const int* ids, int* start, int* end, int B, int N,
                              cudaStream_t stream) {
  const int chunks = (N + kChunk - 1) / kChunk;
  const int span = (chunks + kMaxSpans - 1) / kMaxSpans * kChunk;
  // (a grid's y extent is limited: rows in slices)
  for (int b = 0; b < B; b += 65535) {
    const dim3 grid(static_cast<unsigned>((N + span - 1) / span),
                    static_cast<unsigned>(B - b < 65535 ? B - b : 65535));
    const size_t at = static_cast<size_t>(b) * N;
    const cudaError_t e =
        launch_early(chunks > kMaxSpans ? doc_ranges_kernel<true> : doc_ranges_kernel<false>, grid,
                     kThreads, 0, stream, true, ids + at, start + at, end + at, N, span);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fa
