// mod.cuh -- the score modifications of the _mod calls, as the tensor-core kernels use them.
//
//   z = scale q.k
//   x = cap tanh(z / cap)                       (when a cap is given)
//   x = x - slope_h |p_i - j|                   (when slopes are given)
//   key j is visible to query row i, at position p_i = i + Nk - Nq, when
//       (not causal, or j <= p_i, or j < prefix_b) and both are in the same document.
//
// Documents are runs of tokens, given as the first token and one past the last token of
// the run each token lies in.  A query row's visible keys are then one interval
//       [start[p], min(end[p], causal ? max(p + 1, prefix) : Nk)),
// a key's queries are one interval of positions too,
//       [max(start[j], causal and j >= prefix ? j : 0), end[j]),
// and both ends of either rise with the row.  So the first and the last row of a tile
// give the tiles it meets and the part that needs no element mask, and where one is needed
// 32 entries' visibility is one word of bits.  (Arrays of the caller's making that
// do not rise give unspecified results, never an access out of range: every limit is
// clamped to the sequence.)
#pragma once

#include <cmath>
#include <cstddef>

#include "internal.h"
#include "sm100.cuh"

namespace fa {

// A kernel is compiled for one combination.  The element-wise loops are straight code of
// several KB with two warps to a scheduler, so a second variant inside the same kernel is
// paid for in instruction fetch: with all of them in one kernel the capped dK/dV and dQ
// kernels ran 48 % and 39 % longer (383 and 260 us against 258 and 186 us, B=1 H=16 N=4096
// d=128).  What a tile seldom needs (masks, scores near the cap) is kept short and apart.
constexpr int kModNone = 0;      // scale and causal mask only: the unmodified calls
constexpr int kModMask = 1;      // masks and shared heads
constexpr int kModBias = 3;      // and distance bias
constexpr int kModCap = 5;       // masks, shared heads and capped scores
constexpr int kModCapBias = 7;   // all
constexpr bool has_bias(int mode) { return (mode & 2) != 0; }
constexpr bool has_cap(int mode) { return (mode & 4) != 0; }

__device__ __forceinline__ bool seldom(bool x) { return __builtin_expect(x, 0); }

constexpr float kLog2e = 1.4426950408889634f;

// The tanh cap.  A raw product s becomes tanh's argument y = s * in; the capped score in
// log2 units is x = out * tanh(y) = s q(s^2), q a polynomial, while |s| <= top.  Scores of
// trained models lie well inside their cap, so that is the usual case, and it needs nothing
// of the exponential unit, which the probabilities fill.
struct CapArgs {
  float in;        // scale / cap
  float out;       // cap log2(e)
  float neg_inv_out2;  // -1 / out^2
  float top;       // |s| up to which the forward's usual path goes (see cap_args)
  float poly;      // |s| up to which q holds; top <= poly
  float q[5];      // x = s q(s^2)
  float top_b;     // |s| up to which the backward uses qb and g
  float qb[4];     // x = s qb(s^2)
  float g[3];      // 1 - tanh^2 = g(s^2)
};

// tanh(sqrt(u)) / sqrt(u) as polynomials: to degree 4 for |y| <= 0.8, relative error 1.1e-6
// evaluated in float32, for the forward; to degree 3 for |y| <= 1/2, 5.9e-7, for the
// backward, with sech^2(sqrt(u)) to degree 2, 1.6e-4 (it multiplies dS, which is rounded to
// bf16 next, 2^-8).  Minimax in the relative error, fitted here by iteratively reweighted
// least squares.  The forward pays 6 % for its wider range (B=2 H=16 N=4096 d=128 causal, Q
// and K of deviation 1.5, cap 50: 183 us against 171 with degree 3), because a tile outside
// it costs the forward more: with 1/2, scores of that size under a cap of 20 took 318 us,
// now 183.  The backward would gain nothing from it there (560 us either way) and lose 4 %
// under the larger cap.
// Caps far above the scores use no more than |y| <= 1/5, where the Taylor series of the
// same degrees are off by 5.6e-8 (degree 3; less for 4) and 6e-4 y^2 at most: scores in the
// hundreds then keep float32's digits.
inline CapArgs cap_args(float scale, float softcap) {
  const double fit_q[5] = {0.9999989943428248, -0.33325371953005856, 0.13230565487990226,
                           -0.049180140355985856, 0.01210013750460391};
  const double fit_qb[4] = {0.9999994557706547, -0.33326317933916044, 0.13190296581699465,
                            -0.04440222555557586};
  const double fit_g[3] = {0.9998382199693817, -0.9886407641960892, 0.5423509665406153};
  const double taylor_q[5] = {1.0, -1.0 / 3, 2.0 / 15, -17.0 / 315, 62.0 / 2835};
  const double taylor_g[3] = {1.0, -1.0, 2.0 / 3};
  CapArgs c{};
  if (softcap <= 0.f) return c;
  const double in = static_cast<double>(scale) / softcap;
  const double out = 1.4426950408889634 * softcap;
  c.in = static_cast<float>(in);
  c.out = static_cast<float>(out);
  c.neg_inv_out2 = static_cast<float>(-1.0 / (out * out));
  // In a tile of which a row sees a key, the forward takes the score of the largest |s| for
  // the row's reference maximum.  The visible one is then within 2 * 50 of it, so the largest
  // probability of the row is at least 2^-100, far from float32's (and bf16's) smallest: out *
  // tanh(y) <= 50 bounds y for caps above 52.  (A tile that the row sees nothing of must not
  // set its reference: the visible scores may all lie past the range, down to -out.)
  double y = 0.8;
  if (out * std::tanh(y) > 50.0) y = std::atanh(50.0 / out);
  const bool taylor = y < 0.2;
  c.top = static_cast<float>(y / in);
  c.poly = static_cast<float>((taylor ? 0.2 : 0.8) / in);
  c.top_b = static_cast<float>((taylor ? 0.2 : 0.5) / in);
  const double* q = taylor ? taylor_q : fit_q;
  const double* qb = taylor ? taylor_q : fit_qb;
  const double* g = taylor ? taylor_g : fit_g;
  // (Caps far below the scale, in above 1e5, take the last coefficients past float32, and zero
  // times infinity is a NaN: no product is in such a polynomial's range, zero ones included.)
  double f = 1.0;
  bool holds = true, holds_b = true;
  for (int i = 0; i < 5; ++i, f *= in * in) {
    c.q[i] = static_cast<float>(q[i] * f * out * in);
    holds = holds && std::isfinite(c.q[i]);
    if (i < 4) c.qb[i] = static_cast<float>(qb[i] * f * out * in);
    if (i < 3) c.g[i] = static_cast<float>(g[i] * f);
    holds_b = holds_b && std::isfinite(c.qb[i < 4 ? i : 3]) && std::isfinite(c.g[i < 3 ? i : 2]);
  }
  if (!holds) c.top = c.poly = -1.f;
  if (!holds_b) c.top_b = -1.f;
  return c;
}

struct ModArgs {
  const int* doc_start;  // [B][Nk], or null
  const int* doc_end;
  const int* prefix;     // [B], or null
  const float* slopes;   // [H] (kModBias, kModCapBias)
  int Hkv;               // key heads
  int group;             // query heads of one key head
  int ordered;           // the kernel ranks its units by cost (order_units)
  CapArgs cap;
};

inline ModArgs mod_args(const Problem& p) {
  ModArgs m{};
  m.doc_start = p.doc_start;
  m.doc_end = p.doc_end;
  m.prefix = p.prefix;
  m.slopes = p.slopes;
  m.Hkv = p.Hkv;
  m.group = p.Hkv > 0 ? p.H / p.Hkv : 1;
  m.cap = cap_args(p.scale, p.softcap);
  return m;
}

inline int mod_mode(const Problem& p) {
  if (p.Hkv == 0) return kModNone;
  return kModMask | (p.slopes != nullptr ? 2 : 0) | (p.softcap > 0.f ? 4 : 0);
}

struct RowLimits {
  int lo, hi;  // lo <= hi
};

// Visible keys of query row i of sequence b (0 <= lo <= hi <= Nk).
__device__ __forceinline__ RowLimits mod_row(const ModArgs& m, int b, int i, int off, int Nk,
                                             int causal) {
  const int p = i + off;
  RowLimits r{0, Nk};
  if (causal) {
    r.hi = p + 1;
    if (m.prefix != nullptr) r.hi = max(r.hi, min(m.prefix[b], Nk));
  }
  if (m.doc_start != nullptr) {
    if (p < 0) return RowLimits{0, 0};  // in front of the first key: in no document
    const size_t at = static_cast<size_t>(b) * Nk + p;
    r.lo = min(max(m.doc_start[at], 0), Nk);
    r.hi = min(r.hi, m.doc_end[at]);
  }
  r.hi = max(r.hi, r.lo);
  return r;
}

// Query rows that see key j of sequence b (0 <= lo <= hi <= Nq).
__device__ __forceinline__ RowLimits mod_key(const ModArgs& m, int b, int j, int off, int Nq,
                                             int Nk, int causal) {
  int lo = off, hi = Nk;  // positions; query row 0 sits at off, which may be negative
  if (m.doc_start != nullptr) {
    // (positions in front of the first key are in no document)
    const size_t at = static_cast<size_t>(b) * Nk + j;
    lo = min(max(m.doc_start[at], 0), Nk);
    hi = min(max(m.doc_end[at], 0), Nk);
  }
  if (causal && (m.prefix == nullptr || j >= m.prefix[b])) lo = max(lo, j);
  RowLimits r;
  r.lo = min(max(lo - off, 0), Nq);
  r.hi = max(min(hi - off, Nq), r.lo);
  return r;
}

// Work units of documents differ in cost by far more than causal ones, and not in order of
// their index: the units (n of them, one head's) are ranked by cost(e), dearest first, for
// the persistent kernels' dealing order.  (10000 tokens of 450 to 2550-token documents, d =
// 128: dK/dV 145 -> 127 us, dQ 107 -> 96; equal documents of 512 tokens on tile bounds, which
// the index order suits: 72 -> 78 and 57 -> 63.)  Called by all `threads` threads of a CTA before
// its pipelines start; `scratch` is n uint16, rounded up to 16 bytes, of aligned shared memory
// that a TMA load may write later, `order` n bytes that stay.  A __syncthreads() must follow.
constexpr int kMaxOrdered = 256;

template <typename Cost>
__device__ __forceinline__ void order_units(int n, int threads, uint16_t* scratch, uint8_t* order,
                                            const Cost& cost) {
  const int n8 = (n + 7) / 8;
  for (int e = threadIdx.x; e < 8 * n8; e += threads)
    scratch[e] = e < n ? static_cast<uint16_t>(min(cost(e), 65535)) : 0;
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += threads) {
    const int c = scratch[e];
    int rank = 0;
    for (int g = 0; g < n8; ++g) {  // eight costs a load; equal ones keep their order
      const uint4 v = reinterpret_cast<const uint4*>(scratch)[g];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int o = (w[k / 2] >> (16 * (k % 2))) & 0xffff;
        rank += o > c || (o == c && 8 * g + k < e);
      }
    }
    order[rank] = static_cast<uint8_t>(e);
  }
  sm100::fence_proxy_async_shared();
}

template <int N>
__device__ __forceinline__ float abs_max(const float* s) {
  float a8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) a8[k] = fabsf(s[k]);
#pragma unroll
  for (int c = 8; c < N; c += 2)
    a8[(c / 2) % 8] = sm100::max3(a8[(c / 2) % 8], fabsf(s[c]), fabsf(s[c + 1]));
  return sm100::max3(sm100::max3(a8[0], a8[1], a8[2]), sm100::max3(a8[3], a8[4], a8[5]),
                     fmaxf(a8[6], a8[7]));
}

// Whether some |s| of the warp is past the usual path's range (or not a number).
__device__ __forceinline__ bool cap_over(float amax, float top) {
  return __any_sync(0xffffffffu, !(amax <= top));
}

// q(s^2) of a pair: the factor that takes s to its capped score in log2 units.
__device__ __forceinline__ uint64_t cap_factor(uint64_t s2, const CapArgs& c) {
  using namespace sm100;
  const uint64_t u = mul_x2(s2, s2);
  uint64_t q = fma_x2(u, f32x2(c.q[4], c.q[4]), f32x2(c.q[3], c.q[3]));
  q = fma_x2(u, q, f32x2(c.q[2], c.q[2]));
  q = fma_x2(u, q, f32x2(c.q[1], c.q[1]));
  return fma_x2(u, q, f32x2(c.q[0], c.q[0]));
}

// tanh(s in) = 1 - 2 / (1 + e^{2y}): saturates to +-1 by itself; the error is absolute, one
// float32 rounding at 1.
__device__ __forceinline__ float cap_tanh(float s, const CapArgs& c) {
  const float e = sm100::ex2_approx(s * (2.f * kLog2e * c.in));
  return fmaf(-2.f, sm100::rcp_approx(1.f + e), 1.f);
}

// The capped score in log2 units of any raw product: the polynomial where it holds (its
// error is relative: a cap far above the scores must not cost them their digits), the
// formula beyond.
__device__ __forceinline__ float cap_any(float s, const CapArgs& c) {
  const float u = s * s;
  const float q = fmaf(u, fmaf(u, fmaf(u, fmaf(u, c.q[4], c.q[3]), c.q[2]), c.q[1]), c.q[0]);
  return fabsf(s) <= c.poly ? s * q : c.out * cap_tanh(s, c);
}

// N raw products to capped scores in place, for the tiles with a score past the usual path's
// range: the formula for all of them, in registers, while its absolute error, 2^-23 out, is
// far below the rounding of P (out <= 256).  Larger caps go entry by entry through a copy in
// local memory: a rolled loop, which leaves the instruction cache to the usual path, but
// which the small L1 beside the kernels' shared memory makes many times slower than the
// tile's other work (B=2 H=16 N=4096 d=128 causal, products of deviation 16: cap 100 323 us,
// cap 1000 2068).  A third branch, the polynomial as far as it holds, takes that to 228 and
// costs every capped call its place in the instruction cache (the prompt B=1 H=16 over 4 N=8192
// 289 -> 313 us).
template <int N>
__device__ __forceinline__ void cap_scores_any(float* s, const CapArgs& c) {
  if (c.out <= 256.f) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = c.out * cap_tanh(s[k], c);
  } else {
    float t[N];
#pragma unroll
    for (int k = 0; k < N; ++k) t[k] = s[k];
#pragma unroll 1
    for (int k = 0; k < N; ++k) t[k] = cap_any(t[k], c);
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = t[k];
  }
}

// The same by the polynomial.
template <int N>
__device__ __forceinline__ void cap_scores(float* s, const CapArgs& c) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    const uint64_t s2 = sm100::f32x2(s[k], s[k + 1]);
    sm100::f32x2_split(sm100::mul_x2(s2, cap_factor(s2, c)), s[k], s[k + 1]);
  }
}

// Columns lo .. hi - 1 of 32 as bits (lo, hi any integers).
__device__ __forceinline__ uint32_t range_word(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi <= lo ? 0u : (~0u >> (32 - (hi - lo))) << lo;
}

__device__ __forceinline__ uint64_t abs_x2(uint64_t v) {
  float a, b;
  sm100::f32x2_split(v, a, b);
  return sm100::f32x2(fabsf(a), fabsf(b));
}

struct ColumnStat {  // a statistic per column, in shared memory
  const float* at;
  __device__ __forceinline__ uint64_t operator()(int c) const {
    return *reinterpret_cast<const uint64_t*>(at + c);
  }
};
struct RowStat {  // the same for every column
  uint64_t pair;
  __device__ __forceinline__ uint64_t operator()(int) const { return pair; }
};

// The backward pass's probabilities of N neighbouring entries of a score row or column,
// p = 2^(x - L2) of the raw products s, 0 outside columns [lo, hi) (when `partial`), and
// with kPack the bf16 pairs in pk.  nl(c) gives -L2 of columns c and c + 1 (-inf for a row
// that sees nothing).  The distance bias of column c is neg_slope * |at + c|.  Returns
// whether s now holds capped scores (some were past the polynomials' range).
template <int kMode, int N, bool kPack, typename NL>
__device__ __forceinline__ bool mod_probs(float* s, float* p, uint32_t* pk, const NL& nl,
                                          const ModArgs& m, float scale_log2, float neg_slope,
                                          float at, bool partial, int lo, int hi) {
  using namespace sm100;
  bool over = false;
  float q0 = 0.f, q1 = 0.f, q2 = 0.f, q3 = 0.f;
  if constexpr (has_cap(kMode)) {
    q0 = m.cap.qb[0], q1 = m.cap.qb[1], q2 = m.cap.qb[2], q3 = m.cap.qb[3];
    over = cap_over(abs_max<N>(s), m.cap.top_b);
    if (seldom(over)) {
      cap_scores_any<N>(s, m.cap);
      q0 = 1.f, q1 = q2 = q3 = 0.f;
    }
  }
  const uint64_t scale2 = f32x2(scale_log2, scale_log2), two2 = f32x2(2.f, 2.f);
  const uint64_t slope2 = f32x2(neg_slope, neg_slope);
  uint64_t d2 = f32x2(at, at + 1.f);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t s2 = f32x2(s[c], s[c + 1]);
    uint64_t n2 = nl(c);
    if constexpr (has_bias(kMode)) {
      n2 = fma_x2(slope2, abs_x2(d2), n2);
      d2 = add_x2(d2, two2);
    }
    uint64_t f2 = scale2;
    if constexpr (has_cap(kMode)) {
      const uint64_t u = mul_x2(s2, s2);
      f2 = fma_x2(u, f32x2(q3, q3), f32x2(q2, q2));
      f2 = fma_x2(u, f2, f32x2(q1, q1));
      f2 = fma_x2(u, f2, f32x2(q0, q0));
    }
    exp2_pair(fma_x2(s2, f2, n2), p[c], p[c + 1]);
    if constexpr (kPack) pk[c / 2] = pack_bf16x2(p[c], p[c + 1]);
  }
  if (seldom(partial)) {
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {
      const uint32_t w = range_word(lo - 32 * q, hi - 32 * q);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        if (!((w >> c) & 1u)) p[32 * q + c] = 0.f;
        if (!((w >> (c + 1)) & 1u)) p[32 * q + c + 1] = 0.f;
        if constexpr (kPack) pk[16 * q + c / 2] = pack_bf16x2(p[32 * q + c], p[32 * q + c + 1]);
      }
    }
  }
  return over;
}

// The cap's derivative into the probabilities that dS is made of: p[c] *= 1 - tanh^2, by
// the polynomial of the raw products, or 1 - (x / out)^2 of capped scores (`over`).  Done
// after the probabilities are handed to the MMA warp, while its products run.
template <int N>
__device__ __forceinline__ void mod_slopes(const float* s, float* p, bool over, const CapArgs& cap) {
  using namespace sm100;
  const float g0 = over ? 1.f : cap.g[0], g1 = over ? cap.neg_inv_out2 : cap.g[1],
              g2 = over ? 0.f : cap.g[2];
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t s2 = f32x2(s[c], s[c + 1]);
    const uint64_t u = mul_x2(s2, s2);
    uint64_t g = fma_x2(u, f32x2(g2, g2), f32x2(g1, g1));
    g = fma_x2(u, g, f32x2(g0, g0));
    f32x2_split(mul_x2(f32x2(p[c], p[c + 1]), g), p[c], p[c + 1]);
  }
}

}  // namespace fa
