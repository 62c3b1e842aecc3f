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
// give the tiles it meets and the part that needs no element mask, and an element mask
// costs one subtraction and one unsigned compare.  (Arrays of the caller's making that
// do not rise give unspecified results, never an access out of range: every limit is
// clamped to the sequence.)
#pragma once

#include <cstddef>
#include <type_traits>

#include "internal.h"
#include "sm100.cuh"

namespace fa {

constexpr int kModNone = 0;  // scale and causal mask only: the unmodified calls
constexpr int kModMask = 1;  // masks and distance bias
constexpr int kModCap = 2;   // the same, and scores capped by a tanh

constexpr float kLog2e = 1.4426950408889634f;

// The tanh cap.  A raw product s becomes tanh's argument y = s * in; the capped score in
// log2 units is out * tanh(y) = s q(s^2) with q the polynomial of a tile's range (below).
struct CapArgs {
  float in;             // scale / cap
  float out;            // cap log2(e)
  float inv_out2;       // 1 / out^2
  float top3, top5;     // |s| up to which q3 and q5 hold (0: never)
  float q3[4], q5[6];   // coefficients of (s^2)^i
};

// tanh(sqrt(u)) / sqrt(u) as polynomials in u, minimax in the relative error (fitted here
// by iteratively reweighted least squares): 5.5e-7 for |y| <= 1/2, 5.9e-7 for |y| <= 1.
inline CapArgs cap_args(float scale, float softcap) {
  const double p3[4] = {0.9999994557706547, -0.33326317933916044, 0.13190296581699465,
                        -0.04440222555557586};
  const double p5[6] = {0.9999994135982464, -0.3332904237357338, 0.13281433841588497,
                        -0.05160567291576986, 0.01674311383038407, -0.0030670598357108976};
  CapArgs c{};
  if (softcap <= 0.f) return c;
  const double in = static_cast<double>(scale) / softcap;
  const double out = 1.4426950408889634 * softcap;
  c.in = static_cast<float>(in);
  c.out = static_cast<float>(out);
  c.inv_out2 = static_cast<float>(1.0 / (out * out));
  // (a cap so far below the scale that the scaled coefficients could overflow leaves no
  // score below it to speak of)
  if (in < 100.0) {
    c.top3 = static_cast<float>(0.5 / in);
    c.top5 = static_cast<float>(1.0 / in);
  }
  double f = out * in;
  for (int i = 0; i < 6; ++i, f *= in * in) {
    if (i < 4) c.q3[i] = static_cast<float>(p3[i] * f);
    c.q5[i] = static_cast<float>(p5[i] * f);
  }
  return c;
}

struct ModArgs {
  const int* doc_start;  // [B][Nk], or null
  const int* doc_end;
  const int* prefix;     // [B], or null
  const float* slopes;   // [H], or null
  int Hkv;               // key heads
  int group;             // query heads of one key head
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
  return p.Hkv == 0 ? kModNone : p.softcap > 0.f ? kModCap : kModMask;
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

// How a tile's capped scores are formed, from the largest |s| of the warp's entries:
// kCap3, kCap5: x = s q(s^2), 1 + degree packed multiply-adds an entry (the last product
// merges with the subtraction of the maximum) and nothing on the exponential unit, which
// the probabilities fill already; kCapTanh: tanh(y) = 1 - 2 / (1 + e^{2y}), two more
// exponential-unit operations an entry.  The error of the last is absolute, one float32
// rounding at 1, which next to an entry with |y| > 1 is below that score's own rounding,
// and it saturates to +-1 by itself.  Scores of trained models lie well inside their cap:
// the polynomials are the usual case.
constexpr int kCapTanh = 0, kCap3 = 3, kCap5 = 5;

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

__device__ __forceinline__ int cap_form(float amax, const CapArgs& c) {
  const bool over3 = !(amax <= c.top3), over5 = !(amax <= c.top5);
  if (!__any_sync(0xffffffffu, over3)) return kCap3;
  return __any_sync(0xffffffffu, over5) ? kCapTanh : kCap5;
}

// q(s^2) of a pair (kForm kCap3 or kCap5): the factor that takes s to log2 units.
template <int kForm>
__device__ __forceinline__ uint64_t cap_factor(uint64_t s2, const CapArgs& c) {
  using namespace sm100;
  const uint64_t u = mul_x2(s2, s2);
  if constexpr (kForm == kCap3) {
    uint64_t q = fma_x2(u, f32x2(c.q3[3], c.q3[3]), f32x2(c.q3[2], c.q3[2]));
    q = fma_x2(u, q, f32x2(c.q3[1], c.q3[1]));
    return fma_x2(u, q, f32x2(c.q3[0], c.q3[0]));
  } else {
    uint64_t q = fma_x2(u, f32x2(c.q5[5], c.q5[5]), f32x2(c.q5[4], c.q5[4]));
    q = fma_x2(u, q, f32x2(c.q5[3], c.q5[3]));
    q = fma_x2(u, q, f32x2(c.q5[2], c.q5[2]));
    q = fma_x2(u, q, f32x2(c.q5[1], c.q5[1]));
    return fma_x2(u, q, f32x2(c.q5[0], c.q5[0]));
  }
}

__device__ __forceinline__ float cap_tanh(float s, const CapArgs& c) {
  const float e = sm100::ex2_approx(s * (2.f * kLog2e * c.in));
  return fmaf(-2.f, sm100::rcp_approx(1.f + e), 1.f);
}

// N raw products to capped scores in log2 units, in place.
template <int N>
__device__ __forceinline__ void cap_scores(float* s, const CapArgs& c) {
  using namespace sm100;
  if (cap_form(abs_max<N>(s), c) != kCapTanh) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const uint64_t s2 = f32x2(s[k], s[k + 1]);
      f32x2_split(mul_x2(s2, cap_factor<kCap5>(s2, c)), s[k], s[k + 1]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = c.out * cap_tanh(s[k], c);
  }
}

// Two neighbouring entries of a score row or column in the backward pass, from their raw
// products: the probabilities e = 2^(x - L2) and, with a cap, its derivatives
// g = 1 - tanh^2 = 1 - (x / out)^2.  nl holds -L2 of the two entries, the distance bias is
// sl * (pos_d + k) for entry k, or sl * |pos_d + k| where the tile's keys lie on both sides
// of the position.
template <int kMode, int kForm>
__device__ __forceinline__ void mod_prob_pair(float s0, float s1, const ModArgs& m,
                                              uint64_t scale2, uint64_t nl, float sl, float pos_d,
                                              bool straddles, float& e0, float& e1, float& g0,
                                              float& g1) {
  using namespace sm100;
  if (m.slopes != nullptr) {
    float n0, n1;
    f32x2_split(nl, n0, n1);
    const float d0 = pos_d, d1 = pos_d + 1.f;
    n0 = fmaf(sl, straddles ? fabsf(d0) : d0, n0);
    n1 = fmaf(sl, straddles ? fabsf(d1) : d1, n1);
    nl = f32x2(n0, n1);
  }
  const uint64_t s2 = f32x2(s0, s1);
  if constexpr (kMode == kModCap) {
    uint64_t x;
    if constexpr (kForm == kCapTanh)
      x = f32x2(m.cap.out * cap_tanh(s0, m.cap), m.cap.out * cap_tanh(s1, m.cap));
    else
      x = mul_x2(s2, cap_factor<kForm>(s2, m.cap));
    exp2_pair(add_x2(x, nl), e0, e1);
    const uint64_t g = fma_x2(mul_x2(x, x), f32x2(-m.cap.inv_out2, -m.cap.inv_out2), f32x2(1.f, 1.f));
    f32x2_split(g, g0, g1);
  } else {
    exp2_pair(fma_x2(s2, scale2, nl), e0, e1);
    g0 = g1 = 1.f;
  }
}

// Calls f with the form as a compile-time constant (kCapTanh, kCap3 or kCap5).
template <int kMode, typename F>
__device__ __forceinline__ void with_cap_form(int form, const F& f) {
  if constexpr (kMode == kModCap) {
    if (form == kCap3)
      f(std::integral_constant<int, kCap3>{});
    else if (form == kCap5)
      f(std::integral_constant<int, kCap5>{});
    else
      f(std::integral_constant<int, kCapTanh>{});
  } else {
    f(std::integral_constant<int, kCapTanh>{});
  }
}

}  // namespace fa
