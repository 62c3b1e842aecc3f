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

#include "internal.h"
#include "sm100.cuh"

namespace fa {

constexpr int kModNone = 0;  // scale and causal mask only: the unmodified calls
constexpr int kModMask = 1;  // masks and distance bias
constexpr int kModCap = 2;   // the same, and scores capped by a tanh

constexpr float kLog2e = 1.4426950408889634f;

struct ModArgs {
  const int* doc_start;  // [B][Nk], or null
  const int* doc_end;
  const int* prefix;     // [B], or null
  const float* slopes;   // [H], or null
  int Hkv;               // key heads
  int group;             // query heads of one key head
  float cap_y;           // scale / cap: a raw product s becomes tanh's argument s * cap_y
  float cap_log2;        // cap log2(e)
};

inline ModArgs mod_args(const Problem& p) {
  ModArgs m{};
  m.doc_start = p.doc_start;
  m.doc_end = p.doc_end;
  m.prefix = p.prefix;
  m.slopes = p.slopes;
  m.Hkv = p.Hkv;
  m.group = p.Hkv > 0 ? p.H / p.Hkv : 1;
  if (p.softcap > 0.f) {
    m.cap_y = p.scale / p.softcap;
    m.cap_log2 = static_cast<float>(1.4426950408889634 * p.softcap);
  }
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

// tanh of N raw products times cap_y, in place (a thread's part of a score tile).
//
// Where every |y| of the warp is at most 1, tanh(y) = y P(y^2) with the degree-5 minimax
// polynomial of tanh(sqrt(u)) / sqrt(u) on [0, 1] (fitted here by iteratively reweighted
// least squares; relative error 6.7e-7 with the float32 evaluation): 4 packed
// multiply-adds an entry and nothing on the exponential unit, which the probabilities
// already fill.  Otherwise tanh(y) = 1 - 2 / (1 + e^{2y}), two more exponential-unit
// operations an entry; its error is absolute, one float32 rounding at 1, which next to an
// entry with |y| > 1 is below the rounding of that score, and it saturates to +-1 by
// itself.  Scores of trained models lie well inside their cap, so the first form is the
// usual one.
constexpr float kTanh0 = 0x1.ffffecp-1f, kTanh1 = -0x1.554a16p-2f, kTanh2 = 0x1.1000f6p-3f,
                kTanh3 = -0x1.a6c0f0p-5f, kTanh4 = 0x1.1251b4p-6f, kTanh5 = -0x1.92016ep-9f;

template <int N>
__device__ __forceinline__ void tanh_scores(float* s, const ModArgs& m) {
  using namespace sm100;
  float a8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) a8[k] = fabsf(s[k]);
#pragma unroll
  for (int c = 8; c < N; c += 2)
    a8[(c / 2) % 8] = max3(a8[(c / 2) % 8], fabsf(s[c]), fabsf(s[c + 1]));
  const float amax = max3(max3(a8[0], a8[1], a8[2]), max3(a8[3], a8[4], a8[5]),
                          fmaxf(a8[6], a8[7]));
  if (!__any_sync(0xffffffffu, amax * m.cap_y > 1.f)) {
    const uint64_t k2 = f32x2(m.cap_y, m.cap_y);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint64_t y = mul_x2(f32x2(s[c], s[c + 1]), k2);
      const uint64_t u = mul_x2(y, y);
      uint64_t q = fma_x2(u, f32x2(kTanh5, kTanh5), f32x2(kTanh4, kTanh4));
      q = fma_x2(u, q, f32x2(kTanh3, kTanh3));
      q = fma_x2(u, q, f32x2(kTanh2, kTanh2));
      q = fma_x2(u, q, f32x2(kTanh1, kTanh1));
      q = fma_x2(u, q, f32x2(kTanh0, kTanh0));
      f32x2_split(mul_x2(y, q), s[c], s[c + 1]);
    }
  } else {
    const float k = 2.f * kLog2e * m.cap_y;
#pragma unroll
    for (int c = 0; c < N; ++c)
      s[c] = fmaf(-2.f, rcp_approx(1.f + ex2_approx(s[c] * k)), 1.f);
  }
}

// Two neighbouring entries of a score row or column in the backward pass: the
// probabilities e = 2^(x - L2) and, with a cap, its derivatives g = 1 - tanh^2.  s0 and s1
// are the raw products, or their tanh_scores with a cap; `unit2` turns them into log2
// units.  nl holds -L2 of the two entries, the distance bias is sl * (pos_d + k) for entry
// k, or sl * |pos_d + k| where the tile's keys lie on both sides of the position.
template <int kMode>
__device__ __forceinline__ void mod_prob_pair(float s0, float s1, const ModArgs& m,
                                              uint64_t unit2, uint64_t nl, float sl, float pos_d,
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
  exp2_pair(fma_x2(s2, unit2, nl), e0, e1);
  g0 = g1 = 1.f;
  if constexpr (kMode == kModCap) {
    g0 = fmaf(-s0, s0, 1.f);
    g1 = fmaf(-s1, s1, 1.f);
  }
}

}  // namespace fa
