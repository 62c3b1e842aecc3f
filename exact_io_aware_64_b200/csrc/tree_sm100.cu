// tree_sm100.cu -- attention of a few query rows per sequence (one decoded token, or a
// tree of drafted ones) over a paged key/value cache, on the sm_100a tensor cores.
//
//   O_row = softmax over the visible keys of x . V,   x = scale q.k, capped if asked,
// visible to drafted token t: every cached token before the drafted ones, and drafted
// token u when bit u of t's mask is set.
//
// Bound: HBM reads of the cache.  Every key head's rows (its query heads x its drafted
// tokens) are packed into 128-row tiles, so the cache is read once per 256 of them and
// the tensor cores do whole tiles whatever the row count: at 128 keys x 128 columns a
// tile pair takes 64 KB of K and V, which is 1.5 us of this SM's share of the HBM rate,
// about twice as long as its two products and its softmax.
//
// Measured: 32 sequences of 8192 tokens, 16 heads over 4, d = 128: 94 us, 87 % of the copy
// rate with both kernels and their launches (64 sequences: 173 us, 95 %); d = 64, 64
// sequences: 101 us, 81 %, bound by the chain of products, softmax and barriers of a tile
// half the size.  256 rows a key head (32 drafted tokens x 8 heads), 8 x 32768 tokens: 85 us,
// 104 capped, against 41 for the bytes: the softmax of two full row tiles, 2.8 us a key tile,
// paces it as it does the forward kernel.
//
// Split: the key tiles of all (sequence, key head, row tile pair) segments form one line
// that is cut into equal pieces, one per CTA, so ragged lengths, one long sequence and
// many short ones all load every SM alike.  The lengths are on the device, so each CTA
// forms the prefix sums of the tile counts itself.  A piece of a segment leaves
// its unnormalised float32 output, maximum and sum in the workspace (piece number = CTA
// number + segment number, which is unique along the line), and a second kernel joins a
// row's pieces in a fixed order: no atomics, the same bits on every run.
//
// A page is one TMA box whatever its columns: as a 5-D tensor of (64 columns, 8 rows, column
// halves, 8-row groups, pages) it lands as swizzle atoms of 8 rows x 128 bytes, the halves of
// a group next to each other, which the MMA descriptors step over with a stride of 8 rows.
// With a box per half, 32 boxes of 2 KB a tile pair at 16-token pages held a decode batch to
// 121 us where 64-token pages took 96.
//
// In a CTA (the roles of the forward kernel): warps 0-3 and 4-7 are two softmax
// warpgroups, warp 8 issues the TMA loads, warp 9 the MMAs.  Before the product with a
// sequence's last V tile, warp 9 clears the rows behind the sequence's end: a page's unused
// slots (and the part of the tile that no page was loaded for) may hold anything, and 0
// times a NaN is a NaN.
// With more than 128 rows the two warpgroups own a row tile each and both see every key
// tile; otherwise they own the same rows and take the key tiles in turn.  A warp none of
// whose rows exist only passes the barriers.
//
// With at most 64 (32) rows the row tile holds 2 (4) copies of them, and the warps of copy c
// take the c-th part of a key tile's columns: their probabilities elsewhere are zero, so each
// copy accumulates the output of its own keys, with its own maximum and sum, and is one more
// part for the joining kernel.  A single warp going through 128 columns takes longer than
// the tile's share of the HBM rate (1.7 us against 1.5 us a tile, 2.2 us capped); 32 columns
// each do not.
//
// Roundings: P goes to bf16 as the second product's operand (as in the forward kernel); pieces,
// their statistics and the join are float32, O is rounded once.
#include <cstdint>

#include "internal.h"
#include "mod.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

using namespace sm100;

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168, kRegsControl = 88, kRegsSoftmax = 208;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsControl <= kThreads * kRegsLaunch,
              "register split exceeds the launch pool");
constexpr int kWarpTMA = 8, kWarpMMA = 9;
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in the forward kernel
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Layout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBoxBytes = 128 * 128;    // 64 columns of a Q tile
  static constexpr int kGroupBytes = 8 * D * 2;  // 8 rows of a K or V tile
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kQ = 0;  // two row tiles
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBar = kRing + kStages * kTileBytes;
  static constexpr int kBarQFull = 0, kBarQEmpty = 1;
  static constexpr int kBarKVFull = 2;                       // [kStages]
  static constexpr int kBarKVEmpty = kBarKVFull + kStages;   // [kStages]
  static constexpr int kBarSFull = kBarKVEmpty + kStages;    // [2]
  static constexpr int kBarPReady = kBarSFull + 2;           // [2]
  static constexpr int kBarODone = kBarPReady + 2;           // [2]
  static constexpr int kBarOFree = kBarODone + 2;            // [2]
  static constexpr int kBarDrain = kBarOFree + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kPrefix = kMisc + 16;  // [B + 1] int
  static constexpr int bytes(int B) { return kPrefix + (B + 1) * 4 + 1024; }
};
static_assert(Layout<128>::bytes(kTreeMaxBatch) <= 232448 && Layout<64>::bytes(kTreeMaxBatch) <= 232448,
              "shared memory over the 227 KB per-block limit");

struct Unit {
  int b, head, rt;    // sequence, key head, first row tile
  int j0, j1;         // key tiles of the sequence
  int len, ctx, n;    // cached tokens, those before the drafted ones, drafted ones
  int piece;
};

// Tokens and drafted tokens of sequence b; (0, 0) for one out of range, which is reported.
__device__ __forceinline__ void tree_seq(const TreeArgs& a, int b, int& len, int& n, bool report) {
  len = a.cache_lens[b];
  n = a.seqlens_q != nullptr ? a.seqlens_q[b] : a.T;
  if (len < 0 || len > a.max_len || n < 0 || n > a.T || n > len) {
    if (report) atomicOr(a.err, kErrBadLength);
    len = 0;
    n = 0;
  }
}

// The unit that starts at tile `pos` of the line (prefix: tiles before each sequence).
__device__ __forceinline__ Unit tree_unit(const TreeArgs& a, const int* prefix, int pos, int end) {
  int lo = 0, hi = a.B - 1;  // last b with prefix[b] <= pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (prefix[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  Unit u;
  u.b = lo;
  const int per_seq = a.Hkv * a.pairs;
  const int tiles = (prefix[lo + 1] - prefix[lo]) / per_seq;
  const int seg = (pos - prefix[lo]) / tiles;
  u.head = seg / a.pairs;
  u.rt = (seg - u.head * a.pairs) * 2;
  u.j0 = pos - prefix[lo] - seg * tiles;
  u.j1 = min(tiles, u.j0 + end - pos);
  tree_seq(a, lo, u.len, u.n, false);
  u.ctx = u.len - u.n;
  u.piece = blockIdx.x + lo * per_seq + seg;
  return u;
}

// Visibility of 32 neighbouring keys, the first `d0` behind the first drafted token: keys
// before the drafted ones are seen, drafted ones by their bits, keys from 64 on are not.
__device__ __forceinline__ uint32_t seen_word(unsigned long long bits, int d0) {
  if (d0 >= 64 || d0 <= -32) return d0 >= 64 ? 0u : ~0u;
  return static_cast<uint32_t>(d0 >= 0 ? bits >> d0 : bits << -d0 | ((1ull << -d0) - 1ull));
}

struct KernelArgs : TreeArgs {
  CapArgs cap;
};

template <int D, bool kCap, int kCopies>
__global__ void __launch_bounds__(kThreads, 1)
    tree_sm100_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const KernelArgs a) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int i) -> uint32_t { return base + L::kBar + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  int* prefix = reinterpret_cast<int*>(smem + L::kPrefix);
  auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, a.err));
  };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(bar(L::kBarQFull), 1);
    mbar_init(bar(L::kBarQEmpty), 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarKVFull + s), 1);
      mbar_init(bar(L::kBarKVEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kBarSFull + t), 1);
      mbar_init(bar(L::kBarPReady + t), 4);
      mbar_init(bar(L::kBarODone + t), 1);
      mbar_init(bar(L::kBarOFree + t), 4);
    }
    mbar_init(bar(L::kBarDrain), 1);
    fence_mbar_init();
  }
  if (warp == kWarpTMA && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kWarpMMA) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  // tile counts, then their prefix sums (warp 0)
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    int len, n;
    tree_seq(a, b, len, n, blockIdx.x == 0);
    prefix[b + 1] = n > 0 ? (len + kBN - 1) / kBN * a.Hkv * a.pairs : 0;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int x = b0 + lane < a.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < a.B) prefix[b0 + lane + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int total = prefix[a.B];
  const int share = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int begin = min(total, static_cast<int>(blockIdx.x) * share);
  const int end = min(total, begin + share);
  if (blockIdx.x == 0)  // the joining kernel reads the line's layout from here
    for (int b = threadIdx.x; b <= a.B; b += kThreads) a.prefix_out[b] = prefix[b];
  grid_dependents_launch();  // the joining kernel
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + D};
  // one row tile: the two warpgroups share its rows and take the key tiles in turn
  const bool shared_rows = kCopies > 1 || a.rows <= kBM;
  constexpr int kCopyRows = kBM / kCopies;  // rows of a copy in the row tile
  constexpr int kCols = kBN / kCopies;      // key columns of a warp

  if (warp >= 8) regs_dec<kRegsControl>();
  if (warp == kWarpTMA) {
    int stage = 0;
    uint32_t phase = 0;
    int units = 0;
    bool ok = true;
    int issued[L::kStages];
    uint32_t issued_phase[L::kStages];
    for (int s = 0; s < L::kStages; ++s) issued[s] = 0, issued_phase[s] = 0;
    // This warp paces short tiles (with divisions and a table read per load it took 2060
    // cycles a tile, which held a d = 64 batch of 64 x 8192 tokens to 135 us; 101 as it is),
    // so it divides and reads the table seldom.  Pages below 128
    // tokens are a power of two: a tile is `per` boxes of a page each, lane p fetching box p;
    // larger pages hold `tiles` tiles of one box each.
    const bool small = a.page < kBN;
    const int page_sh = small ? 31 - __clz(a.page) : 7;  // log2 of a box's rows
    const int per = kBN >> page_sh, tiles = small ? 1 : a.page / kBN;
    const uint32_t box_bytes = static_cast<uint32_t>(D * 2) << page_sh;
    auto load = [&](const Unit& u, int j, int id, int tile_in_page, const CUtensorMap* tm) -> bool {
      if (!wait_warp(bar(L::kBarKVEmpty + stage), phase ^ 1)) return false;
      // the boxes of this tile that hold tokens
      const int n = min(per, (u.len - j * kBN + (1 << page_sh) - 1) >> page_sh);
      const uint32_t fb = bar(L::kBarKVFull + stage);
      if (lane == 0) mbar_arrive_expect_tx(fb, n * box_bytes);
      __syncwarp();
      if (lane < n)
        tma_load_5d(base + L::kRing + stage * L::kTileBytes + lane * box_bytes, tm, fb, 0, 0, 0,
                    tile_in_page * (kBN / 8), id * a.Hkv + u.head);
      issued[stage] = 1;
      issued_phase[stage] = phase;
      if (++stage == L::kStages) stage = 0, phase ^= 1;
      return true;
    };
    for (int pos = begin; ok && pos < end;) {
      const Unit u = tree_unit(a, prefix, pos, end);
      // page numbers: a lane holds one of 32 table entries from entry `win` on, and one of
      // the next 32; tile j's entries are e, e + 1, ..
      const int* table = a.block_table + static_cast<size_t>(u.b) * a.max_pages;
      int e = small ? u.j0 * per : u.j0 / tiles;
      int in_page = small ? 0 : u.j0 - e * tiles;
      const int e_end = small ? (min(u.len, u.j1 * kBN) + a.page - 1) >> page_sh
                              : (u.j1 - 1) / tiles + 1;
      auto entry = [&](int i) { return i < e_end ? table[i] : 0; };
      int win = e;
      int ids = entry(win + lane), ids_next = entry(win + 32 + lane);
      if (units > 0) ok = wait_warp(bar(L::kBarQEmpty), (units - 1) & 1);
      if (!ok) break;
      const int row_tiles = min(2, (a.rows - u.rt * kBM + kBM - 1) / kBM);
      mbar_arrive_expect_tx_elect(bar(L::kBarQFull), row_tiles * L::kTileBytes);
      for (int t = 0; t < row_tiles; ++t)
        for (int c = 0; c < D / 64; ++c)
          for (int k = 0; k < kCopies; ++k)  // (a box is kCopyRows rows high)
            tma_load_3d_elect(base + L::kQ + t * L::kTileBytes + c * L::kBoxBytes +
                                  k * kCopyRows * 128,
                              &tmQ, bar(L::kBarQFull), c * 64, (u.rt + t) * kBM,
                              u.b * a.Hkv + u.head);
      ++units;
      auto next_page = [&](int& tile_in_page) -> int {
        if (e - win == 32) {
          win += 32;
          ids = ids_next;
          ids_next = entry(win + 32 + lane);
        }
        int id = __shfl_sync(0xffffffffu, ids, (e - win + (lane & (per - 1))) & 31);
        if (id < 0 || id >= a.num_pages) {  // (entries behind the last token's page are 0 here)
          atomicOr(a.err, kErrBadPage);
          id = 0;
        }
        tile_in_page = in_page;
        if (small) {
          e += per;
        } else if (++in_page == tiles) {
          in_page = 0;
          ++e;
        }
        return id;
      };
      // order of use: K V K V ... (a row tile each), or K K V K V ... V V (shared rows)
      int o0, o1 = 0;
      int id0 = next_page(o0), id1 = 0;
      ok = load(u, u.j0, id0, o0, &tmK);
      for (int j = u.j0; ok && j < u.j1; ++j) {
        const bool more = j + 1 < u.j1;
        if (more) id1 = next_page(o1);
        if (shared_rows && more) ok = load(u, j + 1, id1, o1, &tmK);
        if (ok) ok = load(u, j, id0, o0, &tmV);
        if (ok && !shared_rows && more) ok = load(u, j + 1, id1, o1, &tmK);
        id0 = id1;
        o0 = o1;
      }
      pos += u.j1 - u.j0;
    }
    if (!ok) {
      for (int s = 0; s < L::kStages; ++s)
        if (issued[s]) mbar_wait_drain(bar(L::kBarKVFull + s), issued_phase[s], a.err);
      if (units > 0) mbar_wait_drain(bar(L::kBarQFull), (units - 1) & 1, a.err);
    }
  } else if (warp == kWarpMMA) {
    constexpr uint32_t idS = idesc_bf16_f32(kBN, false);
    constexpr uint32_t idPV = idesc_bf16_f32(D, true);
    int stage = 0, units = 0;
    uint32_t phase = 0;
    int p_count[2] = {0, 0}, o_uses[2] = {0, 0};
    bool ok = true;
    const uint64_t dQ[2] = {desc_kmajor(base + L::kQ), desc_kmajor(base + L::kQ + L::kTileBytes)};
    // K and V tiles: 8-row groups of kGroupBytes, a 1024-byte swizzle atom per 64 columns
    const uint64_t dRingK = smem_desc_sw128(base + L::kRing, 16u, L::kGroupBytes);
    const uint64_t dRingV = smem_desc_sw128(base + L::kRing, 1024u, L::kGroupBytes);
    auto next_slot = [&](int& slot) -> bool {
      slot = stage;
      const bool r = wait_warp(bar(L::kBarKVFull + stage), phase);
      if (++stage == L::kStages) stage = 0, phase ^= 1;
      return r;
    };
    auto issue_s = [&](int t, int q, int kslot) {
      const uint64_t db = dRingK + static_cast<uint64_t>((kslot * L::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        mma_ss_elect(tS[t], dQ[q] + (((kk / 4) * L::kBoxBytes + (kk % 4) * 32) >> 4),
                     db + (((kk / 4) * 1024 + (kk % 4) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
      }
      mma_commit_elect(bar(L::kBarSFull + t));
    };
    // O_t (+)= P_t V; the first product of a unit waits until the last one's O_t is read
    auto issue_pv = [&](int t, int vslot, bool first) -> bool {
      if (first && o_uses[t] > 0 && !wait_warp(bar(L::kBarOFree + t), (o_uses[t] - 1) & 1))
        return false;
      if (!wait_warp(bar(L::kBarPReady + t), p_count[t] & 1)) return false;
      ++p_count[t];
      tc_fence_after();
      const uint64_t db = dRingV + static_cast<uint64_t>((vslot * L::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)
        mma_ts_elect(tO[t], tS[t] + kk * 8,
                     db + static_cast<uint64_t>((kk * 2 * L::kGroupBytes) >> 4), idPV,
                     (!first || kk > 0) ? 1u : 0u);
      mma_commit_elect(bar(L::kBarODone + t));
      return true;
    };
    for (int pos = begin; ok && pos < end;) {
      const Unit u = tree_unit(a, prefix, pos, end);
      const int n = u.j1 - u.j0;
      ok = wait_warp(bar(L::kBarQFull), units & 1);
      if (!ok) break;
      ++units;
      const bool two = !shared_rows && (u.rt + 1) * kBM < a.rows;
      // first score products: key tile 0 (and 1 for the second warpgroup's turn)
      const int lead = shared_rows ? min(2, n) : 1;
      for (int i = 0; ok && i < lead; ++i) {
        int ks;
        ok = next_slot(ks);
        if (!ok) break;
        tc_fence_after();
        issue_s(i, 0, ks);
        if (two) issue_s(1, 1, ks);
        mma_commit_elect(bar(L::kBarKVEmpty + ks));
      }
      for (int i = 0; ok && i < n; ++i) {
        int vs = -1, ks = -1;
        ok = next_slot(vs);
        if (!ok) break;
        if ((u.j0 + i + 1) * kBN > u.len) {
          // the tile's rows behind the sequence's end
          const int r0 = u.len - (u.j0 + i) * kBN;
          uint8_t* v = smem + L::kRing + vs * L::kTileBytes;
          for (int k = lane; k < (kBN - r0) * 8; k += 32) {
            const int row = r0 + k / 8;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              *reinterpret_cast<uint4*>(v + row / 8 * L::kGroupBytes + c * 1024 + row % 8 * 128 +
                                        k % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
        const int t = shared_rows ? i & 1 : 0;
        ok = issue_pv(t, vs, shared_rows ? i < 2 : i == 0);
        if (!ok) break;
        const bool more = i + lead < n && (!shared_rows || lead == 2);
        if (more) {
          ok = next_slot(ks);
          if (!ok) break;
          tc_fence_after();
          issue_s(t, 0, ks);
        }
        if (two) {
          ok = issue_pv(1, vs, i == 0);
          if (!ok) break;
          if (more) issue_s(1, 1, ks);
        }
        // (the unit's last score product is issued: the next unit's rows may be loaded)
        if (i + lead == n - 1 || (i == 0 && n <= lead)) mma_commit_elect(bar(L::kBarQEmpty));
        mma_commit_elect(bar(L::kBarKVEmpty + vs));
        if (ks >= 0) mma_commit_elect(bar(L::kBarKVEmpty + ks));
      }
      if (!ok) break;
      ++o_uses[0];
      if (two || (shared_rows && n > 1)) ++o_uses[1];
      pos += n;
    }
    mma_commit_elect(bar(L::kBarDrain));
    mbar_wait_drain(bar(L::kBarDrain), 0, a.err);
  } else if (warp < 8) {
    regs_inc<kRegsSoftmax>();
    const int t = warp / 4;
    const int copy = (warp % 4) * 32 / kCopyRows;
    const int row0 = (warp % 4) * 32 % kCopyRows;  // the warp's first row of its copy
    const int row = row0 + lane;
    const int col0 = copy * kCols;
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tSrow = tS[t] + lane_off, tOrow = tO[t] + lane_off;
    int s_count = 0, o_count = 0;
    bool ok = true;
    for (int pos = begin; ok && pos < end;) {
      const Unit u = tree_unit(a, prefix, pos, end);
      const int n = u.j1 - u.j0;
      pos += n;
      // the row of the key head's rows (query head x drafted token), and the tiles of this
      // warpgroup: i = i0, i0 + step, ...
      const int tile = u.rt + (shared_rows ? 0 : t);
      const int m_row = tile * kBM + row;
      const int i0 = shared_rows ? t : 0, step = shared_rows ? 2 : 1;
      // the workspace keeps a piece's rows once per warpgroup and copy (shared rows), or two
      // row tiles
      const size_t slot = static_cast<size_t>(u.piece) * a.piece_rows +
                          (shared_rows ? (t * kCopies + copy) * a.rows : t * kBM) + row;
      if (tile * kBM >= a.rows || i0 >= n) {
        // (shared rows, one key tile: this warpgroup's part of the piece is empty)
        if (shared_rows && m_row < a.rows) a.stats[slot] = make_float2(-INFINITY, 0.f);
        continue;
      }
      const bool active = tile * kBM + row0 < a.rows;
      const int tok = m_row % a.T;
      unsigned long long bits = 0;  // drafted tokens that this row sees
      if (m_row < a.rows && tok < u.n) {
        bits = a.tree_mask != nullptr ? a.tree_mask[static_cast<size_t>(u.b) * a.T + tok]
                                      : (2ull << tok) - 1ull;
        if (u.n < 64) bits &= (1ull << u.n) - 1ull;
      }
      float m = -INFINITY, l = 0.f;
      int done = 0;
      for (int i = i0; i < n; i += step, ++done) {
        ok = wait_warp(bar(L::kBarSFull + t), s_count & 1);
        if (!ok) break;
        ++s_count;
        if (!active) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarPReady + t));
          continue;
        }
        tc_fence_after();
        float s[kCols];
        {
          uint32_t sr[kCols];
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tSrow + col0 + c * 32, &sr[c * 32]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = __uint_as_float(sr[c]);
        }
        const int kv0 = (u.j0 + i) * kBN + col0;
        // log2-unit score of entry c: s[c] * unit, or (capped) s[c] q(s[c]^2)
        float unit = a.scale_log2, amax = 0.f;
        bool capped = false;
        const bool tail = kv0 + kCols > u.ctx;
        // drafted tokens are seen by their bits; slots behind the sequence's end have none
        auto hide = [&](float value) {
          if (!tail) return;
#pragma unroll
          for (int q = 0; q < kCols / 32; ++q) {
            const uint32_t w = seen_word(bits, kv0 + 32 * q - u.ctx);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((w >> c) & 1u)) s[32 * q + c] = value;
          }
        };
        if constexpr (kCap) {
          hide(0.f);  // (what lies behind the end does not choose the form)
          amax = abs_max<kCols>(s);
          const bool over = cap_over(amax, a.cap.top);
          capped = !tail && !over;
          if (!capped) {
            if (seldom(over))
              cap_scores_any<kCols>(s, a.cap);
            else
              cap_scores<kCols>(s, a.cap);
            unit = 1.f;
          }
        }
        hide(-INFINITY);
        float m_tile;
        if (kCap && capped) {  // (the score of the largest |s| is a reference as good: cap_args)
          m_tile = a.cap.out * cap_tanh(amax, a.cap);
        } else {
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = s[k];
#pragma unroll
          for (int c = 8; c < kCols; c += 2)
            mx8[(c / 2) % 8] = max3(mx8[(c / 2) % 8], s[c], s[c + 1]);
          m_tile = unit * max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]),
                               fmaxf(mx8[6], mx8[7]));
        }
        float alpha = 1.f;
        bool rescale = false;
        if (m_tile > m + kRescaleThreshold || m == -INFINITY) {
          const float m_new = fmaxf(m, m_tile);
          alpha = (m == -INFINITY) ? 0.f : ex2_approx(m - m_new);
          m = m_new;
          rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale && done > 0)) {
          ok = wait_warp(bar(L::kBarODone + t), (o_count + done - 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(tOrow + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
            tmem_st32(tOrow + c * 32, v);
          }
        }
        l *= alpha;
        const float mref = (m == -INFINITY) ? 0.f : m;
        uint32_t pk[kCols / 2];
        const uint64_t unit2 = f32x2(unit, unit), negm2 = f32x2(-mref, -mref);
        uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
        if (kCap && capped) {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            const uint64_t s2 = f32x2(s[2 * c], s[2 * c + 1]);
            float p0, p1;
            exp2_pair(fma_x2(s2, cap_factor(s2, a.cap), negm2), p0, p1);
            ls2[c % 4] = add_x2(ls2[c % 4], f32x2(p0, p1));
            pk[c] = pack_bf16x2(p0, p1);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            float p0, p1;
            exp2_pair(fma_x2(f32x2(s[2 * c], s[2 * c + 1]), unit2, negm2), p0, p1);
            ls2[c % 4] = add_x2(ls2[c % 4], f32x2(p0, p1));
            pk[c] = pack_bf16x2(p0, p1);
          }
        }
        float ls[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) f32x2_split(ls2[k], ls[2 * k], ls[2 * k + 1]);
        l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
        if constexpr (kCopies == 1) {
          tmem_st32(tSrow, &pk[0]);
          tmem_st32(tSrow + 32, &pk[32]);
        } else {
          // (16 columns of the operand hold 32 keys; the other copies' keys are zeros here)
          uint32_t zero[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) zero[k] = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            constexpr int kOwn = kCols / 32;
            if (k / kOwn != copy) tmem_st16(tSrow + 16 * k, zero);
          }
#pragma unroll
          for (int k = 0; k < kCols / 32; ++k)
            tmem_st16(tSrow + col0 / 2 + 16 * k, &pk[16 * k]);
        }
        tmem_wait_st();
        warp_arrive(bar(L::kBarPReady + t));
      }
      if (!ok) break;
      // the piece's part of the rows: unnormalised output, maximum (log2 units) and sum
      ok = wait_warp(bar(L::kBarODone + t), (o_count + done - 1) & 1);
      if (!ok) break;
      o_count += done;
      tc_fence_after();
      if (active) {
        float* dst = a.parts + slot * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tOrow + c * 32, ov);
          tmem_wait_ld();
          if (m_row < a.rows) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(dst + c * 32 + 4 * k) = make_float4(
                  __uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                  __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
          }
        }
      }
      warp_arrive(bar(L::kBarOFree + t));
      if (m_row < a.rows) a.stats[slot] = make_float2(m, l);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of one row per block: with M the largest maximum,
// O = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p.  Bound by latency: the D / 4 lanes of
// a group go through the group's parts in one pass with a running maximum, kBatch parts'
// statistics and output rows (16 bytes a lane) in flight together, and the groups' results
// are joined in a fixed order.  Few rows take 256 threads each (a long sequence's row has
// hundreds of parts); from kManyRows rows on, whose sequences share the SMs and have few
// parts, 64 threads each.  It is launched while the first kernel runs and waits for its
// results on the device.
constexpr int kManyRows = 1024;
constexpr int kBatch = 4;

template <int D, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads)
    tree_join_kernel(const TreeArgs a, __nv_bfloat16* O, float* LSE, int grid, int copies) {
  constexpr int kLanes = D / 4;                    // threads of one part's row
  constexpr int kGroups = kJoinThreads / kLanes;   // parts read at once
  __shared__ float2 red_s[kGroups];
  __shared__ float4 red_o[kGroups][kLanes];
  const long long out_row = blockIdx.x;  // row of [B][Hkv][rows]
  const int r = static_cast<int>(out_row % a.rows);
  const int bh = static_cast<int>(out_row / a.rows);
  const int b = bh / a.Hkv, head = bh % a.Hkv;
  grid_dependency_wait();
  const int n = a.seqlens_q != nullptr ? a.seqlens_q[b] : a.T;
  const int len = a.cache_lens[b];
  const int before = a.prefix_out[b], after = a.prefix_out[b + 1], total = a.prefix_out[a.B];
  // a row behind the sequence's drafted tokens, or of a sequence out of range: left alone
  if (len < 0 || len > a.max_len || n < 0 || n > a.T || n > len || r % a.T >= n) return;
  const bool shared_rows = a.rows <= kBM;
  const int per_seq = a.Hkv * a.pairs;
  const int share = (total + grid - 1) / grid;
  const int tiles = (after - before) / per_seq;
  const int seg = head * a.pairs + r / (2 * kBM);
  const int first = before + seg * tiles;  // the segment on the line
  const int c0 = first / share, c1 = (first + tiles - 1) / share;
  const int per_piece = shared_rows ? 2 * copies : 1;  // warpgroups x copies of the rows
  const int parts = (c1 - c0 + 1) * per_piece;
  // part p's row: the rows of a piece's parts follow one another, and so do pieces
  const size_t row0 = static_cast<size_t>(c0 + b * per_seq + seg) * a.piece_rows +
                      (shared_rows ? r : r % (2 * kBM));
  const int step = shared_rows ? a.rows : a.piece_rows;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = group; p0 < parts; p0 += kGroups * kBatch) {
    float2 st[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int p = p0 + k * kGroups;
      st[k] = make_float2(-INFINITY, 0.f);
      if (p < parts) {
        const size_t at = row0 + static_cast<size_t>(p) * step;
        st[k] = a.stats[at];
        v[k] = *reinterpret_cast<const float4*>(a.parts + at * D + lane * 4);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, st[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float alpha = ex2_approx(m - ref);
    acc.x *= alpha, acc.y *= alpha, acc.z *= alpha, acc.w *= alpha;
    l *= alpha;
    m = top;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      // (an empty part has -inf and 0; its output row may never have been written)
      if (st[k].y == 0.f) continue;
      const float w = ex2_approx(st[k].x - ref);
      l = fmaf(w, st[k].y, l);
      acc.x = fmaf(w, v[k].x, acc.x);
      acc.y = fmaf(w, v[k].y, acc.y);
      acc.z = fmaf(w, v[k].z, acc.z);
      acc.w = fmaf(w, v[k].w, acc.w);
    }
  }
  if (lane == 0) red_s[group] = make_float2(m, l);
  red_o[group][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  float M = red_s[0].x;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) M = fmaxf(M, red_s[g].x);
  const float ref = M == -INFINITY ? 0.f : M;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float w = ex2_approx(red_s[g].x - ref);
    const float4 v = red_o[g][lane];
    l = fmaf(w, red_s[g].y, l);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that sees no key: 0 and -inf)
  *reinterpret_cast<uint2*>(O + static_cast<size_t>(out_row) * D + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (LSE != nullptr && lane == 0)
    LSE[out_row] = l == 0.f ? -INFINITY : (ref + __log2f(l)) * 0.69314718055994531f;
}

template <int D, bool kCap, int kCopies>
cudaError_t launch_t(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                     void* O, float* LSE, const TreeArgs& a, int num_sms, cudaStream_t stream) {
  auto* kernel = tree_sm100_kernel<D, kCap, kCopies>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = ready_kernel(kernel, kRegsLaunch, Layout<D>::bytes(kTreeMaxBatch), ready);
  if (e != cudaSuccess) return e;
  KernelArgs ka;
  static_cast<TreeArgs&>(ka) = a;
  ka.cap = cap_args(a.scale, a.softcap);
  e = launch_early(kernel, dim3(num_sms), kThreads, Layout<D>::bytes(a.B), stream, true, tmQ, tmK,
                   tmV, ka);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.B) * a.Hkv * a.rows;
  const int threads = rows < kManyRows ? 256 : 64;
  return launch_early(threads == 256 ? tree_join_kernel<D, 256> : tree_join_kernel<D, 64>,
                      dim3(static_cast<unsigned>(rows)), threads, 0, stream, true, a,
                      static_cast<__nv_bfloat16*>(O), LSE, num_sms, kCopies);
}

}  // namespace

cudaError_t launch_tree_sm100(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                              const CUtensorMap& tmV, void* O, float* LSE, const TreeArgs& a,
                              int d, int num_sms, cudaStream_t stream) {
  auto launch = [&](auto* k) { return k(tmQ, tmK, tmV, O, LSE, a, num_sms, stream); };
  switch (tree_copies(a.rows) * 4 + (d == 128) * 2 + (a.softcap > 0.f)) {
    case 4: return launch(launch_t<64, false, 1>);
    case 5: return launch(launch_t<64, true, 1>);
    case 6: return launch(launch_t<128, false, 1>);
    case 7: return launch(launch_t<128, true, 1>);
    case 8: return launch(launch_t<64, false, 2>);
    case 9: return launch(launch_t<64, true, 2>);
    case 10: return launch(launch_t<128, false, 2>);
    case 11: return launch(launch_t<128, true, 2>);
    case 16: return launch(launch_t<64, false, 4>);
    case 17: return launch(launch_t<64, true, 4>);
    case 18: return launch(launch_t<128, false, 4>);
    default: return launch(launch_t<128, true, 4>);
  }
}

}  // namespace fa
