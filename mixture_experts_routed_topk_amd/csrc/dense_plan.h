// Choice of tiles and splits of the dense operators' matrix products: host code without HIP, so that it can be
// compiled and looked at by itself.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {
namespace {

template <typename T>
constexpr int ks() { return 128 / (int)sizeof(T); }   // k per slice

struct Plan {
  int tile;      // rows of a tile
  int splits;
  int slices;    // per split
};
struct TileCost {
  int rows, cols, per_cu;
  double alone, shared, fixed;
};
struct JoinCost {
  double us, bytes_per_us;
};
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};

// The last round of 256-row tiles runs as halves when those find a CU each (8192 x 2048 x 7168, 3.5 rounds:
// 247 -> 235 us a call, 277 -> 267 in calls back to back; 0.7 to 0.8 of a whole tile's time).  The plan does not count on it: in 16 of 16 products where
// that would have moved the choice from 128-row tiles these stayed faster, by 1 to 14%.
inline int64_t whole_tiles(int rows, int64_t tiles) { return rows == 256 && tiles % 256 <= 128 ? tiles / 256 * 256 : tiles; }

// The tile and split of a forward product with the least estimated time.  Tiles go over the 256 CUs in
// rounds of the workgroups that a CU holds; a slice takes a workgroup at least `alone` us, and `shared`
// us of its CU; `fixed` us go to a tile's first DMA and epilogue, and a split adds a second launch
// and a pass over its partial sums.
template <typename T, int NT>
Plan plan_forward(const TileCost (&costs)[NT], JoinCost joined, int64_t M, int64_t N, int64_t K, int gated) {
  const int64_t cols = gated ? 2 * N : N;
  const int64_t KT = (K + ks<T>() - 1) / ks<T>();
  Plan best{128, 1, (int)KT};
  double best_us = 1e30;
  for (const TileCost& t : costs) {
    const int64_t tiles = ((M + t.rows - 1) / t.rows) * ((cols + t.cols - 1) / t.cols);
    for (int want : kSplits) {
      if (want > 1 && KT / want < 3) break;
      const int64_t per = (KT + want - 1) / want;
      const int s = (int)((KT + per - 1) / per);      // (every split has slices)
      const int64_t queue = (tiles * s + 255) / 256;  // workgroups of one CU
      const int64_t rest = queue % t.per_cu;
      double us = (queue / t.per_cu) * (per * fmax(t.alone, t.per_cu * t.shared) + t.fixed);
      if (rest) us += per * fmax(t.alone, rest * t.shared) + t.fixed;
      if (s > 1) us += joined.us + (double)M * cols * 4 * (s + 1) / joined.bytes_per_us;
      if (us < best_us) best_us = us, best = Plan{t.rows, s, (int)per};
    }
  }
  return best;
}
inline int64_t part_pitch(int64_t N, int gated) { return ((gated ? 2 * N : N) + 7) / 8 * 8; }

// Bytes of partial sums of a forward product: of a split contraction, and of an output whose rows
// cannot be stored in pieces
inline size_t forward_part(const Plan& p, int64_t M, int64_t N, int gated, int vec) {
  return p.splits > 1 || !vec ? (size_t)p.splits * M * part_pitch(N, gated) * 4 : 0;
}

// ---------------------------------------------------------------------------- plan of the gradients
struct PairPlan {
  int tiles;                     // index into the pairs of tiles
  int splits[2], slices[2];      // dx, dw
};
// dx [M0][N] over K0 and dw [M1][N] over K1; a product with no rows is left out.  Their tiles share
// the CUs: the time is the work of all of them over 256 CUs, at least the longest tile's own,
// and half a tile more for the uneven end.
template <typename T, int NP, int NT>
PairPlan plan_pair(const int (&pairs)[NP][2], const TileCost (&costs)[NT], JoinCost joint, const int64_t (&M)[2], int64_t N, const int64_t (&K)[2]) {
  constexpr int kTry[] = {1, 2, 4, 8, 16};
  PairPlan best{0, {1, 1}, {1, 1}};
  double best_us = 1e30;
  for (int t = 0; t < NP; ++t) {
    for (int a : kTry) {
      for (int b : kTry) {
        PairPlan p{t, {a, b}, {1, 1}};
        double work = 0, longest = 0, shortest = 1e30, joined = 0;
        bool ok = true;
        for (int j = 0; j < 2; ++j) {
          const int want = j ? b : a;
          if (M[j] == 0 || K[j] == 0) {
            p.splits[j] = 1;
            ok = ok && want == 1;
            continue;
          }
          const TileCost& c = costs[pairs[t][j]];
          const int64_t KT = (K[j] + ks<T>() - 1) / ks<T>();
          const double whole = (double)((M[j] + c.rows - 1) / c.rows) * ((N + c.cols - 1) / c.cols);
          if (want > 1 && (KT / want < 3 || whole >= 512)) {   // (too short, or no need)
            ok = false;
            break;
          }
          const int64_t per = (KT + want - 1) / want;
          p.splits[j] = (int)((KT + per - 1) / per);
          p.slices[j] = (int)per;
          const double tiles = whole * p.splits[j];
          work += tiles * (per * c.shared + c.fixed);
          const double own = per * c.alone + c.fixed;
          longest = fmax(longest, own);
          shortest = fmin(shortest, own);
          if (p.splits[j] > 1) joined += (double)M[j] * N * 4 * (p.splits[j] + 1);
        }
        if (!ok) continue;
        double us = fmax(work / 256 + 0.47 * shortest, longest);
        if (joined > 0) us += joint.us + joined / joint.bytes_per_us;
        if (us < best_us) best_us = us, best = p;
      }
    }
  }
  return best;
}
// bytes of the partial sums of product j; two_parts: two rows of dx's product add up to one
inline size_t pair_part(const PairPlan& p, int j, int64_t M, int64_t N, bool two_parts) {
  return p.splits[j] > 1 || (two_parts && j == 0) ? ((size_t)p.splits[j] * M * N * 4 + 255) & ~size_t(255) : 0;
}

template <typename T, int NP, int NT>
size_t gradients_part(const int (&pairs)[NP][2], const TileCost (&costs)[NT], JoinCost joint, int64_t rows, int64_t N,
                      int64_t cols, bool two_parts) {
  size_t most = 0;
  for (int which = 1; which < 4; ++which) {        // dx, dw or both may be asked for
    const int64_t M[2] = {which & 1 ? rows : 0, which & 2 ? cols : 0}, K[2] = {cols, rows};
    const PairPlan p = plan_pair<T>(pairs, costs, joint, M, N, K);
    const size_t need = pair_part(p, 0, M[0], N, two_parts) + pair_part(p, 1, M[1], N, two_parts);
    most = need > most ? need : most;
  }
  return most;
}

// ---------------------------------------------------------------------------- costs, bf16
// Fitted to 43 products of 60 to 8192 rows on operands that stay in the caches, each measured with every tile and
// split (rms error of the estimate 13%; the choices take 1.6% longer than the best ones).  `shared` of the 128-row tiles
// is 8% above its fit: they draw twice the operands of the 256-row ones, which shows when operands come from HBM.
// Over 152 products of 137 to 8192 rows with other operands at every call, half of them drawn where the choice hangs on
// this figure, the tiles chosen take 5.3% longer than the best measured with 0.38, and 5.6% with the fit's 0.352, 5.6% with
// 0.39, 6.6% with 0.40 and 7.2% with 0.41 (there 128-row tiles give way to 64-row ones that are slower by 15%).
constexpr TileCost kTilesBf16[] = {{256, 256, 1, 1.115, 1.115, 7.0}, {128, 128, 2, 0.549, 0.38, 0.57}, {64, 128, 3, 0.328, 0.251, 0.02}};
constexpr JoinCost kJoinBf16 = {2.8, 3.36e6};

// The gradients' tiles: pairs for dx and dw.  Fitted to 23 backward passes with every pair of tiles
// and splits (rms error 12%, choices 1% longer than the best; here the 64-row tiles
// have the LDS of the 128-row ones, two to a CU).
constexpr TileCost kPairTilesBf16[] = {{256, 256, 1, 1.31, 1.21, 4.8}, {128, 128, 2, 0.638, 0.343, 0.82}, {64, 128, 2, 0.512, 0.405, 0.04}};
constexpr int kPairsBf16[][2] = {{0, 0}, {1, 1}, {2, 1}};
constexpr JoinCost kPairJoinBf16 = {3.7, 3.3e6};

inline Plan plan_bf16(int64_t M, int64_t N, int64_t K, int gated) {
  return plan_forward<uint16_t>(kTilesBf16, kJoinBf16, M, N, K, gated);
}

// ---------------------------------------------------------------------------- costs, float32
// (a slice's MFMAs alone: 32 x RR x 128 products at 256 flops a cycle, 1.7 us of 128 rows at 2.4 GHz)
constexpr TileCost kTilesF32[] = {{128, 128, 2, 1.9, 1.9, 3.0}, {64, 128, 3, 1.0, 1.0, 2.0}, {32, 128, 3, 0.6, 0.55, 2.0}};
constexpr JoinCost kJoinF32 = {3.5, 3.3e6};
constexpr TileCost kPairTilesF32[] = {{128, 128, 2, 1.9, 1.9, 3.0}, {64, 128, 2, 1.0, 1.0, 2.0}, {32, 128, 2, 0.6, 0.55, 2.0}};
constexpr int kPairsF32[][2] = {{0, 0}, {1, 0}, {2, 0}};

inline Plan plan_f32(int64_t M, int64_t N, int64_t K, int gated) {
  return plan_forward<float>(kTilesF32, kJoinF32, M, N, K, gated);
}

}  // namespace
}  // namespace moe
