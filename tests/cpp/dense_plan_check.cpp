// Prints the tiles and splits the dense operators choose.  Each line of the input is a forward product
// "fwd bf16|f32 M N K gated" -> "tile_rows splits halves", or the gradients of T rows
// "grad bf16|f32 T K cols" -> "dx_tile_rows dw_tile_rows dx_splits dw_splits".
#include <cstdio>
#include <cstring>

#include "dense_plan.h"

using namespace moe;

int main() {
  char kind[8], type[8];
  long long a, b, c;
  while (std::scanf("%7s %7s %lld %lld %lld", kind, type, &a, &b, &c) == 5) {
    const bool f32 = !std::strcmp(type, "f32");
    if (!std::strcmp(kind, "fwd")) {
      int gated = 0;
      if (std::scanf("%d", &gated) != 1) return 1;
      const Plan p = f32 ? plan_f32(a, b, c, gated) : plan_bf16(a, b, c, gated);
      const int cols = p.tile == 256 ? 256 : 128;
      const int64_t tiles = (a + p.tile - 1) / p.tile * (((gated ? 2 * b : b) + cols - 1) / cols);
      std::printf("%d %d %d\n", p.tile, p.splits, p.splits == 1 && whole_tiles(p.tile, tiles) < tiles);
    } else {
      const int64_t M[2] = {a, c}, K[2] = {c, a};
      const PairPlan p = f32 ? plan_pair<float>(kPairsF32, kPairTilesF32, kJoinF32, M, b, K)
                             : plan_pair<uint16_t>(kPairsBf16, kPairTilesBf16, kPairJoinBf16, M, b, K);
      const TileCost* t = f32 ? kPairTilesF32 : kPairTilesBf16;
      const int* pair = f32 ? kPairsF32[p.tiles] : kPairsBf16[p.tiles];
      std::printf("%d %d %d %d\n", t[pair[0]].rows, t[pair[1]].rows, p.splits[0], p.splits[1]);
    }
  }
  return 0;
}
