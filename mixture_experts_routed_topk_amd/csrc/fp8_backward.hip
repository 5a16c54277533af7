// e4m3 products with block scales, the two gradients in one launch (gfx950).  fp8_tile.h has the tiles.
//
// dx = dz w reads the weights along their rows, as they are stored, and applies their block scales; dw = dz^T x reads
// both operands along their rows.  dz's and x's scales are powers of two, so dw's MFMAs apply all scales
// themselves, and dx's too with UE8M0 weights.
//
// One launch: the product with the shorter tiles fills the CUs that the other's last round leaves (Fill, Share).  2731 rows, 2048 <- 5632:
// 91 us, against 62 and 43 in two launches.
#include "dense_tile.h"
#include "fp8_tile.h"

namespace moe {
namespace {

template <int NX, int NW>
void launch_pair(const Fp8Job& dx, const Fp8Job& dw, Fill fill, bool fold, dim3 grid, hipStream_t s) {
  if (fold) hipLaunchKernelGGL((fp8_gradients_kernel<NX, NW, true>), grid, dim3(512), 0, s, dx, dw, fill);
  else hipLaunchKernelGGL((fp8_gradients_kernel<NX, NW, false>), grid, dim3(512), 0, s, dx, dw, fill);
}

// Rows of the tiles by runs; dw's rows are the weights'.  Backward passes of 8 to 64 runs, with dw's other height: 512 -> 640, 384: equal, 1 to 4%
// faster with 128; 2048 -> 1408, 4096 -> 2048: 3 to 10% faster with 256.  With dx's: 256 rows a run on average: equal to 8%
// faster with 128; 512: 3 to 8% faster with 256 but for 512 columns (3% slower).
int dw_height(int64_t cols) { return cols % 256 == 0 || cols > 1024 ? 256 : 128; }

// us of a slice of dx (block scales folded by fmas, or applied by the MFMAs) and of dw, by tile height 256 or 128, of a tile
// besides, and of the splits' sum.  Fitted to 54 backward passes of 136 to 16384 rows, each measured with every pair of heights and
// most splits (rms error 6%; the choices take 0.3% longer than the best measured, 12% at most).
constexpr double kSlice[3][2] = {{1.83, 1.06}, {1.33, 0.96}, {1.51, 0.90}};
constexpr double kFixed[2] = {6.0, 4.3};
constexpr JoinCost kJoinGradients = {5.9, 5.6e6};
int kind_of(int product, bool fold) { return product ? 2 : fold ? 0 : 1; }

// The longest time of a workgroup when `tiles` of `us` each are shared as fp8_gradients_kernel does
double shared_time(const int64_t (&tiles)[2], const double (&us)[2], Fill* fill) {
  Fill f{};
  f.dw = us[1] < us[0] || !tiles[0];
  if (!tiles[1]) f.dw = 0;
  const int a = !f.dw, b = f.dw;                  // b fills
  const int64_t G = fp8_grid(tiles[0] + tiles[1]).x, heavy = tiles[a] % G;
  f.extra = (int)(us[a] / us[b] + 0.5);
  f.others_first = f.extra * us[b] <= us[a];
  *fill = f;
  if (!heavy) f = Fill{f.dw, 0, 0};               // (as the kernel has it, which counts a's tiles itself)
  const int64_t early = f.extra * (G - heavy), late = tiles[b] > early ? tiles[b] - early : 0;
  const double whole = (tiles[a] / G) * us[a], rounds = (late / G) * us[b];
  const int64_t rest = late % G, firsts = f.others_first ? G - heavy : heavy;    // workgroups that the last round begins with
  // loads of those with a tile of a more and of the others, the last round apart
  const int64_t sent = tiles[b] < early ? tiles[b] : early;
  const double load_h = whole + (heavy ? us[a] : 0) + rounds, load_o = whole + (G > heavy ? (double)((sent + G - heavy - 1) / (G - heavy)) * us[b] : 0) + rounds;
  const double first = f.others_first ? load_o : load_h, second = f.others_first ? load_h : load_o;
  double longest = fmax(heavy ? load_h : 0, load_o);
  if (rest) longest = fmax(longest, (firsts ? first : second) + us[b]);
  if (rest > firsts) longest = fmax(longest, second + us[b]);
  return longest;
}

// The tile heights and splits of the two products over one matrix with the least estimated time
struct Gradients {
  int height[2], splits[2], slices[2];
  Fill fill;
};
Gradients plan_of(int64_t T, int64_t N, int64_t cols, bool dx, bool dw, bool fold) {
  const int64_t M[2] = {dx ? T : 0, dw ? cols : 0}, KT[2] = {cols / 128, (T + 127) / 128}, nt = (N + 255) / 256;
  constexpr int kTry[] = {1, 2, 4, 8, 16};
  Gradients best{};
  double best_us = 1e30;
  for (int pair = 0; pair < 4; ++pair)
    for (int a : kTry)
      for (int b : kTry) {
        Gradients g{{pair & 2 ? 128 : 256, pair & 1 ? 128 : 256}, {a, b}, {}, {}};
        int64_t tiles[2];
        double us[2], joined = 0;
        bool ok = true;
        for (int i = 0; i < 2; ++i) {
          const int64_t whole = (M[i] + g.height[i] - 1) / g.height[i] * nt;
          // (too short, or no need)
          if (g.splits[i] > 1 && (!M[i] || KT[i] / g.splits[i] < 3 || whole >= 512)) ok = false;
          g.slices[i] = (int)((KT[i] + g.splits[i] - 1) / g.splits[i]);
          g.splits[i] = (int)((KT[i] + g.slices[i] - 1) / g.slices[i]);        // (every split has slices)
          tiles[i] = whole * g.splits[i];
          us[i] = g.slices[i] * kSlice[kind_of(i, fold)][g.height[i] == 128] + kFixed[g.height[i] == 128];
          if (g.splits[i] > 1) joined += (double)M[i] * N * 4 * (g.splits[i] + 1);
        }
        if (fold && g.height[0] == 128 && g.slices[0] > kLongestShortTile) ok = false;      // (its block scales do not fit)
        if (!ok) continue;
        double time = shared_time(tiles, us, &g.fill);
        if (joined > 0) time += kJoinGradients.us + joined / kJoinGradients.bytes_per_us;
        if (time < best_us) best_us = time, best = g;
      }
  return best;
}
size_t part_bytes(const Gradients& p, int i, int64_t M, int64_t N) {
  return p.splits[i] > 1 ? ((size_t)p.splits[i] * M * N * 4 + 255) & ~size_t(255) : 0;
}

}  // namespace

int fp8_dx_height(int64_t T, int E, int64_t cols, bool ue8m0) {
  return T >= (int64_t)384 * E || (!ue8m0 && cols / 128 > kLongestShortTile) ? 256 : 128;
}

size_t fp8_gradients_workspace(int64_t T, int64_t N, int64_t cols, int E) {
  if (T == 0 || E) return 0;
  size_t most = 0;
  for (int which = 2; which < 8; ++which) {        // dx, dw or both may be asked for, with either kind of scales
    const Gradients p = plan_of(T, N, cols, which & 2, which & 4, which & 1);
    const size_t need = part_bytes(p, 0, which & 2 ? T : 0, N) + part_bytes(p, 1, which & 4 ? cols : 0, N);
    most = need > most ? need : most;
  }
  return most;
}

hipError_t launch_fp8_gradients(const Fp8Gemm* dx, const Fp8Gemm* dw, void* ws, hipStream_t s) {
  const Fp8Gemm* g[2] = {dx, dw};
  const Fp8Gemm& any = dx ? *dx : *dw;
  const int64_t N = any.g.e.N;
  const bool fold = dx && !dx->cs.bytes;
  Fp8Job job[2] = {};
  int tile[2] = {256, 256};
  int64_t tiles[2] = {};
  Job sum[2] = {};
  int join_blocks[2] = {};
  Gradients plan{};
  if (!any.E) plan = plan_of(dx ? dx->g.M : dw->g.K, N, dx ? dx->g.K : dw->g.M, dx, dw, fold);
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    if (!g[i]) continue;
    Job j{};
    j.g = g[i]->g;
    j.crows = (int)N;
    j.nt = (int)((N + 255) / 256);
    if (any.E) {
      tile[i] = i ? dw_height(j.g.M) : any.runs.height;
      j.splits = 1;
      j.slices = (int)(j.g.K / 128);
      j.mt = i ? (int)((j.g.M + tile[i] - 1) / tile[i]) : (int)max_row_tiles(j.g.M, any.E, tile[i]);
    } else {
      tile[i] = plan.height[i];
      j.splits = plan.splits[i];
      j.slices = plan.slices[i];
      j.mt = (int)((j.g.M + tile[i] - 1) / tile[i]);
      if (j.splits > 1) {
        j.part = reinterpret_cast<float*>(static_cast<char*>(ws) + at);
        j.ldpart = N;
        at += part_bytes(plan, i, j.g.M, N);
        sum[i] = j;
        join_blocks[i] = (int)((j.g.M * (N / 8) + 255) / 256);
      }
    }
    job[i] = fp8_job(*g[i], j);
    tiles[i] = (int64_t)j.mt * j.nt * (any.E && i ? any.E : j.splits);
  }
  if (any.E) {
    // (how many rows a run has is not known here: an average)
    double us[2];
    for (int i = 0; i < 2; ++i)
      us[i] = (i ? (double)job[1].j.slices / any.E : job[0].j.slices) * kSlice[kind_of(i, fold)][tile[i] == 128] + kFixed[tile[i] == 128];
    shared_time(tiles, us, &plan.fill);
  }
  const dim3 grid = fp8_grid(tiles[0] + tiles[1]);
  if (tile[0] == 256 && tile[1] == 256) launch_pair<2, 2>(job[0], job[1], plan.fill, fold, grid, s);
  else if (tile[0] == 256) launch_pair<2, 1>(job[0], job[1], plan.fill, fold, grid, s);
  else if (tile[1] == 256) launch_pair<1, 2>(job[0], job[1], plan.fill, fold, grid, s);
  else launch_pair<1, 1>(job[0], job[1], plan.fill, fold, grid, s);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !(join_blocks[0] + join_blocks[1])) return err;
  hipLaunchKernelGGL(dense_join_pair_kernel<uint16_t>, dim3((unsigned)(join_blocks[0] + join_blocks[1])), dim3(256), 0, s, sum[0], sum[1],
                     join_blocks[0]);
  return hipGetLastError();
}

}  // namespace moe
