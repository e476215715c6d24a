// Which kernel runs a product, and in how many parts of K: a model of the
// kernels' times, fitted to sweeps on one MI355X.  It compares kernels with one
// another; the rate of memory and the host's share are left out.
#include <math.h>

#include "launch_products.h"

namespace fp8moe {

namespace {

constexpr int kMaxSplits = 8, kPartSteps = 8;      // parts of K, and the fewest steps of one
constexpr size_t kMaxPartial = (size_t)16 << 20;   // the parts' sums stay in the last-level cache

// us of a K step of one workgroup with TS sub-tiles a wave (base + per * TS), of
// a round's start and end, and how many workgroups share a CU, each then taking
// `shared` times as long.  Dense products, row-major, us (model | measured, 256 x
// 256, 256 x 128, 128 x 128, 128 x 64; 128 x 128 of eight waves):
//   8192 x 4096 x 7168: 250, 287, 321, 435; 343 | 240, 282, 281, 349; 341
//   2048 x 4096 x 7168: 127, 75, 83, 112; 89 | 111, 74, 74, 95; 87
//   1111 x 4096 x 7168: 118, 75, 75, 85; 89 | 104, 64, 66, 72; 79
//   4096 x 7168 x 2048: 82, 92, 88, 117; 99 | 78, 91, 87, 105; 101
//   512 x 7168 x 2048:  43, 26, 23, 20; 17.5 | 37, 24, 21, 18.6; 16.4
//   512 x 1500 x 7168:  127, 75, 65, 40; 46 | 129, 77, 65, 38; 49
//   2048 x 1500 x 7168: 127, 75, 65, 54; 46 | 130, 77, 65, 53; 49
//   1111 x 2000 x 1936: 40, 26, 23, 18; 17.5 | 37, 25, 20, 18; 16
// grouped, MFMA-tiled:
//   256 groups of 256 rows, 7168 x 2048: 1403, 1545, 1687, 2035; 1897 | 1402, 1590, 1551, 1879; 1929
//   128 of 256, 1536 x 2048: 171, 180, 184, 222; 207 | 178, 189, 183, 213; 221
//   128 of 100, 1536 x 2048: 88, 70, 76, 109; 85 | 103, 101, 100, 114; 110 (its weights alone take 75)
//   8 of 160, 4096 x 4096:   60, 41, 45, 51; 54 | 61, 48, 48, 55; 53
//
// The rate of memory: few rows of large weights take longer than the model says
// with every kernel, and the one it picks is within a tenth of the best.  Row-major,
// us of 1, 8, 33, 64 rows, streaming 32 weight rows in one part | 128 x 64 in the
// parts that are picked:
//   36864 x 7168 (43 at the rate of a long read): 49, 54, 100, 141 | 54, 55, 65, 72
//   7168 x 18432 (22):                            27, 30, 49, 71   | 30, 31, 34, 38
//   65536 x 2048 (22):                            28, 30, 58, 79   | 25, 26, 28, 30
// The host: a call in parts makes two launches, which the model counts as the GPU
// does.  512 x 7168, streaming 16 weight rows, one | four parts, us in a graph: one
// row 7.0 | 6.1, MFMA-tiled 5.4 | 5.6; 16 rows 10.6 | 7.5, tiled 8.4 | 6.9; outside
// of graphs 7.4 | 10.0, 7.2 | 10.0; 10.6 | 10.2, 8.4 | 10.2.
struct TileCost {
  ProductShape shape;
  int tn, tm, wm, per_cu;
  float base, per, shared, ends;
};
constexpr TileCost kTiles[] = {
    {kTile128x64, 128, 64, 2, 2, 0.43f, 0.10f, 1.5f, 1.0f},
    {kTile128x128x8, 128, 128, 4, 1, 0.44f, 0.14f, 1.0f, 2.0f},
    {kTile128x128, 128, 128, 2, 2, 0.72f, 0.085f, 1.3f, 2.0f},
    {kTile256x128, 256, 128, 2, 1, 0.62f, 0.15f, 1.0f, 2.5f},
    {kTile256x256, 256, 256, 2, 1, 0.75f, 0.17f, 1.0f, 5.0f},
};
constexpr float kLaunch = 4.f;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `groups` groups of about `share` rows each.  Chance gives some of them more
// rows than the average: where the average comes near a tile's height they need
// one tile more, on average a half.
float tile_us(const TileCost& c, int64_t groups, int64_t share, int N, int steps, int splits, int num_cu) {
  float cut = (float)ceil_div(share, c.tm);
  if (groups > 1 && share + 2 * sqrtf((float)share) > c.tm) cut = fmaxf(1.f, (float)share / c.tm + 0.5f);
  const float ts = fminf((float)(c.tm / (16 * c.wm)), ceilf(share / cut / (16 * c.wm)));
  const float tiles = groups * cut * ceil_div(N, c.tn) * splits, cus = (float)num_cu;
  float step = c.base + c.per * ts, rounds;
  if (c.per_cu == 1) {
    rounds = ceilf(tiles / cus);
  } else {
    if (tiles > cus) step *= 1.f + (c.shared - 1.f) * (0.5f + 0.5f * fminf(1.f, tiles / cus - 1.f));
    rounds = fmaxf(1.f, ceilf(tiles / cus) / 2);
  }
  return kLaunch + rounds * (ceil_div(steps, splits) * step + c.ends);
}

// writing the parts' sums, reading them, and the launch between
float join_us(int64_t rows, int N, int splits) { return splits > 1 ? 3.f + 2e-6f * splits * rows * N : 0.f; }

}  // namespace

size_t partial_bytes(int64_t rows, int N, int steps) {
  if (steps < 2 * kPartSteps || rows == 0) return 0;
  const size_t n = (size_t)(rows < (int64_t)kMaxPartial ? rows : (int64_t)kMaxPartial) * ((N + 7) & ~7) * sizeof(float) *
                   kMaxSplits;
  return n < kMaxPartial ? (n + 255) / 256 * 256 : kMaxPartial;
}

ProductPlan plan_product(int64_t rows, int N, int steps, int E, int num_cu) {
  const bool grouped = E > 0;
  const int64_t groups = grouped ? (rows < E ? rows : E) : 1;
  const int64_t share = ceil_div(rows, groups);
  const int64_t small = groups * ceil_div(N, 128);   // workgroups of 128 x 64 tiles where each group is one
  // Groups of a few rows: streaming where weights are read once for them, or
  // tiles would be few.  128 groups, 1536 x 2048, tiled, us, streaming | 128 x 64:
  // 4 rows 69, 71, 12 rows 77, 74, 24 rows 106, 78; 2 rows in bf16 67, 79; 8
  // groups of 4 rows, 4096 x 4096: 27, 28.
  if (grouped && (share <= 4 || (share <= 16 && small < num_cu))) return {kStream, 2, 1, 1};
  auto fits = [&](int s) {
    return s == 1 || (!grouped && steps >= kPartSteps * s && (size_t)rows * ((N + 7) & ~7) * s * sizeof(float) <= kMaxPartial);
  };
  ProductPlan best{kTile256x256, 0, 0, 1};
  float us = 1e30f;
  for (const TileCost& c : kTiles) {
    // tiles are numbered in 31 bits (256 x 256 ones of 2^30 rows and 2^16 columns fit)
    if ((rows / c.tm + groups + 64) * ceil_div(N, c.tn) >= (int64_t)1 << 31) continue;
    for (int s = 1; s <= (c.shape == kTile128x64 || c.shape == kTile128x128x8 ? kMaxSplits : 1); s *= 2) {
      if (!fits(s)) continue;
      const float t = tile_us(c, groups, share, N, steps, s, num_cu) + join_us(rows, N, s);
      if (t < us) us = t, best = {c.shape, 0, 0, s};
    }
  }
  if (grouped || rows > 1024) return best;
  // Streaming: what a step of 16 or 32 weight rows by 16 ts rows takes a CU.
  const int64_t cut = ceil_div(rows, 64);
  const int ts = (int)ceil_div(ceil_div(rows, cut), 16);
  for (int bands = 1; bands <= 2; ++bands) {
    const float step = bands == 1 ? 0.06f + 0.07f * ts : 0.09f + 0.09f * ts;
    for (int s = 1; s <= kMaxSplits; s *= 2) {
      if (!fits(s)) continue;
      const float wgs = (float)(cut * ceil_div(N, 16 * bands) * s);
      const float t = kLaunch + ceilf(wgs / num_cu) * ceil_div(steps, s) * step + join_us(rows, N, s);
      if (t < us) us = t, best = {kStream, bands, ts, s};
    }
  }
  return best;
}

ProductTileSize product_tile_size(const ProductPlan& plan, bool grouped) {
  for (const TileCost& c : kTiles)
    if (c.shape == plan.shape) return {c.tn, c.tm, c.tn / 64 * c.wm};
  return {16 * plan.bands, 16 * plan.sub_tiles, grouped ? 4 : 8};
}

hipError_t launch_product(const ProductArgs& P, const ProductPlan& plan, hipStream_t stream) {
  const hipError_t err = plan.shape == kStream ? launch_product_stream(P, plan.bands, plan.sub_tiles, stream)
                                               : launch_product_tile(P, plan.shape, stream);
  if (err != hipSuccess || P.splits == 1) return err;
  return launch_product_join(P, stream);
}

}  // namespace fp8moe
