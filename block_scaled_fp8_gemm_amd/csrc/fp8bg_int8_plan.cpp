// The int8 products' choice of a kernel configuration (pure host code).
#include <math.h>

#include "fp8bg.h"
#include "fp8bg_int8_configs.h"

namespace fbg {

namespace {

enum Kind { ANY, SKINNY, SLIM, TILE };

// What a configuration costs, in microseconds: `start` once per workgroup and
// `step` per 128 bytes of K, rising from `step` for one workgroup alone to
// `full` with `per_cu` on every compute unit; past that the rounds queue up,
// and `again` is the share of `start` that a queued round still shows.
// Least-squares fits in the logarithm to 167 dense shapes of M 1 .. 16384, N
// 64 .. 8192 and K 256, 1024 and 4096 (configurations 2-12, 16-byte rows; the
// fits' own deviation is 4-11%) and to 79 of the same range with odd K (any
// rows, contiguous, from before the output stores took any alignment; 9-22%),
// `per_cu` being the count that fits best, not an occupancy.  Choosing by it
// costs 1.4% over the best configuration of each shape on average and 13% at
// worst, as the kernels are now (any rows: 1.9% and 19%).
struct Cost {
  Kind kind;
  int rows, cols, per_cu, waves;
  float start, step, full, again;
};
constexpr Cost kFast[kNumI8Cfgs] = {
    {ANY, 64, 64, 4, 4, 0, 0, 0, 0},
    {ANY, 32, 64, 4, 4, 0, 0, 0, 0},
    {SKINNY, 8, 16, 8, 8, 2.400f, 0.072f, 0.747f, 0.590f},
    {SKINNY, 16, 16, 8, 8, 2.385f, 0.084f, 0.904f, 0.652f},
    {SKINNY, 16, 32, 8, 4, 2.351f, 0.146f, 1.365f, 0.969f},
    {TILE, 32, 64, 3, 2, 2.614f, 0.213f, 0.437f, 0.737f},
    {TILE, 64, 64, 2, 4, 2.828f, 0.238f, 0.447f, 0.667f},
    {TILE, 64, 128, 2, 4, 3.343f, 0.280f, 0.697f, 0.841f},
    {TILE, 128, 128, 2, 4, 3.959f, 0.511f, 1.221f, 0.968f},
    {TILE, 128, 256, 1, 4, 7.084f, 0.546f, 0.968f, 0.925f},
    {TILE, 256, 256, 1, 4, 11.821f, 0.976f, 1.581f, 0.975f},
    {SLIM, 32, 32, 2, 4, 2.504f, 0.091f, 0.226f, 0.727f},
    {SLIM, 32, 32, 3, 4, 2.521f, 0.130f, 0.331f, 0.857f},
};
constexpr Cost kAny[kI8FirstTile] = {
    {ANY, 64, 64, 2, 4, 4.149f, 0.391f, 0.922f, 0.983f},
    {ANY, 32, 64, 1, 4, 3.584f, 0.299f, 0.316f, 0.578f},
    {SKINNY, 8, 16, 2, 8, 3.019f, 0.178f, 0.537f, 0.250f},
    {SKINNY, 16, 16, 1, 8, 3.066f, 0.223f, 0.304f, 0.216f},
    {SKINNY, 16, 32, 1, 4, 3.141f, 0.401f, 0.487f, 0.285f},
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

double estimate(const Cost& c, double tiles, int64_t steps, int cus) {
  const double cap = (double)cus * c.per_cu;
  if (tiles <= cap) return c.start + steps * (c.step + (c.full - c.step) * (tiles / cap));
  return ceil(tiles / cus) / c.per_cu * (c.start * c.again + steps * c.full);
}

const Cost& cost(int cfg, bool fast) { return fast ? kFast[cfg] : kAny[cfg]; }

}  // namespace

int int8_cfg_for(int64_t E, int64_t M, int64_t N, int64_t K, bool fast, int cus) {
  const int64_t steps = ceil_div(K, 128);
  int first = fast ? kI8FirstSkinny : 0, end = fast ? kNumI8Cfgs : kI8FirstTile;
  const double mean = E > 0 ? (double)M / (double)E : 0.0;
  if (E > 0 && mean <= 12.0) {
    // Small experts: the weights of those that hold rows are what is read.
    // 16-byte rows: over a long K the slim kernel streams them best (64 tokens,
    // 8 of 256 experts of 512 x 4096: 79 us, 5.8 TB/s, skinny 83, 32 x 64 tile
    // 97; 8 rows to an expert on average 88 us, 105 and 110), and the skinny one
    // while that makes at most two workgroups per compute unit (8 experts of
    // 1-8 rows: 5.5-6.1 us, slim 8.5, the tile 10.7); over a short K the tile
    // does (of 1536 x 1024: 64 us, slim 79, skinny 71).  Any rows: the
    // 32-column skinny form up to a few workgroups per compute unit (64 rows
    // over 8 experts of 515 x 776: 3.8 us, the 32 x 64 tile 5.1), else the
    // 32 x 64 tile (256 experts: 27.7 us against 32.9).
    if (!fast) return E * ceil_div(N, 32) <= 4 * cus ? 4 : 1;
    if (K < 2048) return 5;
    return E * ceil_div(N, 16) > 2 * cus || mean > 8.0 ? 12 : mean > 4.0 ? 3 : 2;
  }
  // Up to four rows: the skinny tile's other rows repeat them, so that it reads
  // less than the fit, made over full tiles, supposes.  With at most one such
  // workgroup per compute unit it is the fastest (1 x 4096 x 4096 5.5 us, slim
  // 6.0; 1 x 1536 x 4096 4.9 and 5.8; 4 x 4096 x 4096 5.9 and 6.0; 8 rows 6.2
  // and 6.0; past that 1 x 8192 x 4096 8.6 and 8.1).
  if (E == 0 && fast && M <= 4 && ceil_div(N, 16) <= cus) return 2;
  // Larger experts: the skinny kernel's fits, over dense products, say nothing
  // of its grouped form.
  if (E > 0 && fast) first = kI8FirstTile;
  if (E > 0 && !fast) end = kI8FirstSkinny;
  int best = first;
  double least = 0.0;
  for (int c = first; c < end; ++c) {
    const Cost& k = cost(c, fast);
    const double across = (double)ceil_div(N, k.cols);
    // Grouped: an expert's last tile is half empty on average.
    const double down = E > 0 ? (double)E * (mean / k.rows + 0.5) : (double)ceil_div(M, k.rows);
    const double t = estimate(k, (E > 0 && down < E ? (double)E : down) * across, steps, cus);
    if (c == first || t < least) {
      least = t;
      best = c;
    }
  }
  return best;
}

int64_t int8_grid(int cfg, int64_t E, int64_t M, int64_t N) {
  const Cost& c = kFast[cfg];
  const int64_t across = ceil_div(N, c.cols);
  if (E == 0) return ceil_div(M, c.rows) * across;
  return (M / c.rows + E) * across;
}

}  // namespace fbg

extern "C" int fbg_int8_plan(int64_t E, int64_t M, int64_t N, int64_t K, int aligned_rows, int cu_count,
                             fbg_plan* out) {
  if (!out || E < 0 || M < 0 || N < 0 || K < 0 || cu_count <= 0) return FBG_ERROR_INVALID_VALUE;
  if (M > fbg::kMaxExtent || N > fbg::kMaxExtent || E > fbg::kMaxExtent || K > fbg::kMaxInt8K)
    return FBG_ERROR_UNSUPPORTED;
  *out = fbg_plan{};
  out->variant = FBG_VARIANT_INT8;
  out->split_k = 1;
  out->config = -1;
  if (M == 0 || N == 0 || K < 16) return FBG_SUCCESS;
  const int cfg = fbg::int8_cfg_for(E, M, N, K, aligned_rows != 0 && K % 16 == 0, cu_count);
  const fbg::Cost& c = fbg::kFast[cfg];
  const int64_t grid = fbg::int8_grid(cfg, E, M, N);
  if (grid > fbg::kMaxI8Grid) return FBG_ERROR_UNSUPPORTED;
  out->tile_m = c.rows;
  out->tile_n = c.cols;
  out->waves = c.waves;
  out->config = cfg;
  out->grid = grid;
  return FBG_SUCCESS;
}
