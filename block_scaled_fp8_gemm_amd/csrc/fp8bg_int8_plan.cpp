// The int8 products' choice of a kernel configuration (pure host code).
#include <math.h>

#include "fp8bg.h"
#include "fp8bg_int8_configs.h"

namespace fbg {

namespace {

enum Kind { ANY, SKINNY, TILE };

// What a configuration costs, in microseconds: `start` once per workgroup and
// `step` per 128 bytes of K, rising from `step` for one workgroup alone to
// `full` with `per_cu` on every compute unit; past that the rounds queue up,
// and `again` is the share of `start` that a queued round still shows.
// Least-squares fits in the logarithm to 167 dense shapes of M 1 .. 16384, N
// 64 .. 8192 and K 256, 1024 and 4096 (configurations 2-10, 16-byte rows; the
// fits' own deviation is 4-13%) and to 79 of the same range with odd K (any
// rows).  Choosing by it costs 2.0% over the best configuration of each shape
// on average (any rows: 2.9%).
struct Cost {
  Kind kind;
  int rows, cols, per_cu, waves;
  float start, step, full, again;
};
constexpr Cost kFast[kNumI8Cfgs] = {
    {ANY, 64, 64, 4, 4, 0, 0, 0, 0},
    {ANY, 32, 64, 4, 4, 0, 0, 0, 0},
    {SKINNY, 8, 16, 3, 8, 2.615f, 0.075f, 0.264f, 0.654f},
    {SKINNY, 16, 16, 3, 8, 2.655f, 0.081f, 0.328f, 0.744f},
    {SKINNY, 16, 32, 3, 8, 2.385f, 0.151f, 0.549f, 0.800f},
    {TILE, 32, 64, 3, 2, 2.700f, 0.218f, 0.455f, 0.751f},
    {TILE, 64, 64, 2, 4, 2.828f, 0.238f, 0.447f, 0.667f},
    {TILE, 64, 128, 2, 4, 3.343f, 0.280f, 0.697f, 0.841f},
    {TILE, 128, 128, 2, 4, 3.959f, 0.511f, 1.221f, 0.968f},
    {TILE, 128, 256, 1, 4, 7.084f, 0.546f, 0.968f, 0.925f},
    {TILE, 256, 256, 1, 4, 11.821f, 0.976f, 1.581f, 0.975f},
};
constexpr Cost kAny[kI8FirstTile] = {
    {ANY, 64, 64, 4, 4, 4.169f, 0.367f, 1.924f, 1.769f},
    {ANY, 32, 64, 4, 4, 3.796f, 0.240f, 1.487f, 1.532f},
    {SKINNY, 8, 16, 3, 8, 3.263f, 0.176f, 0.901f, 0.629f},
    {SKINNY, 16, 16, 3, 8, 3.174f, 0.206f, 1.046f, 0.826f},
    {SKINNY, 16, 32, 3, 8, 3.135f, 0.329f, 1.429f, 0.736f},
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
    // 16-byte rows: the 32 x 64 tile (256 experts of 512 x 4096, 64 tokens of 8
    // experts each: 97 us, skinny 93-100, 64 x 128 tile 103; of 1536 x 1024:
    // 64 us against 91-127 and 64), except over a long K with at most two
    // skinny workgroups per compute unit, where those are faster (8 experts
    // of 512 x 4096: 5.6 us at 64 rows, 10.4 in the tile).  Any rows: the
    // 32-column skinny form up to about one workgroup per compute unit (64
    // rows over 64 experts of 512 x 1000: 6.4 us, the 32 x 64 tile 6.4; 8
    // experts: 4.0 against 5.1), else the 32 x 64 tile (256 experts: 27.7 us
    // against 32.9).
    if (fast) return K >= 2048 && E * ceil_div(N, 16) <= 2 * cus ? 3 : 5;
    return E * ceil_div(N, 32) <= 4 * cus ? 4 : 1;
  }
  // A skinny workgroup walks an expert's rows one pass after the other.
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
  return (c.kind == SKINNY ? E : M / c.rows + E) * across;
}

}  // namespace fbg

extern "C" int fbg_int8_plan(int64_t E, int64_t M, int64_t N, int64_t K, int aligned_rows, int cu_count,
                             fbg_plan* out) {
  if (!out || E < 0 || M < 0 || N < 0 || K < 0 || cu_count <= 0) return FBG_ERROR_INVALID_VALUE;
  if (M > INT32_MAX || N > INT32_MAX || E > INT32_MAX - 1 || K > 131071) return FBG_ERROR_UNSUPPORTED;
  *out = fbg_plan{};
  out->variant = FBG_VARIANT_INT8;
  out->split_k = 1;
  out->config = -1;
  if (M == 0 || N == 0 || K < 16) return FBG_SUCCESS;
  const int cfg = fbg::int8_cfg_for(E, M, N, K, aligned_rows != 0 && K % 16 == 0, cu_count);
  const fbg::Cost& c = fbg::kFast[cfg];
  out->tile_m = c.rows;
  out->tile_n = c.cols;
  out->waves = c.waves;
  out->config = cfg;
  out->grid = fbg::int8_grid(cfg, E, M, N);
  return FBG_SUCCESS;
}
