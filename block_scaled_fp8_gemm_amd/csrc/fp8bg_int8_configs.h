// Kernel configurations of the int8 products and the choice among them (host
// code without HIP, shared by the planner and the launcher).
#pragma once

#include <stdint.h>

namespace fbg {

// X(index, kernel, rows, columns, then the kernel's other sizes)
//   ANY: rows x columns tile, steps in flight (any alignment)
//   SKINNY: rows x columns, waves, K slices per group, whether 16-byte rows
//           have a form of their own (else it takes them like any others)
//   SLIM: rows x columns tile, steps per round, ring slots (16-byte rows)
//   TILE: rows x columns tile, waves of each, ring slots (16-byte rows)
#define FBG_I8_CFGS(X)              \
  X(0, ANY, 64, 64, 2)              \
  X(1, ANY, 32, 64, 4)              \
  X(2, SKINNY, 8, 16, 8, 4, true)   \
  X(3, SKINNY, 16, 16, 8, 4, true)  \
  X(4, SKINNY, 16, 32, 4, 4, false) \
  X(5, TILE, 32, 64, 1, 2, 4)       \
  X(6, TILE, 64, 64, 2, 2, 4)       \
  X(7, TILE, 64, 128, 2, 2, 3)      \
  X(8, TILE, 128, 128, 2, 2, 2)     \
  X(9, TILE, 128, 256, 2, 2, 3)     \
  X(10, TILE, 256, 256, 2, 2, 2)    \
  X(11, SLIM, 32, 32, 2, 4)         \
  X(12, SLIM, 32, 32, 1, 6)

constexpr int kNumI8Cfgs = 13;
constexpr int kI8FirstTile = 5;  // configurations from here on (tiles and slim) take 16-byte rows only
constexpr int kI8FirstSkinny = 2;

// Largest K: int32 sums of products of int8 codes, -128 included, 2^14 * K < 2^31.
constexpr int64_t kMaxInt8K = ((int64_t)1 << 17) - 1;

// Largest row, column and expert counts: the kernels round them up to a tile,
// or step over them, in 32 bits.
constexpr int64_t kMaxExtent = INT32_MAX - 1024;

// Largest count of a product's tiles, which are numbered in 32 bits.
constexpr int64_t kMaxI8Grid = INT32_MAX;

// The configuration for M rows (of E experts in the grouped form, E = 0 for
// the dense one), N columns and K bytes on a device of `cus` compute units;
// `fast`: the rows start on 16-byte boundaries and hold whole 16-byte chunks.
int int8_cfg_for(int64_t E, int64_t M, int64_t N, int64_t K, bool fast, int cus);

// The launch grid of a configuration (workgroups; may exceed INT32_MAX).
int64_t int8_grid(int cfg, int64_t E, int64_t M, int64_t N);

}  // namespace fbg
