// gfx950 kernels between a router's logits and the grouped products: which
// experts a token takes and with which weights, the copy of its row to each of
// them in expert order, and the weighted sum on the way back.  The formulas
// stand in include/fp8bg_tokens.h.
#include "fp8bg_device.hpp"
#include "fp8bg_internal.h"
#include "fp8bg_tokens.h"

namespace fbg {

namespace {

constexpr float kInf = __builtin_huge_valf();

// A launch holds less than 2^32 threads along x: many workgroups take a grid of
// two dimensions.
constexpr int64_t kGridX = 1 << 20;
inline dim3 wide_grid(int64_t blocks) {
  return blocks <= kGridX ? dim3((unsigned)blocks) : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
constexpr int kGridY = 1 << 15;
__device__ __forceinline__ int64_t block_of_grid() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// What the lanes of a wave wrote to LDS before it, all of them read behind it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const T u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Lanes' exchanges by data-parallel primitives, in rows of 16.
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(dpp<CTRL>(__float_as_int(x)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)dpp<CTRL>((int)x);
}
constexpr int kRor = 0x120;  // rotation of a row
constexpr int64_t kNone64 = (int64_t)1 << 63;

// op over the L lanes of a token, in all of them: within a row by rotations, over
// the four rows through scalar registers.
template <int L, typename V, typename Op>
__device__ __forceinline__ V over_lanes(V x, const Op& op) {
  x = op(x, dpp<kRor + 8>(x));
  x = op(x, dpp<kRor + 4>(x));
  x = op(x, dpp<kRor + 2>(x));
  x = op(x, dpp<kRor + 1>(x));
  if constexpr (L == 64) {
    const auto row = [&](int r) {
      const int v = __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * r);
      return __builtin_bit_cast(V, v);
    };
    x = op(op(row(0), row(1)), op(row(2), row(3)));
  }
  return x;
}

// Bits of a float as an integer of the same order, and back.
__device__ __forceinline__ int ordered(float v) {
  const int b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// ---------------------------------------------------------------------------
// Routing.  What is compared is c = score + bias in 64 bits, or the logits
// themselves without a bias (the scores' order, exactly).
// ---------------------------------------------------------------------------

// A token by a whole wave, everything in 64 bits; lane l holds the experts
// l * VPL .. l * VPL + VPL - 1, so that of equal values the lowest expert is in the
// lowest lane and first in it.  shared: 64 * VPL values of LDS for this wave.
template <typename T, int VPL>
__device__ void route_exactly(const RouteArgs& a, int64_t t, double* shared) {
  const int lane = threadIdx.x & 63;
  float* wo = a.weights + t * a.topk;
  int* eo = a.experts + t * a.topk;
  if (a.mask && a.mask[t]) {
    if (lane < a.topk) wo[lane] = 0.0f, eo[lane] = -1;
    return;
  }
  const T* row = reinterpret_cast<const T*>(a.logits) + t * a.ld;
  float z[VPL];
  bool bad = false;
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    z[i] = e < a.E ? (float)row[e] : -kInf;
    bad |= !(z[i] < kInf);
    top = z[i] > top ? z[i] : top;
  }
  top = wave_max(top);
  if (a.score == FBG_SCORE_SOFTMAX) bad |= top == -kInf;
  double s[VPL], c[VPL];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = lane * VPL + i < a.E;
    if (a.score == FBG_SCORE_SOFTMAX) {
      s[i] = in ? exp((double)z[i] - (double)top) : 0.0;
      sum += s[i];
    } else {
      s[i] = 1.0 / (1.0 + exp(-(double)z[i]));
    }
  }
  if (a.score == FBG_SCORE_SOFTMAX) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] /= sum;
  }
  bool allowed[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    allowed[i] = e < a.E;
    c[i] = (double)z[i];
    if (a.bias) {
      const float b = allowed[i] ? a.bias[e] : 0.0f;
      bad |= !(b < kInf);
      c[i] = s[i] + (double)b;
    }
  }
  if (__ballot(bad)) {
    if (lane < a.topk) wo[lane] = __builtin_nanf(""), eo[lane] = lane;
    return;
  }
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    wave_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (allowed[i]) shared[lane * VPL + i] = a.group_score == FBG_GROUP_MAX || a.bias ? c[i] : s[i];
    wave_sync();
    double best = -kInf, second = -kInf;
    if (lane < a.groups) {
#pragma unroll 8
      for (int i = 0; i < size; ++i) {
        const double u = shared[lane * size + i];
        second = u > best ? best : u > second ? u : second;
        best = u > best ? u : best;
      }
      if (a.group_score == FBG_GROUP_TOP2 && size > 1) best += second;
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double u = __shfl(best, g, 64);
      better += u > best || (u == best && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && better < a.topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i) allowed[i] = allowed[i] && ((kept >> ((lane * VPL + i) / size)) & 1);
  }
  // The values as integers of their order; the scores, as weights, to LDS.
  wave_sync();
  float* scores = reinterpret_cast<float*>(shared);
  int64_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    scores[lane * VPL + i] = (float)s[i];
    const int64_t bits = __builtin_bit_cast(int64_t, c[i] + 0.0);  // of two zeros none is larger
    key[i] = allowed[i] ? bits ^ ((bits >> 63) & 0x7fffffffffffffff) : kNone64;
  }
  wave_sync();
  float mine = 0.0f;
  int expert = 0;
  const auto more = [](auto x, auto y) { return x > y ? x : y; };
  for (int j = 0; j < a.topk; ++j) {
    int64_t best = key[0];
    int place = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > best) best = key[i], place = i;
    // The high words' maximum, then the low ones' among those that have it.
    const int high = (int)(best >> 32), top_high = over_lanes<64>(high, more);
    const uint32_t low = (uint32_t)best, top_low = over_lanes<64>(high == top_high ? low : 0u, more);
    const int winner = __builtin_ctzll(__ballot(high == top_high && low == top_low));
    const int e = winner * VPL + __builtin_amdgcn_readlane(place, winner);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i == e) key[i] = kNone64;
    if (lane == j) mine = scores[e], expert = e;
  }
  if (a.renormalize) {
    const float total = wave_sum(mine);
    mine = mine / (total < 1e-20f ? 1e-20f : total);
  }
  if (lane < a.topk) wo[lane] = mine * a.scale, eo[lane] = expert;
}

// For whatever the kernel below does not take.
template <typename T, int VPL>
__global__ __launch_bounds__(256) void k_route_exactly(RouteArgs a) {
  __shared__ double shared[4][64 * VPL];
  const int64_t t = block_of_grid() * 4 + (threadIdx.x >> 6);
  if (t < a.T) route_exactly<T, VPL>(a, t, shared[threadIdx.x >> 6]);
}

constexpr int kNone = (int)0x80000000;  // below every value's key
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// L lanes per token, VPL experts each.  The comparisons are of 32-bit integers: the
// value's bits in order, the lowest ones replaced by the place, inverted, so
// that a maximum names its expert, and of equal ones the lowest.
//
// EXACT (16-bit logits without a bias): the value takes 16 or 19 bits, the
// expert the last 10, and nothing is lost.  Else the values are c in 32 bits with the
// lane's place in the last bits, and the choice holds if each of the first topk is
// above the next by more than both c can be off.  With U = 2^-24: a product for
// exp2's argument, its constant and its result make exp(x) off by (1.5 |x| + 2) U of
// itself, so 1 / (1 + exp(-z)), with one sum and a reciprocal, is off by
// (1.5 |z| + 2) U s (1 - s) + 3 U s < 2^-22, and a softmax, whose sum adds the mean of its
// terms' errors (2.5 ln E + 2) U and its additions' 22 U, by less than 2^-18 of the
// largest score.  fp32 logits without a bias are compared as they are.
//
// Values that are too near (in one row of 400 for random fp32 logits and biases) are
// compared in 64 bits, the first topk + 1 of them alone; where that does not settle a row
// (three in a heap, the line between groups, a softmax with a bias), it is done again by
// the whole wave, which takes 5 us.  A group's two best are taken in 32
// bits, by its lanes where it is 2^p of them, else by one lane from LDS, and the kept
// and the others are checked against each group's own bound (scores without a bias
// are off by 1.5 |z| U < 2^-16.9 of themselves, or by 2^-126).
//
// 16384 tokens of 256 fp32 logits, sigmoid, bias, 4 of 8 groups, 8 experts: 16.1 us (18
// MB, whose copy takes 3.4; every score in 64 bits took 54).  Vector instructions bind it,
// most of them comparisons: 1552 a wave of four cycles each, four waves to a SIMD, are 24.8
// thousand of the 25.5 thousand cycles that a wave lives.  About one row a call is done again by its whole wave
// (the trace's maximum is 21.7 us).  16-bit logits without bias or groups take 7.1 us.  Few
// tokens are bound by latency: 64 of them 6.2 us, one of bf16 logits 3.0.
template <typename T, int L, int VPL, bool EXACT>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
  constexpr int kExact = L == 16 ? VPL < 4 ? 1 : VPL / 4 : VPL;  // experts per lane of a whole wave
  constexpr int kPlace = EXACT ? 1023 : VPL - 1;
  constexpr int kChunks = VPL * (int)sizeof(T) / 16;  // of 16 bytes per lane
  constexpr int kShared = 64 * (2 * kChunks > kExact ? 2 * kChunks : VPL / 2 > kExact ? VPL / 2 : kExact);
  __shared__ double shared[4][kShared];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l = lane & (L - 1);
  const int e0 = l * VPL;
  const int64_t t0 = (block_of_grid() * 4 + w) * (64 / L);
  if (t0 >= a.T) return;  // whole waves, which meet at no barrier
  const int64_t mine = t0 + lane / L, t = mine < a.T ? mine : a.T - 1;
  const T* row = reinterpret_cast<const T*>(a.logits) + t * a.ld;
  const bool masked = a.mask && a.mask[t];
  T raw[VPL];
  if constexpr (kChunks > 1) {
    // The token's lanes read it 16 bytes next to one another, and take their own
    // experts from LDS; chunk q lies where 16 lanes' reads meet 64 banks.
    typedef uint32_t U4a __attribute__((ext_vector_type(4)));
    U4a* rows = reinterpret_cast<U4a*>(shared[w]) + lane / L * (L * kChunks);
    const auto place = [](int q) { return (q & ~(kChunks - 1)) | ((q + (q >> 4)) & (kChunks - 1)); };
    constexpr int CE = 16 / (int)sizeof(T);
    U4a got[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int at = (k * L + l) * CE;
      if (at + CE <= a.E) {
        __builtin_memcpy(&got[k], row + at, 16);
      } else {
        T v[CE];
#pragma unroll
        for (int i = 0; i < CE; ++i) v[i] = row[at + i < a.E ? at + i : 0];
        __builtin_memcpy(&got[k], v, 16);
      }
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) rows[place(k * L + l)] = got[k];
    wave_sync();
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      got[k] = rows[place(l * kChunks + k)];
      __builtin_memcpy(raw + k * CE, &got[k], 16);
    }
  } else if (e0 + VPL <= a.E) {
    __builtin_memcpy(raw, row + e0, sizeof(raw));
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) raw[i] = row[e0 + i < a.E ? e0 + i : 0];
  }
  float b[VPL];
  if (!EXACT && a.bias) {
    if (e0 + VPL <= a.E) {
      __builtin_memcpy(b, a.bias + e0, sizeof(b));
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) b[i] = a.bias[e0 + i < a.E ? e0 + i : 0];
    }
  }
  const auto larger = [](float x, float y) { return x > y ? x : y; };
  const auto plus = [](float x, float y) { return x + y; };
  const auto more = [](int x, int y) { return x > y ? x : y; };
  float c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) c[i] = e0 + i < a.E ? (float)raw[i] + 0.0f : -kInf;  // of two zeros none is larger
  bool bad = false;
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    bad |= !(c[i] < kInf);
    top = larger(c[i], top);
  }
  const bool softmax = a.score == FBG_SCORE_SOFTMAX;
  float total = 1.0f;
  if (softmax) {
    top = over_lanes<L>(top, larger);
    bad |= top == -kInf;
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += fast_exp(c[i] - top);
    total = over_lanes<L>(total, plus);
  }
  const float inverse = 1.0f / total;
  const auto score_of = [&](float z) {
    return softmax ? fast_exp(z - top) * inverse : __builtin_amdgcn_rcpf(1.0f + fast_exp(-z));
  };
  // How far a score may be off, and c by more than its own rounding.
  const float off = EXACT || !a.bias ? 0.0f : softmax ? 0x1p-18f * inverse : 0x1p-22f;
  if (!EXACT && a.bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      bad |= !(b[i] < kInf);
      c[i] = score_of(c[i]) + b[i];
      if (e0 + i >= a.E) c[i] = -kInf;
    }
  }
  bool sure = true;
  uint32_t kept = ~0u;  // which of the lane's experts are of groups that stay
  const int base = lane & ~(L - 1);
  if (a.groups > 1) {
    const bool aligned = a.group_lanes > 0;
    const bool two = a.group_score == FBG_GROUP_TOP2;
    float best = -kInf, second = -kInf;
    const auto take = [&](float u) {
      second = __builtin_amdgcn_fmed3f(best, second, u);
      best = larger(best, u);
    };
    if (aligned) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) take(c[i]);
      // Over the lanes of a group; after each step those of half a group agree.
      const auto join = [&](float u, float v) {
        second = larger(best < u ? best : u, larger(second, v));
        best = larger(best, u);
      };
      if (a.group_lanes > 1) join(dpp<0xb1>(best), dpp<0xb1>(second));
      if (a.group_lanes > 2) join(dpp<0x4e>(best), dpp<0x4e>(second));
      if (a.group_lanes > 4) join(dpp<0x141>(best), dpp<0x141>(second));
      if (a.group_lanes > 8) join(dpp<0x140>(best), dpp<0x140>(second));
      if (L == 64 && a.group_lanes > 16) join(__shfl_xor(best, 16, 64), __shfl_xor(second, 16, 64));
    } else {  // a lane looks at a whole group
      float* values = reinterpret_cast<float*>(shared[w]) + lane / L * (L * VPL);
      wave_sync();
#pragma unroll
      for (int i = 0; i < VPL; ++i) values[e0 + i] = c[i];
      wave_sync();
      const int size = a.E / a.groups;
      if (l < a.groups) {
#pragma unroll 8
        for (int i = 0; i < size; ++i) take(values[l * size + i]);
      }
    }
    // A group's value and how far it may be off: each sum by its score and its own
    // rounding (U of it), whatever is left of the two when they cancel.  With the mean
    // for the sum of two, so that none passes the largest number, that is at most off and
    // U (|best| + |second|) / 2; the mean's rounding and that of a bound added to it are no more
    // than the latter each.  (A -infinity is exact.)
    float value = best, magnitude = __builtin_fabsf(best);
    if (two && (EXACT || !a.bias)) {
      value = score_of(best) + (a.E > a.groups ? score_of(second) : 0.0f);
    } else if (two && a.E > a.groups) {
      value = 0.5f * best + 0.5f * second;
      magnitude = 0.5f * magnitude + 0.5f * __builtin_fabsf(second);
    }
    float value_off = off > 0.0f ? off + 0x1.8p-23f * magnitude : 0x1p-16f * value;
    value_off += 0x1p-120f;
    if (value == -kInf) value_off = 0.0f;
    const int lanes = aligned ? a.group_lanes : 1, last = aligned ? L : a.groups;
    const bool real = aligned ? e0 < a.E : l < a.groups;
    if (!real) value = -kInf;
    int better = 0;  // groups that come before this lane's
    for (int o = aligned ? lanes : 0; o < last; o += lanes) {
      const int other = aligned ? (l + o) & (L - 1) : o;
      const float u = __shfl(value, other + base, 64);
      better += u > value || (u == value && other < l);
    }
    const bool stays = real && better < a.topk_groups;
    if (two || off > 0.0f) {
      // The least that one that stays may be, and the most that another may be: not only
      // the two next to the line, since each group has a bound of its own.
      const auto smaller = [](float x, float y) { return x < y ? x : y; };
      const float low = over_lanes<L>(stays ? value - value_off : kInf, smaller);
      const float high = over_lanes<L>(real && !stays ? value + value_off : -kInf, larger);
      sure = low > high || high == -kInf;
    }
    if (aligned) {
      kept = stays ? ~0u : 0;
    } else {
      const uint64_t stay = __ballot(stays) >> (L == 64 ? 0 : lane & 48);
      kept = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)  // the group of an expert by its inverse, exact below 1024
        kept |= (uint32_t)((stay >> (((uint32_t)(e0 + i) * a.group_inverse >> 20) & 63)) & 1) << i;
    }
  }
  int key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int place = EXACT ? 1023 - (e0 + i) : VPL - 1 - i;
    key[i] = (kept >> i & 1) && e0 + i < a.E ? (ordered(c[i]) & ~kPlace) | place : kNone;
  }
  int rank_key = kNone, expert = 0;
  const int rounds = a.topk + (EXACT ? 0 : 2);
  for (int r = 0; r < rounds; ++r) {
    int m = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = more(m, key[i]);
    const int local = m;
    m = over_lanes<L>(m, more);
    int e, gone = m;
    if constexpr (EXACT) {
      e = 1023 - (m & 1023);
    } else {
      const uint64_t holds = __ballot(local == m);
      int winner;
      if constexpr (L == 64) winner = __builtin_ctzll(holds);
      else winner = __builtin_ctz((uint32_t)(holds >> (lane & 48)) & 0xffff);
      e = winner * VPL + (VPL - 1 - (m & kPlace));
      gone = l == winner ? m : kNone;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = key[i] == gone ? kNone : key[i];
    if (l == r) rank_key = m, expert = e;
  }
  // Lane l has the token's expert number l; lanes topk and topk + 1 the first two
  // of the others.
  expert = expert < a.E ? expert : a.E - 1;
  float z = l < rounds ? (float)row[expert] : 0.0f;
  if constexpr (!EXACT) {
    const int other_key = __shfl(rank_key, base + a.topk + 1, 64);
    // What the others behind lane topk's are at most: the key's value and all that the
    // place took from another's.
    const float rest = other_key == kNone ? -kInf : unordered(other_key | kPlace);
    // And how far above it one of them may be: the sum's rounding grows with the value, so
    // a lower one stays below the same line.  (A -infinity is exact.)
    const float rest_off = off > 0.0f && rest > -kInf ? off + 0x1p-24f * __builtin_fabsf(rest) : 0.0f;
    const bool there = l <= a.topk && rank_key != kNone;
    float v = z, most = 0.0f;
    if (a.bias && there) {
      v = score_of(z) + a.bias[expert];
      most = off + 0x1p-24f * __builtin_fabsf(v);
    }
    const float next = __shfl(v, lane + 1, 64), lim = most + __shfl(most, lane + 1, 64);
    const bool next_there = __shfl((int)there, lane + 1, 64) != 0;
    bool clear = true;
    if (l < a.topk && next_there) clear = v - next > lim;
    if (l == a.topk - 1 && other_key != kNone) clear = clear && v - rest > most + rest_off;
    const bool again = !clear && !(softmax && a.bias);
    sure = sure && (clear || again);
    if (__ballot(again)) {
      // Lanes 0 .. topk are put in order by their values in 64 bits (softmax with a
      // bias: their sum is not known to 64); the others are far enough below the last of
      // them that is chosen, or the row goes the long way.
      double d = (double)z;
      if (a.bias && there) d = 1.0 / (1.0 + exp(-(double)z)) + (double)a.bias[expert];
      int rank = 0;
      for (int o = 0; o <= a.topk; ++o) {
        const double u = __shfl(d, base + o, 64);
        const int ue = __shfl(expert, base + o, 64);
        const bool ut = __shfl((int)there, base + o, 64) != 0;
        rank += ut && (u > d || (u == d && ue < expert));
      }
      int* order = reinterpret_cast<int*>(shared[w]) + base;
      wave_sync();
      if (there) order[rank] = lane;
      wave_sync();
      const int from = there ? order[l] : lane;
      expert = __shfl(expert, from, 64);
      z = __shfl(z, from, 64);
      d = __shfl(d, from, 64);
      if (l == a.topk - 1 && other_key != kNone) sure = sure && d - (double)rest > (double)rest_off;
    }
  }
  float weight = 0.0f;
  if (l < a.topk) {
    weight = softmax ? expf(z - top) * inverse : z < 0.0f ? expf(z) / (1.0f + expf(z)) : 1.0f / (1.0f + expf(-z));
  }
  if (a.renormalize) {
    const float sum = over_lanes<L>(weight, plus);
    weight = weight / (sum < 1e-20f ? 1e-20f : sum);
  }
  weight *= a.scale;
  const uint64_t token = L == 64 ? ~0ull : 0xffffull << (lane & 48);
  if (__ballot(bad) & token) weight = __builtin_nanf(""), expert = l, sure = true;
  if (masked) weight = 0.0f, expert = -1, sure = true;
  const uint64_t unsure = __ballot(!sure && mine < a.T);
  if (mine < a.T && l < a.topk && !(unsure & token)) {
    a.weights[t * a.topk + l] = weight;
    a.experts[t * a.topk + l] = expert;
  }
  for (int i = 0; i < 64 / L; ++i)
    if (unsure & ((L == 64 ? ~0ull : 0xffffull) << (i * L & 63))) route_exactly<T, kExact>(a, t0 + i, shared[w]);
}

template <typename T, int L, int VPL>
hipError_t route(const RouteArgs& a) {
  const dim3 g = wide_grid(((int64_t)a.T * L + 255) / 256), b(256);
  if constexpr (sizeof(T) == 2) {
    if (!a.bias) {
      hipLaunchKernelGGL((k_route<T, L, VPL, true>), g, b, 0, a.stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_route<T, L, VPL, false>), g, b, 0, a.stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t route(RouteArgs a) {
  // Whether L lanes of vpl experts hold them all, a rank for every choice and two
  // more, and a lane for every group.
  const auto fits = [&](int L, int vpl) {
    if (a.E > L * vpl || a.topk + 2 > L || a.groups > L) return false;
    const int size = a.E / a.groups, lanes = size / vpl;
    const bool aligned = size % vpl == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 32;
    a.group_lanes = aligned ? lanes : 0;
    a.group_inverse = (1u << 20) / size + 1;
    return true;
  };
  // Many tokens: four to a wave.  Few: a wave each, for its shorter way to an answer.
  // 256 experts with bias and groups, us with 16 lanes and with 64: 2048 tokens 8.8 and
  // 6.8, 4096 8.9 and 8.4, 6000 8.9 and 10.0, 16384 16.4 and 21.2; 64 experts: 2048 6.1
  // and 5.7, 4096 6.2 and 6.4, 16384 8.9 and 15.2.  More than 256 experts take a wave a
  // token always: 16384 of 384 50 us, of 1024 47 (bf16 without bias and groups 26 and 24).
  if (a.T > 2048 && fits(16, 4)) return route<T, 16, 4>(a);
  if (a.T > 4096 && fits(16, 16)) return route<T, 16, 16>(a);
  if (fits(64, 1)) return route<T, 64, 1>(a);
  if (fits(64, 4)) return route<T, 64, 4>(a);
  if (fits(64, 16)) return route<T, 64, 16>(a);
  const dim3 g = wide_grid(((int64_t)a.T + 3) / 4), b(256);
  if (a.E <= 64) hipLaunchKernelGGL((k_route_exactly<T, 1>), g, b, 0, a.stream, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route_exactly<T, 4>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_route_exactly<T, 16>), g, b, 0, a.stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Into expert order: a stable counting sort of the T * topk choices by expert.
// ---------------------------------------------------------------------------

// Where a choice's expert is held here, its number, else kNoExpert.  (first and
// first + E are within 0 .. 2^31 - 1, so a negative id wraps to a number past E.)
constexpr int kNoExpert = 0x7fffffff;
__device__ __forceinline__ int local_expert(int id, int first, int E) {
  const uint32_t e = (uint32_t)id - (uint32_t)first;
  return e < (uint32_t)E ? (int)e : kNoExpert;
}

typedef unsigned int U4 __attribute__((ext_vector_type(4), aligned(1)));

// The bytes of one token, row and scales, to `slots` (in LDS, -1 for none) by
// TPT threads.  The first 16 bytes of each thread are loaded before the slots
// are known (`head`).
template <int TPT>
struct Mover {
  const uint8_t* x;
  int64_t bytes;
  int t;
  U4 head;
  __device__ __forceinline__ Mover(const DispatchArgs& a, int64_t token, int t_)
      : x(a.x + token * a.x_pitch), bytes(a.row_bytes), t(t_) {
    if ((int64_t)t * 16 < bytes && bytes >= 16) head = *reinterpret_cast<const U4*>(x + start(t * 16));
  }
  // The last 16 bytes of a row overlap those before them.
  __device__ __forceinline__ int64_t start(int64_t at) const { return at + 16 <= bytes ? at : bytes - 16; }
  __device__ __forceinline__ void put(const DispatchArgs& a, int64_t token, const int* slots) const {
    for (int64_t at = (int64_t)t * 16; at < bytes; at += TPT * 16) {
      if (bytes >= 16) {
        const int64_t s = start(at);
        const U4 v = at < TPT * 16 ? head : *reinterpret_cast<const U4*>(x + s);
        for (int j = 0; j < a.topk; ++j)
          if (slots[j] >= 0) *reinterpret_cast<U4*>(a.rows + slots[j] * a.rows_pitch + s) = v;
      } else {
        for (int64_t i = at; i < bytes; ++i) {
          const uint8_t v = x[i];
          for (int j = 0; j < a.topk; ++j)
            if (slots[j] >= 0) a.rows[slots[j] * a.rows_pitch + i] = v;
        }
      }
    }
    if (a.x_scale) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(a.x_scale + token * a.scale_bytes);
      for (int64_t i = t; i < a.scale_bytes / 4; i += TPT) {
        const uint32_t v = from[i];
        for (int j = 0; j < a.topk; ++j)
          if (slots[j] >= 0) reinterpret_cast<uint32_t*>(a.row_scale + slots[j] * a.scale_bytes)[i] = v;
      }
    }
  }
};

// Exclusive sums of values[0 .. 1024) over a workgroup of THREADS threads,
// 1024 / THREADS next to one another each; sums: THREADS / 64 words of LDS.
template <int THREADS>
__device__ __forceinline__ void exclusive_sums(int (&v)[1024 / THREADS], int* sums) {
  constexpr int N = 1024 / THREADS;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int total = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = v[i];
    v[i] = total;
    total += c;
  }
  int run = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(run, o, 64);
    if (lane >= o) run += u;
  }
  if (lane == 63) sums[w] = run;
  __syncthreads();
  int before = run - total;
  for (int i = 0; i < w; ++i) before += sums[i];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += before;
}

// Few choices: one launch.  A workgroup per token finds the rows of its choices
// by counting, over all choices, those of lower experts and the earlier ones of
// the same: the lanes' comparisons are masks in scalar registers, whose bits
// the scalar unit counts.  The first workgroup makes the offsets.  64 tokens of 8
// choices and 4096 bytes: 5.3 us, bound by latency.
__global__ __launch_bounds__(256) void k_dispatch_few(DispatchArgs a) {
  __shared__ int shared[1024];
  __shared__ int sums[4];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x == 0) {
    for (int i = tid; i < 1024; i += 256) shared[i] = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += 256) {
      const int e = local_expert(a.experts[i], a.first, a.E);
      if (e != kNoExpert) atomicAdd(&shared[e], 1);
    }
    __syncthreads();
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = shared[tid * 4 + i];
    exclusive_sums<256>(v, sums);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tid * 4 + i <= a.E) a.offsets[tid * 4 + i] = v[i];
    if (tid == 255 && a.E == 1024) a.offsets[1024] = v[3] + shared[1023];
    return;
  }
  const int t = blockIdx.x - 1, i0 = t * a.topk;
  const Mover<256> mover(a, t, tid);
  int* counts = shared;  // [wave][choice]
  for (int j0 = 0; j0 < a.topk; j0 += 8) {
    const int targets = a.topk - j0 < 8 ? a.topk - j0 : 8;
    int target[8], count[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      target[j] = j < targets ? local_expert(a.experts[i0 + j0 + j], a.first, a.E) : kNoExpert;
    for (int c = w * 64; c < a.n; c += 256) {
      const int e = c + lane < a.n ? local_expert(a.experts[c + lane], a.first, a.E) : kNoExpert;
      const int earlier = i0 + j0 - c;  // how many of these 64 come before the first choice
      if (earlier >= 64 || earlier <= -8) {
        const int bound = earlier >= 64;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < targets) count[j] += __popcll(__ballot(e < target[j] + bound && e != kNoExpert));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t before = earlier + j >= 64 ? ~0ull : earlier + j <= 0 ? 0 : (1ull << (earlier + j)) - 1;
          count[j] += __popcll(__ballot(e < target[j])) + __popcll(__ballot(e == target[j]) & before);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane == j && j < targets) counts[w * 64 + j0 + j] = target[j] == kNoExpert ? -1 : count[j];
  }
  __syncthreads();
  if (tid < a.topk) {
    int s = counts[tid];
    if (s >= 0) s += counts[64 + tid] + counts[128 + tid] + counts[192 + tid];
    counts[256 + tid] = s;
    a.slots[i0 + tid] = s;
  }
  __syncthreads();
  mover.put(a, t, counts + 256);
}

// Many choices, two launches: the choices' rows, and then the rows themselves.
// Each workgroup counts all choices by expert, those before its own apart (LDS
// atomics on integers: their order changes nothing), which gives its starts without a
// word from the others, and ranks its own, 1024 at a time: a wave finds the lanes
// of each expert bit by bit, and the waves' counts are summed in their order.  32768
// choices: 8.3 us.  (The counting is by all workgroups of all choices, so past some hundred
// thousand of them it grows with their number.)
__global__ __launch_bounds__(1024) void k_slots(DispatchArgs a) {
  extern __shared__ int wave_counts[];  // [16][E]
  __shared__ int counts[2048], sums[16];  // choices before its own by expert, and the others
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t own = blockIdx.x * a.own, end = own + a.own < a.n ? own + a.own : a.n;
  counts[tid] = counts[1024 + tid] = 0;
  __syncthreads();
  // A wave takes 256 choices at a time, which lie on one side of its own.
  typedef int I4 __attribute__((ext_vector_type(4), aligned(4)));
  constexpr int kStep = 4096, kAhead = 2;
  for (int64_t c = (int64_t)w * 256; c < a.n; c += kStep * kAhead) {
    I4 id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t i = c + u * kStep + lane * 4;
      if (i + 4 <= a.n) {
        id[u] = *reinterpret_cast<const I4*>(a.experts + i);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) id[u][k] = i + k < a.n ? a.experts[i + k] : -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      int* side = counts + (c + u * kStep < own ? 0 : 1024);
      const int lead = __builtin_amdgcn_readfirstlane(id[u][0]);
      if (__ballot(id[u][0] != lead || id[u][1] != lead || id[u][2] != lead || id[u][3] != lead) == 0) {
        const int e = local_expert(lead, a.first, a.E);  // a popular expert's run: one addition
        if (lane == 0 && e != kNoExpert) atomicAdd(&side[e], 256);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = local_expert(id[u][k], a.first, a.E);
          if (e != kNoExpert) atomicAdd(&side[e], 1);
        }
      }
    }
  }
  __syncthreads();
  int all[1] = {counts[tid] + counts[1024 + tid]};
  const int count = all[0];
  exclusive_sums<1024>(all, sums);
  if (blockIdx.x == 0) {
    if (tid <= a.E) a.offsets[tid] = all[0];
    if (tid == a.E - 1) a.offsets[a.E] = all[0] + count;
  }
  int start = all[0] + counts[tid];  // of expert tid's next choice here
  int* mine = wave_counts + w * a.E;
  for (int64_t base = own; base < end; base += 1024) {
    const int64_t at = base + tid;
    const int e = at < end ? local_expert(a.experts[at], a.first, a.E) : kNoExpert;
    for (int k = lane; k < a.E; k += 64) mine[k] = 0;
    uint64_t same = __ballot(e != kNoExpert);
    for (int bit = 1; bit < a.E; bit <<= 1) {
      const uint64_t set = __ballot((e & bit) != 0);
      same &= (e & bit) ? set : ~set;
    }
    const int ahead = __popcll(same & ((1ull << lane) - 1));
    wave_sync();
    if (e != kNoExpert && ahead == 0) mine[e] = __popcll(same);
    __syncthreads();
    if (tid < a.E) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int c = wave_counts[k * a.E + tid];
        wave_counts[k * a.E + tid] = start;
        start += c;
      }
    }
    __syncthreads();
    if (at < end) a.slots[at] = e != kNoExpert ? mine[e] + ahead : -1;
    wave_sync();  // a wave's counts are its own again
  }
}

// TPT threads per token.  4096 tokens of 8 x 4096 bytes: 30.4 us, 151 MB at 5.0 TB/s
// (a large copy: 5.2).
template <int TPT>
__global__ __launch_bounds__(256) void k_move(DispatchArgs a) {
  __shared__ int shared[256 / TPT][64];
  const int t = threadIdx.x % TPT, which = threadIdx.x / TPT;
  const int64_t token = block_of_grid() * (256 / TPT) + which;
  const bool here = token < a.T;
  const Mover<TPT> mover(a, here ? token : 0, t);
  if (here && t < a.topk) shared[which][t] = a.slots[token * a.topk + t];
  __syncthreads();
  if (here) mover.put(a, token, shared[which]);
}

// ---------------------------------------------------------------------------
// Back into token order: a thread sums 16 bytes' worth of a token's columns, the
// loads of up to kRows rows in flight together.  A token's slots and weights are in
// scalar registers.  4096 tokens of 8 x 4096 bf16 with a base: 64.2 us, 336 MB at 5.2
// TB/s (one row after the other 82); 64 tokens 3.6, latency.
// ---------------------------------------------------------------------------
template <typename T, int VE>
__device__ __forceinline__ void load_floats(const void* p, int64_t at, int n, float (&v)[VE]) {
  const T* q = reinterpret_cast<const T*>(p) + at;
  if (n >= VE) {
    T c[VE];
    __builtin_memcpy(c, q, sizeof(c));
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = (float)c[i];
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = i < n ? (float)q[i] : 0.0f;
  }
}

template <typename T, typename O>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a) {
  constexpr int VE = 16 / (int)sizeof(T), kRows = 8;
  typedef T Raw __attribute__((ext_vector_type(VE)));
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.z * kGridY + blockIdx.y;
  int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VE;
  if (t >= a.T || at - lane * VE >= a.D) return;  // whole waves: any lane's slot is read below
  const int slot_of = lane < a.topk ? a.slots[t * a.topk + lane] : -1;
  const float weight_of = lane < a.topk ? a.weights[t * a.topk + lane] : 0.0f;
  // A last chunk that D cuts is taken from the row's end; its first columns are
  // another thread's, and not stored.  A lane past it takes it too and stores none.
  const bool whole = a.D >= VE;
  const int n = whole ? VE : at == 0 ? a.D : 0;
  int cut = 0;
  if (whole && at + VE > a.D) cut = at < a.D ? (int)(at + VE - a.D) : VE, at = a.D - VE;
  if (!whole) at = 0;
  float acc[VE] = {};
  if (a.base) {
    if (a.base_is_out) load_floats<O>(a.base, t * a.ldbase + at, n, acc);
    else load_floats<T>(a.base, t * a.ldbase + at, n, acc);
  }
  const T* rows = reinterpret_cast<const T*>(a.rows) + at;
  for (int j0 = 0; j0 < a.topk; j0 += kRows) {
    Raw raw[kRows];
    int slot[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      slot[j] = j0 + j < a.topk ? __builtin_amdgcn_readlane(slot_of, j0 + j) : -1;
      if (slot[j] < 0 || slot[j] >= a.R) continue;
      const T* p = rows + slot[j] * a.ldrows;
      if (whole) {
        __builtin_memcpy(&raw[j], p, 16);
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) raw[j][i] = p[i < n ? i : 0];
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (slot[j] < 0 || slot[j] >= a.R) continue;
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight_of), j0 + j));
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[i] = __builtin_fmaf(w, (float)raw[j][i], acc[i]);
    }
  }
  if (cut == VE || n == 0) return;  // a lane past the last column
  O* out = reinterpret_cast<O*>(a.out) + t * a.ldout + at;
  O o[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) o[i] = (O)acc[i];
  if (whole && cut == 0) {
    __builtin_memcpy(out, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i >= cut && i < n) out[i] = o[i];
  }
}

template <typename T, typename O>
hipError_t combine(const CombineArgs& a) {
  constexpr int kCols = 256 * 16 / (int)sizeof(T);
  const unsigned y = a.T < kGridY ? a.T : kGridY;
  const dim3 g((unsigned)(((int64_t)a.D + kCols - 1) / kCols), y, (a.T + y - 1) / y);
  hipLaunchKernelGGL((k_combine<T, O>), g, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t combine(const CombineArgs& a) {
  switch (a.out_dtype) {
    case kOutBF16: return combine<T, __bf16>(a);
    case kOutFP16: return combine<T, _Float16>(a);
    default: return combine<T, float>(a);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a) {
  switch (a.dtype) {
    case kOutBF16: return route<__bf16>(a);
    case kOutFP16: return route<_Float16>(a);
    default: return route<float>(a);
  }
}

// Up to this many pairs of a token and a choice the kernel that compares them all is the
// faster one.  us with it and without, rows of 4096 bytes: 64 tokens of 8 choices 5.1 and
// 7.3, 256 of 8 8.1 and 8.6, 320 of 8 9.4 and 9.1, 512 of 8 12.8 and 10.3; 512 of 4 7.4
// and 8.3, 1024 of 1 5.9 and 7.2, 2048 of 1 12.2 and 8.7.
constexpr int64_t few_comparisons(int topk) { return (int64_t)1 << (topk <= 4 ? 20 : 19); }

hipError_t launch_dispatch(DispatchArgs a) {
  if ((int64_t)a.T * a.n <= few_comparisons(a.topk)) {
    hipLaunchKernelGGL(k_dispatch_few, dim3(a.n > 0 ? a.T + 1 : 1), dim3(256), 0, a.stream, a);
    return hipGetLastError();
  }
  a.own = ((int64_t)a.n + 256 * 1024 - 1) / (256 * 1024) * 1024;  // at most a workgroup per compute unit
  hipLaunchKernelGGL(k_slots, dim3((unsigned)((a.n + a.own - 1) / a.own)), dim3(1024), 16 * a.E * sizeof(int), a.stream,
                     a);
  // A wave per token for short rows, else four.  16384 tokens of 6 experts, us of the two
  // kernels with one and with four: 256 bytes 23.9 and 28.9, 1024 39.4 and 45.3, 2048 62.8
  // and 63.2, 4096 113 and 103; 1001 tokens: 1024 bytes 8.7 and 8.8, 2048 10.4 and 9.9.
  if (a.row_bytes <= 1024)
    hipLaunchKernelGGL(k_move<64>, wide_grid(((int64_t)a.T + 3) / 4), dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL(k_move<256>, wide_grid(a.T), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a) {
  switch (a.dtype) {
    case kOutBF16: return combine<__bf16>(a);
    case kOutFP16: return combine<_Float16>(a);
    default: return combine<float>(a);
  }
}

}  // namespace fbg
