// gfx950 kernels for low-rank adapters of many requests at once:
//
//   out[m] = y[m] + scales[a] * B[a] (A[a] x[m]),   a = adapters[m]
//
// in two launches: h = A[a] x (a token's R values, kept in fp32) and the product
// with B[a] added to y.  A tile holds 16 tokens whatever their adapters; it
// goes over the different ones among them, so that tokens share an adapter's
// reads wherever they stand, and a run of one adapter is one pass.
#include "fp8bg_device.hpp"
#include "fp8bg_internal.h"

namespace fbg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kMaxSplits = 4;

// Grids: splits of K or blocks of columns along x, tiles of 16 tokens along y
// and, past kGridY of them, z; with several workers per tile they stand along z.
// (No flat index: its 64-bit divisions took longer than a decode tile's loads.)
constexpr int kGridY = 1 << 15;
inline dim3 tile_grid(int64_t x, int64_t tiles, int workers) {
  const int64_t y = tiles < kGridY ? tiles : kGridY;
  return dim3((unsigned)x, (unsigned)y, workers > 1 ? (unsigned)workers : (unsigned)((tiles + y - 1) / y));
}
__device__ __forceinline__ int64_t first_token(int workers) {
  return ((workers > 1 ? 0 : (int64_t)blockIdx.z * kGridY) + blockIdx.y) * 16;
}
__device__ __forceinline__ int worker_of(int workers) { return workers > 1 ? blockIdx.z : 0; }

template <typename T> struct Vec8;
template <> struct Vec8<__bf16> { typedef v8bf type; };
template <> struct Vec8<_Float16> { typedef v8h type; };

__device__ __forceinline__ v4f mfma32(const v8bf& a, const v8bf& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma32(const v8h& a, const v8h& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// N elements from row[at ..] at any alignment, zeros from row[n] on.
template <int N, typename T>
__device__ __forceinline__ void load_some(const T* row, int at, int n, T (&v)[N]) {
  if (at + N <= n) {
    __builtin_memcpy(v, row + at, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = at + i < n ? row[at + i] : (T)0.0f;
  }
}
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type load8(const T* row, int at, int n) {
  T v[8] = {};
  if (at < n) load_some(row, at, n, v);
  typename Vec8<T>::type r;
  __builtin_memcpy(&r, v, sizeof(r));
  return r;
}

// The adapter of token m, -1 for none or past the last token.
__device__ __forceinline__ int adapter_of(const AdapterArgs& a, int64_t m) {
  const int id = m < a.M && a.L > 0 ? a.adapters[m] : -1;
  return id >= 0 && id < a.L ? id : -1;
}

// The passes of a tile of 16 tokens: one for each different adapter among them.
// Of `workers` (a power of two) number `worker` does every workers-th.
template <typename F>
__device__ __forceinline__ void for_passes(int id, int worker, int workers, const F& pass) {
  uint64_t todo = __ballot(id >= 0) & 0xffff;
  for (int p = 0; todo; ++p) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == cur);
    if ((p & (workers - 1)) == worker) pass(cur);
  }
}

// h of 16 tokens over one slice of K for one adapter of theirs, or each in
// turn; the waves split the slice, and their sums meet in LDS.  RT tiles
// of 16 ranks at a time; the loads of U steps are in flight together.
template <typename T, int RT>
__global__ __launch_bounds__(256) void k_shrink(AdapterArgs a) {
  constexpr int W = 4;
  constexpr int U = RT == 1 ? 8 : 4;
  typedef typename Vec8<T>::type V;
  __shared__ v4f part[RT][W][64];  // [tile of 16 ranks][wave][lane]
  const int split = blockIdx.x, worker = worker_of(a.workers);
  const int64_t m0 = first_token(a.workers);
  if (m0 >= a.M) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), j = lane & 15, g = lane >> 4;
  const int id = adapter_of(a, m0 + j);
  const int first = (split * W + w) * a.share;
  const int last = first + a.share < a.K ? first + a.share : a.K;
  float* h = a.h + ((int64_t)split * a.M + m0 + j) * a.pitch;
  for_passes(id, worker, a.workers, [&](int cur) {
    const bool mine = id == cur;
    const uint64_t meant = __ballot(mine);  // asked of all lanes: not inside the choice below
    // Lanes of other tokens read the row of one that is meant.
    const int64_t m = m0 + (mine ? j : __builtin_ctzll(meant));
    const T* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
    const T* A = reinterpret_cast<const T*>(a.A) + (int64_t)cur * a.R * a.K;
    for (int r0 = 0; r0 < a.R; r0 += 16 * RT) {
      const T* row[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) row[i] = A + (int64_t)(r0 + 16 * i + j < a.R ? r0 + 16 * i + j : a.R - 1) * a.K;
      v4f acc[RT] = {};
      int k = first;
      for (; k + 32 * U <= last; k += 32 * U) {
        V xf[U], af[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          __builtin_memcpy(&xf[u], x + k + 32 * u + 8 * g, 16);
#pragma unroll
          for (int i = 0; i < RT; ++i) __builtin_memcpy(&af[u][i], row[i] + k + 32 * u + 8 * g, 16);
        }
        __builtin_amdgcn_sched_barrier(0);  // all loads before the first use of one
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i] = mfma32(af[u][i], xf[u], acc[i]);
      }
      for (; k + 64 <= last; k += 64) {
        V xf[2], af[2][RT];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          __builtin_memcpy(&xf[u], x + k + 32 * u + 8 * g, 16);
#pragma unroll
          for (int i = 0; i < RT; ++i) __builtin_memcpy(&af[u][i], row[i] + k + 32 * u + 8 * g, 16);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i] = mfma32(af[u][i], xf[u], acc[i]);
      }
      for (; k < last; k += 32) {
        const V xf = load8(x, k + 8 * g, a.K);
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = mfma32(load8(row[i], k + 8 * g, a.K), xf, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) part[i][w][lane] = acc[i];
      __syncthreads();
      if (w < RT && r0 + 16 * w < a.R) {  // wave w: ranks r0 + 16 w ..
        const int r = r0 + 16 * w + 4 * g;
        v4f s = part[w][0][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) s += part[w][i][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i >= a.R) s[i] = 0.0f;
        if (mine) *reinterpret_cast<v4f*>(h + r) = s;
      }
      __syncthreads();
    }
  });
}

// h in the weights' type, as a sum that the MFMA takes term by term: each term
// is what the ones before it leave, rounded.  bf16 has fp32's range: two terms are
// off by 2^-18 of a value, which a 16-bit output does not see, three by 2^-26.  fp16
// goes relative to the largest of a token's ranks (`unit`, a power of two), the second
// term times 2^11 to stay above its smallest steps, with sums of its own: off
// by 2^-22.
template <typename T, typename O> struct Terms;
template <typename O> struct Terms<__bf16, O> {
  static constexpr int kCount = sizeof(O) == 4 ? 3 : 2, kSums = 1;
};
template <typename O> struct Terms<_Float16, O> {
  static constexpr int kCount = 2, kSums = 2;
};

// How the eight ranks of a lane are read: in one piece where R is a multiple of
// eight; else as two of four, the row's last four shifted to where they belong; fewer
// than four one by one.
enum Ranks { kWhole, kPart, kTiny };

// 16 tokens by blocks of 64 columns, four blocks next to one another on the
// four waves.  Row i of the first operand's tile t is column 32 (t / 2) + 8 (i / 4) +
// 4 (t % 2) + i % 4 of the block, so that a lane's results are of one token and 8
// columns next to one another, twice.  Each token belongs to one pass, which
// alone writes its row; the first worker writes the rows without an adapter.  NC
// chunks of 32 ranks at a time; DEEP: more than those, h read again for each block
// of columns.
//
// The loads of the next block are in flight while one is computed: they stay
// raw dwords until they are used, and have no branch between lanes (a lane of
// another token reads the row of one that is meant), since the compiler waits
// for a load where it unpacks its value or where the lanes meet again.  A last
// block that N cuts goes element by element.
template <typename T, typename O, int NC, bool DEEP, Ranks RANKS>
__global__ __launch_bounds__(256) void k_expand(AdapterArgs a) {
  constexpr int YC = 2 * (int)sizeof(O) / 4;  // 16-byte chunks of 8 outputs
  constexpr int kTerms = Terms<T, O>::kCount, kSums = Terms<T, O>::kSums;
  typedef typename Vec8<T>::type V;
  typedef uint32_t U4 __attribute__((ext_vector_type(4)));
  typedef uint64_t L2 __attribute__((ext_vector_type(2)));
  typedef O O8 __attribute__((ext_vector_type(8)));
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int worker = worker_of(a.workers);
  const int64_t m0 = first_token(a.workers), n_block = (int64_t)blockIdx.x * a.cols;
  const int64_t n_first = n_block + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64, n_end = n_block + a.cols;
  if (m0 >= a.M || n_first >= a.N) return;  // whole waves, which meet at no barrier
  const int64_t n_last = n_end < a.N ? n_end : a.N;
  const int id = adapter_of(a, m0 + j);
  const int column = 8 * (j >> 2) + (j & 3);
  struct Weights {
    L2 v[NC][4];
  };
  struct Outputs {
    U4 v[2][YC];
  };
  const auto load_y = [&](const O* row, int64_t n0) {
    Outputs y;
#pragma unroll
    for (int q = 0; q < 2; ++q) __builtin_memcpy(y.v[q], row + n0 + 32 * q + 8 * g, sizeof(y.v[q]));
    return y;
  };
  for_passes(id, worker, a.workers, [&](int cur) {
    const bool mine = id == cur;
    const uint64_t meant = __ballot(mine);
    const int64_t m = m0 + (mine ? j : __builtin_ctzll(meant));
    const O* yrow = reinterpret_cast<const O*>(a.y) + m * a.ldy;
    O* orow = reinterpret_cast<O*>(a.out) + m * a.ldout;
    const T* B = reinterpret_cast<const T*>(a.B) + (int64_t)cur * a.N * a.R;
    const float* hrow = a.h + m * a.pitch;
    const int64_t h_split = (int64_t)a.M * a.pitch;
    const auto load_b = [&](int64_t n0, int r0) {
      Weights b;
      const T* base = B + n0 * a.R;
      const int most = a.N - n0 < 64 ? (int)(a.N - n0) - 1 : 63;  // a column past the last one: the last one's
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int n = 32 * (t >> 1) + 4 * (t & 1) + column;
        const T* row = base + (n < most ? n : most) * a.R;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int r = r0 + 32 * c + 8 * g;
          if constexpr (RANKS == kTiny) {
            T v[8] = {};
#pragma unroll
            for (int k = 0; k < 3; ++k) v[k] = row[k < a.R ? k : 0];
            __builtin_memcpy(&b.v[c][t], v, 16);
          } else if constexpr (RANKS == kWhole) {
            __builtin_memcpy(&b.v[c][t], row + (r < a.R ? r : 0), 16);
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint64_t v;
              __builtin_memcpy(&v, row + (r + 4 * k < a.R - 4 ? r + 4 * k : a.R - 4), 8);
              b.v[c][t][k] = v;
            }
          }
        }
      }
      return b;
    };
    // A lane's weights, zeros from rank R on.
    const auto weights = [&](const L2& raw, int r) {
      L2 v = raw;
      if constexpr (RANKS == kWhole) {
        if (r >= a.R) v = L2{0, 0};
      } else if constexpr (RANKS == kTiny) {
        v = r == 0 ? L2{v[0] & ((1ull << (16 * a.R)) - 1), 0} : L2{0, 0};
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int past = r + 4 * k > a.R - 4 ? r + 4 * k - (a.R - 4) : 0;
          v[k] = past < 4 ? v[k] >> (16 * past) : 0;
        }
      }
      return __builtin_bit_cast(V, v);
    };
    const float scale = a.scales ? a.scales[cur] : 1.0f;
    V h[NC][kTerms];
    float unit = 1.0f;
    const auto load_h = [&](int r0) {
      float v[NC][8];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int r = r0 + 32 * c + 8 * g;
        v4f part[kMaxSplits][2];
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
          if (s < a.splits) __builtin_memcpy(part[s], hrow + s * h_split + (r < a.pitch ? r : 0), 32);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int s = 1; s < kMaxSplits; ++s)
            if (s < a.splits) part[0][k] += part[s][k];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][4 * k + i] = r < a.pitch ? part[0][k][i] * scale : 0.0f;
        }
      }
      if constexpr (kSums == 2) {
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, __builtin_fabsf(v[c][i]));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // The power of two at or below it, kept where it and its inverse are normal.
        const uint32_t e = __float_as_uint(top) & 0x7f800000u;
        unit = __uint_as_float(e < 0x01000000u ? 0x01000000u : e > 0x7e000000u ? 0x7e000000u : e);
        const float inverse = 1.0f / unit;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] *= inverse;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float rest = v[c][i];
#pragma unroll
          for (int t = 0; t < kTerms; ++t) {
            const T term = (T)rest;
            h[c][t][i] = term;
            rest = (rest - (float)term) * (kSums == 2 ? 2048.0f : 1.0f);
          }
        }
    };
    const auto multiply = [&](const Weights& b, int r0, v4f (&acc)[4]) {
      v4f sum[kSums][4] = {};
      if constexpr (kSums == 1) {
#pragma unroll
        for (int t = 0; t < 4; ++t) sum[0][t] = acc[t];
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        V w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = weights(b.v[c][t], r0 + 32 * c + 8 * g);
#pragma unroll
        for (int i = kTerms - 1; i >= 0; --i)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            v4f& to = sum[kSums == 2 ? i : 0][t];
            to = mfma32(w[t], h[c][i], to);
          }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (kSums == 1) acc[t] = sum[0][t];
        else acc[t] += (sum[0][t] + sum[1][t] * 0x1p-11f) * unit;
      }
    };
    // The products of one block, the weights of its first ranks in hand.
    const auto block = [&](int64_t n0, const Weights& b, v4f (&acc)[4]) {
      if constexpr (DEEP) {
        Weights now = b;
        for (int r0 = 0; r0 < a.R; r0 += 32 * NC) {
          const Weights then = load_b(n0, r0 + 32 * NC < a.R ? r0 + 32 * NC : r0);
          load_h(r0);
          multiply(now, r0, acc);
          now = then;
        }
      } else {
        multiply(b, 0, acc);
      }
    };
    Weights b = load_b(n_first, 0);
    Outputs y;
    int64_t n0 = n_first;
    if (n0 + 64 <= n_last) y = load_y(yrow, n0);
    if constexpr (!DEEP) load_h(0);
    // A lane's results are of its own token: those of the others' adapters,
    // which may hold infinities, go nowhere.
    for (; n0 + 64 <= n_last; n0 += 256) {
      Weights b_next;
      Outputs y_next;
      if (n0 + 320 <= n_last) {
        b_next = load_b(n0 + 256, 0);
        y_next = load_y(yrow, n0 + 256);
      }
      __builtin_amdgcn_sched_barrier(0);  // on their way before the products
      v4f acc[4] = {};
      block(n0, b, acc);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        O8 v = __builtin_bit_cast(O8, y.v[q]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (O)((float)v[i] + acc[2 * q + (i >> 2)][i & 3]);
        if (mine) __builtin_memcpy(orow + n0 + 32 * q + 8 * g, &v, sizeof(v));
      }
      b = b_next;
      y = y_next;
    }
    if (n0 < n_last) {
      O v[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t n = n0 + 32 * q + 8 * g + i;
          v[q][i] = yrow[n < a.N ? n : a.N - 1];
        }
      if (n0 > n_first) b = load_b(n0, 0);
      v4f acc[4] = {};
      block(n0, b, acc);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t n = n0 + 32 * q + 8 * g + i;
          if (mine && n < a.N) orow[n] = (O)((float)v[q][i] + acc[2 * q + (i >> 2)][i & 3]);
        }
    }
  });
  const int64_t m = m0 + j;
  if (worker == 0 && !a.in_place && m < a.M && id < 0) {
    const O* yrow = reinterpret_cast<const O*>(a.y) + m * a.ldy;
    O* orow = reinterpret_cast<O*>(a.out) + m * a.ldout;
    for (int64_t n0 = n_first; n0 < n_last; n0 += 256) {
      if (n0 + 64 <= n_last) {
        const Outputs y = load_y(yrow, n0);
#pragma unroll
        for (int q = 0; q < 2; ++q) __builtin_memcpy(orow + n0 + 32 * q + 8 * g, y.v[q], sizeof(y.v[q]));
      } else {
        for (int64_t n = n0 + 8 * g; n < n0 + 64; n += 32)
          for (int i = 0; i < 8; ++i)
            if (n + i < a.N) orow[n + i] = yrow[n + i];
      }
    }
  }
}

template <typename T, typename O, Ranks RANKS>
void expand(const AdapterArgs& a, dim3 g) {
  const dim3 b(256);
  if (a.R <= 32) hipLaunchKernelGGL((k_expand<T, O, 1, false, RANKS>), g, b, 0, a.stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL((k_expand<T, O, 2, false, RANKS>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_expand<T, O, 2, true, RANKS>), g, b, 0, a.stream, a);
}

template <typename T, typename O>
void expand(const AdapterArgs& a, dim3 g) {
  if (a.R < 4) hipLaunchKernelGGL((k_expand<T, O, 1, false, kTiny>), g, dim3(256), 0, a.stream, a);
  else if (a.R % 8 == 0) expand<T, O, kWhole>(a, g);
  else expand<T, O, kPart>(a, g);
}

template <typename T>
hipError_t add(AdapterArgs a) {
  const int64_t tiles = ((int64_t)a.M + 15) / 16;
  // Few tokens: a worker for each adapter that a tile may hold.  Many: the
  // tiles cover the device, and their tokens come in runs.
  a.workers = tiles <= 64 ? 16 : tiles <= 512 ? 4 : 1;
  while (a.workers / 2 >= a.M) a.workers /= 2;
  if (a.R > 0 && a.L > 0 && a.K > 0) {
    const dim3 g = tile_grid(a.splits, tiles, a.workers);
    const dim3 b(256);
    a.share = ((a.K + 31) / 32 + a.splits * 4 - 1) / (a.splits * 4) * 32;  // a wave's: whole steps of 32
    if (a.R <= 16) hipLaunchKernelGGL((k_shrink<T, 1>), g, b, 0, a.stream, a);
    else if (a.R <= 32) hipLaunchKernelGGL((k_shrink<T, 2>), g, b, 0, a.stream, a);
    else hipLaunchKernelGGL((k_shrink<T, 4>), g, b, 0, a.stream, a);
  } else {
    a.L = 0;  // no adapter at all
  }
  // Blocks of columns one after the other where there are many tokens.
  const int64_t blocks = ((int64_t)a.N + 255) / 256;
  int64_t per = tiles * a.workers * blocks / 2048;
  per = per < 1 ? 1 : per > 4 ? 4 : per;
  a.cols = (int)per * 256;
  const dim3 g = tile_grid((blocks + per - 1) / per, tiles, a.workers);
  switch (a.out_dtype) {
    case kOutBF16: expand<T, __bf16>(a, g); break;
    case kOutFP16: expand<T, _Float16>(a, g); break;
    default: expand<T, float>(a, g); break;
  }
  return hipGetLastError();
}

}  // namespace

// How many workgroups split K: enough that few tokens still cover the device.
int adapter_splits(int64_t M, int64_t K) {
  const int64_t tiles = (M + 15) / 16;
  int64_t most = (K + 255) / 256;
  most = most < kMaxSplits ? most : kMaxSplits;
  const int64_t s = 2048 / (tiles > 0 ? tiles : 1);
  return (int)(s < 1 ? 1 : s < most ? s : most);
}

hipError_t launch_add_adapters(const AdapterArgs& a) {
  return a.dtype == kOutBF16 ? add<__bf16>(a) : add<_Float16>(a);
}

}  // namespace fbg
