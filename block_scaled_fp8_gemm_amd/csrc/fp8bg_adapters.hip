// gfx950 kernels for low-rank adapters of many requests at once:
//
//   out[m] = y[m] + scales[a] * B[a] (A[a] x[m]),   a = adapters[m]
//
// in two launches: h = A[a] x (a token's R values, kept in fp32) and the product
// with B[a] added to y.  A tile holds 16 tokens whatever their adapters; it
// goes over the different ones among them, so that tokens share an adapter's
// reads wherever they stand, and a run of one adapter is one pass.
//
// 16384 tokens of 16 adapters of rank 16, 4096 to 4096 columns, bf16: 39 us for the
// first product (136 MB read by the counters, 3.5 TB/s) and 64 for the second (146 read
// and 134 written, 4.4 TB/s); a large copy reaches 5.2.  Neither computes for long (vector
// and matrix instructions take 3% and 2% of the first's time, 32% and 6% of the second's).
// 64 tokens of a request each: 4.6 and 5.1 us, bound by latency.  One kernel for both, a
// workgroup per 16 tokens with h in LDS, took 11.4 us there against 8.9 in a graph, and
// was no faster for many (104 both).
#include <type_traits>

#include "fp8bg_device.hpp"
#include "fp8bg_internal.h"

namespace fbg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kMaxSplits = 4;
// Whether `tiles` tiles of 16 tokens go four to a workgroup: it reads an adapter once for
// all of its tokens, and fewer workgroups share the work.  K = N = 4096, 16 tokens
// per workgroup and 64, us, a batch of 8 prompts / of a request per token over 16
// adapters: rank 64, 256 tokens 14.9 and 20.6 / 37.8 and 27.5, 512 20.3 and 24.6 / 57.5 and
// 36.6, 2048 39.5 and 30.9 / 198 and 112; rank 128, 256 tokens 17.1 and 24.0 / 54.7 and
// 36.5, 512 29.2 and 29.3 / 99 and 56; rank 256, 64 tokens 17.3 and 26.4 / 31.0 and 28.0,
// 256 26.9 and 30.4 / 98.5 and 58.8.  Up to rank 32 the first product alone: 8 prompts of
// rank 16, 2048 tokens 17.7 and 18.7, 4096 30.4 and 27.1.
bool many_tokens(int64_t tiles, int64_t R) { return R > 32 ? tiles * R >= 2048 : tiles > 200; }

// Grids: splits of K or blocks of columns along x, tiles of 16 tokens along y
// and, past kGridY of them, z; with several workers per tile they stand along z.
// (No flat index: its 64-bit divisions took longer than a decode tile's loads.)
constexpr int kGridY = 1 << 15;
inline dim3 tile_grid(int64_t x, int64_t tiles, int workers) {
  const int64_t y = tiles < kGridY ? tiles : kGridY;
  return dim3((unsigned)x, (unsigned)y, workers > 1 ? (unsigned)workers : (unsigned)((tiles + y - 1) / y));
}
__device__ __forceinline__ int64_t tile_of(int workers) {
  return (workers > 1 ? 0 : (int64_t)blockIdx.z * kGridY) + blockIdx.y;
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

// The passes of a tile of 16 MT tokens (lane l holds the adapter of token l of
// them, or l modulo their number): one for each different adapter, with the mask
// of its tokens.  Of `workers` (a power of two) number `worker` does every
// workers-th.
template <int MT, typename F>
__device__ __forceinline__ void for_passes(int id, int worker, int workers, const F& pass) {
  uint64_t todo = __ballot(id >= 0) & (MT == 4 ? ~0ull : (1ull << (16 * MT & 63)) - 1);
  for (int p = 0; todo; ++p) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t meant = todo & __ballot(id == cur);
    todo &= ~meant;
    if ((p & (workers - 1)) == worker) pass(cur, meant);
  }
}

// h of 16 MT tokens over one slice of K for one adapter of theirs, or each in
// turn; the waves split the slice, and their sums meet in LDS.  RT tiles of 16
// ranks to a workgroup; the loads of U steps are in flight together.  Many tokens
// take MT = 4, which reads the adapter's rows from L2 once for 64 tokens (16384
// tokens of rank 64: 16 tokens' workgroups read 537 MB of them).
template <typename T, int RT, int MT>
__global__ __launch_bounds__(256) void k_shrink(AdapterArgs a) {
  constexpr int W = 4, TM = 16 * MT;
  constexpr int U = MT > 1 ? 2 : RT > 1 ? 4 : 8;
  typedef typename Vec8<T>::type V;
  __shared__ v4f part[RT * MT][W][64];  // [tile of 16 ranks by 16 tokens][wave][lane]
  // Ranks past 64 are other workgroups'.
  const int chunk = (int)gridDim.x == a.splits ? 0 : blockIdx.x / a.splits, r0 = chunk * 16 * RT;
  const int split = blockIdx.x - chunk * a.splits, worker = worker_of(a.workers);
  const int64_t m0 = tile_of(a.workers) * TM;
  if (m0 >= a.M) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), j = lane & 15, g = lane >> 4;
  const int id = adapter_of(a, m0 + (lane & (TM - 1)));
  const int first = (split * W + w) * a.share;
  const int last = first + a.share < a.K ? first + a.share : a.K;
  for_passes<MT>(id, worker, a.workers, [&](int cur, uint64_t meant) {
    const T* x[MT];
    bool some[MT];  // a tile of tokens without this adapter is left out
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t bits = (uint32_t)(meant >> (16 * t)) & 0xffff;
      some[t] = MT == 1 || bits;
      // Lanes of other tokens read the row of one that is meant.
      const int at = (bits >> j) & 1 ? j : __builtin_ctz(bits | 0x10000) & 15;
      const int64_t m = m0 + 16 * t + at < a.M ? m0 + 16 * t + at : a.M - 1;
      x[t] = reinterpret_cast<const T*>(a.x) + m * a.ldx;
    }
    const T* A = reinterpret_cast<const T*>(a.A) + (int64_t)cur * a.R * a.K;
    const T* row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = A + (int64_t)(r0 + 16 * i + j < a.R ? r0 + 16 * i + j : a.R - 1) * a.K;
    v4f acc[MT][RT] = {};
    const auto steps = [&](int k, auto count) {
      constexpr int N = decltype(count)::value;
      V xf[MT][N], af[N][RT];
#pragma unroll
      for (int u = 0; u < N; ++u) {
#pragma unroll
        for (int i = 0; i < RT; ++i) __builtin_memcpy(&af[u][i], row[i] + k + 32 * u + 8 * g, 16);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (some[t]) {
#pragma unroll
          for (int u = 0; u < N; ++u) __builtin_memcpy(&xf[t][u], x[t] + k + 32 * u + 8 * g, 16);
        }
      __builtin_amdgcn_sched_barrier(0);  // all loads before the first use of one
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (some[t]) {
#pragma unroll
          for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[t][i] = mfma32(af[u][i], xf[t][u], acc[t][i]);
        }
    };
    int k = first;
    for (; k + 32 * U <= last; k += 32 * U) steps(k, std::integral_constant<int, U>{});
    for (; k + 64 <= last; k += 64) steps(k, std::integral_constant<int, 2>{});
    for (; k < last; k += 32) {
      V af[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) af[i] = load8(row[i], k + 8 * g, a.K);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (some[t]) {
          const V xf = load8(x[t], k + 8 * g, a.K);
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[t][i] = mfma32(af[i], xf, acc[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < RT; ++i) part[t * RT + i][w][lane] = acc[t][i];
    __syncthreads();
    for (int q = w; q < MT * RT; q += W) {  // a wave: some of the tiles
      const int t = q / RT, i = q % RT, r = r0 + 16 * i + 4 * g;
      if (r0 + 16 * i >= a.R) continue;
      v4f s = part[q][0][lane];
#pragma unroll
      for (int k = 1; k < W; ++k) s += part[q][k][lane];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + k >= a.R) s[k] = 0.0f;
      const int m = 16 * t + j;
      if ((meant >> m) & 1) *reinterpret_cast<v4f*>(a.h + ((int64_t)split * a.M + m0 + m) * a.pitch + r) = s;
    }
    __syncthreads();
  });
}

// h in the weights' type, as a sum that the MFMA takes term by term: each term
// is what the ones before it leave, rounded.  bf16 has fp32's range: a value in [1, 2)
// leaves at most 2^-8, that at most 2^-17 and that, of fp32's 24 bits, nothing.  So
// three terms are h, and two are off by 2^-17 of it: for 16-bit outputs, whose rounding is
// 2^-8 or 2^-11 of theirs, which only a y that cancels the product goes below (the third term
// would cost them 1 to 3% of a call up to rank 64, 6% at rank 256).  fp16 goes relative to the
// largest of a token's 32 ranks (a power of two, returned), the second term times 2^11
// to stay above its smallest steps, with sums of its own: off by 2^-22 of the largest.
template <typename T, typename O>
constexpr int kTermsOf = std::is_same<T, __bf16>::value && sizeof(O) == 4 ? 3 : 2;

template <typename T, int TERMS>
__device__ __forceinline__ float split_terms(const float (&v)[8], typename Vec8<T>::type (&h)[TERMS]) {
  constexpr bool kHalf = std::is_same<T, _Float16>::value;
  float unit = 1.0f, inverse = 1.0f;
  if constexpr (kHalf) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, __builtin_fabsf(v[i]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    // The power of two at or below it, kept where it and its inverse are normal.
    const uint32_t e = __float_as_uint(top) & 0x7f800000u;
    unit = __uint_as_float(e < 0x01000000u ? 0x01000000u : e > 0x7e000000u ? 0x7e000000u : e);
    inverse = 1.0f / unit;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = v[i] * inverse;
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      const T term = (T)rest;
      h[t][i] = term;
      rest = (rest - (float)term) * (kHalf ? 2048.0f : 1.0f);
    }
  }
  return unit;
}

// acc[t] += weights w[t] (rows) times h (columns: tokens).
template <int TERMS, typename V>
__device__ __forceinline__ void add_products(const V (&w)[4], const V (&h)[TERMS], float unit, v4f (&acc)[4]) {
  if constexpr (std::is_same<V, v8h>::value) {
    v4f first[4] = {}, second[4] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t) first[t] = mfma32(w[t], h[0], first[t]);
#pragma unroll
    for (int t = 0; t < 4; ++t) second[t] = mfma32(w[t], h[1], second[t]);
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] += (first[t] + second[t] * 0x1p-11f) * unit;
  } else {
#pragma unroll
    for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = mfma32(w[t], h[i], acc[t]);
  }
}

// h's ranks r .. r + 7 of one token, summed over the parts of K.
__device__ __forceinline__ void load_hidden(const AdapterArgs& a, const float* row, int r, float (&v)[8]) {
  v4f part[kMaxSplits][2];
  const int64_t next = (int64_t)a.M * a.pitch;
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s)
    if (s < a.splits) __builtin_memcpy(part[s], row + s * next + (r < a.pitch ? r : 0), 32);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int s = 1; s < kMaxSplits; ++s)
      if (s < a.splits) part[0][k] += part[s][k];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * k + i] = r < a.pitch ? part[0][k][i] : 0.0f;
  }
}

// Whether one of a token's 32 ranks, eight in each of its four lanes, is a NaN.
__device__ __forceinline__ bool holds_nan(const float (&v)[8], int j) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) nan |= v[i] != v[i];
  const uint64_t b = __ballot(nan), c = b | b >> 32;
  return (c | c >> 16) >> j & 1;
}

__device__ __forceinline__ bool holds_nan(const v4f (&acc)[4]) {
  const v4f s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  const float t = (s[0] + s[1]) + (s[2] + s[3]);
  return t != t;
}

// Results that are no number though the token's h, `row`, holds none that is not: the
// terms are not h where that is infinite or next to the largest number, and cancel
// times an infinite weight.  They are summed as the formula has them, rank by rank in
// fp32, one after the other (eight at once took 30 registers of every call's, and 512
// tokens of rank 64 51 us instead of 37).
template <typename T>
__device__ __forceinline__ void sum_again(const AdapterArgs& a, const T* B, const float* row, int64_t n0, int g,
                                          v4f (&acc)[4]) {
  asm volatile("" : "+v"(g), "+v"(row));  // nothing of this is computed ahead of the branch (5 registers)
  const int64_t next = (int64_t)a.M * a.pitch;
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const int64_t n = n0 + 32 * (k >> 3) + 8 * g + (k & 7);
    const T* w = B + (n < a.N ? n : a.N - 1) * a.R;
    float s = 0.0f;
#pragma unroll 1
    for (int r = 0; r < a.R; ++r) {
      float h = row[r];
#pragma unroll 1
      for (int p = 1; p < a.splits; ++p) h += row[p * next + r];
      s = __builtin_fmaf((float)w[r], h, s);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = acc[i >> 2][i & 3];
      acc[i >> 2][i & 3] = i == k && v != v ? s : v;
    }
  }
}

// How the eight ranks of a lane are read: in one piece where R is a multiple of
// eight; else as two of four, the row's last four shifted to where they belong; fewer
// than four one by one.
enum Ranks { kWhole, kPart, kTiny };

typedef uint64_t L2 __attribute__((ext_vector_type(2)));

// Ranks r .. r + 7 of the weights of a block's 64 columns from n0 on: row i of
// tile t is column 32 (t / 2) + 8 (i / 4) + 4 (t % 2) + i % 4, so that a lane's results
// are of one token and 8 columns next to one another, twice.  A column past the
// last one reads the last one's.
template <typename T, Ranks RANKS>
__device__ __forceinline__ void load_weights(const T* B, int64_t n0, int N, int r, int R, int j, L2 (&v)[4]) {
  const T* base = B + n0 * R;
  const int most = N - n0 < 64 ? (int)(N - n0) - 1 : 63;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int n = 32 * (t >> 1) + 4 * (t & 1) + 8 * (j >> 2) + (j & 3);
    const T* row = base + (n < most ? n : most) * R;
    if constexpr (RANKS == kTiny) {
      T u[8] = {};
#pragma unroll
      for (int k = 0; k < 3; ++k) u[k] = row[k < R ? k : 0];
      __builtin_memcpy(&v[t], u, 16);
    } else if constexpr (RANKS == kWhole) {
      __builtin_memcpy(&v[t], row + (r < R ? r : 0), 16);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint64_t u;
        __builtin_memcpy(&u, row + (r + 4 * k < R - 4 ? r + 4 * k : R - 4), 8);
        v[t][k] = u;
      }
    }
  }
}

// The same as the MFMA takes them, zeros from rank R on.
template <typename T, Ranks RANKS>
__device__ __forceinline__ typename Vec8<T>::type weights_of(L2 v, int r, int R) {
  if constexpr (RANKS == kWhole) {
    if (r >= R) v = L2{0, 0};
  } else if constexpr (RANKS == kTiny) {
    v = r == 0 ? L2{v[0] & ((1ull << (16 * R)) - 1), 0} : L2{0, 0};
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int past = r + 4 * k > R - 4 ? r + 4 * k - (R - 4) : 0;
      v[k] = past < 4 ? v[k] >> (16 * past) : 0;
    }
  }
  return __builtin_bit_cast(typename Vec8<T>::type, v);
}

// 16 tokens by blocks of 64 columns, four blocks next to one another on the
// four waves.  Each token belongs to one pass, which alone writes its row; the
// first worker writes the rows without an adapter.  NC chunks of 32 ranks.
//
// The loads of the next block are in flight while one is computed: they stay
// raw dwords until they are used, and have no branch between lanes (a lane of
// another token reads the row of one that is meant), since the compiler waits
// for a load where it unpacks its value or where the lanes meet again.  A last
// block that N cuts goes element by element.
template <typename T, typename O, int NC, Ranks RANKS>
__global__ __launch_bounds__(256) void k_expand(AdapterArgs a) {
  constexpr int YC = 2 * (int)sizeof(O) / 4;  // 16-byte chunks of 8 outputs
  constexpr int kTerms = kTermsOf<T, O>;
  typedef typename Vec8<T>::type V;
  typedef uint32_t U4 __attribute__((ext_vector_type(4)));
  typedef O O8 __attribute__((ext_vector_type(8)));
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int worker = worker_of(a.workers);
  const int64_t m0 = tile_of(a.workers) * 16, n_block = (int64_t)blockIdx.x * a.cols;
  const int64_t n_first = n_block + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64, n_end = n_block + a.cols;
  if (m0 >= a.M || n_first >= a.N) return;  // whole waves, which meet at no barrier
  const int64_t n_last = n_end < a.N ? n_end : a.N;
  const int id = adapter_of(a, m0 + j);
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
  for_passes<1>(id, worker, a.workers, [&](int cur, uint64_t meant) {
    const bool mine = id == cur;
    const int64_t m = m0 + (mine ? j : __builtin_ctzll(meant));
    const O* yrow = reinterpret_cast<const O*>(a.y) + m * a.ldy;
    O* orow = reinterpret_cast<O*>(a.out) + m * a.ldout;
    const T* B = reinterpret_cast<const T*>(a.B) + (int64_t)cur * a.N * a.R;
    const float* hrow = a.h + m * a.pitch;
    const auto load_b = [&](int64_t n0) {
      Weights b;
#pragma unroll
      for (int c = 0; c < NC; ++c) load_weights<T, RANKS>(B, n0, a.N, 32 * c + 8 * g, a.R, j, b.v[c]);
      return b;
    };
    const float scale = a.scales ? a.scales[cur] : 1.0f;
    V h[NC][kTerms];
    float unit[NC];
    bool number = true;
    const auto products = [&](const Weights& b, int64_t n0, v4f (&acc)[4]) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        V w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = weights_of<T, RANKS>(b.v[c][t], 32 * c + 8 * g, a.R);
        add_products<kTerms>(w, h[c], unit[c], acc);
      }
      if (mine && number && holds_nan(acc)) sum_again(a, B, hrow, n0, g, acc);
    };
    Weights b = load_b(n_first);
    Outputs y;
    int64_t n0 = n_first;
    if (n0 + 64 <= n_last) y = load_y(yrow, n0);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
      load_hidden(a, hrow, 32 * c + 8 * g, v);
      number = number && !holds_nan(v, j);
      unit[c] = split_terms<T, kTerms>(v, h[c]);
    }
    // A lane's results are of its own token: those of the others' adapters,
    // which may hold infinities, go nowhere.
    for (; n0 + 64 <= n_last; n0 += 256) {
      Weights b_next;
      Outputs y_next;
      if (n0 + 320 <= n_last) {
        b_next = load_b(n0 + 256);
        y_next = load_y(yrow, n0 + 256);
      }
      __builtin_amdgcn_sched_barrier(0);  // on their way before the products
      v4f acc[4] = {};
      products(b, n0, acc);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        O8 v = __builtin_bit_cast(O8, y.v[q]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (O)__builtin_fmaf(acc[2 * q + (i >> 2)][i & 3], scale, (float)v[i]);
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
      if (n0 > n_first) b = load_b(n0);
      v4f acc[4] = {};
      products(b, n0, acc);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t n = n0 + 32 * q + 8 * g + i;
          if (mine && n < a.N) orow[n] = (O)__builtin_fmaf(acc[2 * q + (i >> 2)][i & 3], scale, (float)v[q][i]);
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

// Two waves to a SIMD where that costs few registers: in bf16 four tiles and ranks in parts
// take 260 (16384 tokens of rank 60 136 us, 156 with one wave), fp16's terms 294.
template <typename T>
constexpr int kDeepWaves = std::is_same<T, __bf16>::value ? 2 : 1;

// The same for any rank, in chunks of 32: h's terms are made once per pass, by all
// waves, and stay in LDS.  Many tokens take 16 MT of them to a workgroup, so that a
// block's weights come from L2 once for all (rank 64 and 16384 tokens by 4096 columns:
// 16 tokens' workgroups read 537 MB of them, four times the outputs).
template <typename T, typename O, int MT, Ranks RANKS>
__global__ __launch_bounds__(256, kDeepWaves<T>) void k_expand_deep(AdapterArgs a) {
  constexpr int YC = 2 * (int)sizeof(O) / 4, TM = 16 * MT, kTerms = kTermsOf<T, O>;
  typedef typename Vec8<T>::type V;
  typedef uint32_t U4 __attribute__((ext_vector_type(4)));
  typedef O O8 __attribute__((ext_vector_type(8)));
  // [tile of tokens][chunk][term][lane], then the units [tile][chunk][16], NaN where h is.
  extern __shared__ v4f staged[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), j = lane & 15, g = lane >> 4;
  const int worker = worker_of(a.workers), chunks = (a.R + 31) / 32;
  float* units = reinterpret_cast<float*>(staged + MT * chunks * kTerms * 64);
  const int64_t m0 = tile_of(a.workers) * TM, n_block = (int64_t)blockIdx.x * a.cols;
  if (m0 >= a.M) return;  // a whole workgroup
  const int64_t n_first = n_block + w * 64, n_end = n_block + a.cols;
  const int64_t n_last = n_end < a.N ? n_end : a.N;
  const int id = adapter_of(a, m0 + (lane & (TM - 1)));
  struct Outputs {
    U4 v[2][YC];
  };
  const auto load_y = [&](const O* row, int64_t n0) {
    Outputs y;
#pragma unroll
    for (int q = 0; q < 2; ++q) __builtin_memcpy(y.v[q], row + n0 + 32 * q + 8 * g, sizeof(y.v[q]));
    return y;
  };
  for_passes<MT>(id, worker, a.workers, [&](int cur, uint64_t meant) {
    bool some[MT], mine[MT];
    int row_of[MT];  // in the workgroup's
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t bits = (uint32_t)(meant >> (16 * t)) & 0xffff;
      some[t] = bits != 0;
      mine[t] = (bits >> j) & 1;
      // Lanes of other tokens read the row of one that is meant.
      const int m = 16 * t + (mine[t] ? j : __builtin_ctz(bits | 0x10000) & 15);
      row_of[t] = m0 + m < a.M ? m : (int)(a.M - 1 - m0);
    }
    const O* y_first = reinterpret_cast<const O*>(a.y) + m0 * a.ldy;
    O* out_first = reinterpret_cast<O*>(a.out) + m0 * a.ldout;
    const T* B = reinterpret_cast<const T*>(a.B) + (int64_t)cur * a.N * a.R;
    const float scale = a.scales ? a.scales[cur] : 1.0f;
    for (int q = w; q < MT * chunks; q += 4) {  // a wave: some of the chunks
      const int t = q / chunks, c = q % chunks;
      if (!((meant >> (16 * t)) & 0xffff)) continue;
      const uint32_t bits = (uint32_t)(meant >> (16 * t)) & 0xffff;
      const int64_t m = m0 + 16 * t + ((bits >> j) & 1 ? j : __builtin_ctz(bits));
      float v[8];
      V h[kTerms];
      load_hidden(a, a.h + m * a.pitch, 32 * c + 8 * g, v);
      const bool nan = holds_nan(v, j);
      const float unit = split_terms<T, kTerms>(v, h);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) __builtin_memcpy(&staged[(q * kTerms + i) * 64 + lane], &h[i], 16);
      if (g == 0) units[q * 16 + j] = nan ? __builtin_nanf("") : unit;
    }
    __syncthreads();
    const auto products = [&](const L2 (&raw)[4], int c, v4f (&acc)[MT][4]) {
      V wt[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) wt[t] = weights_of<T, RANKS>(raw[t], 32 * c + 8 * g, a.R);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (some[t]) {
          const int q = t * chunks + c;
          V h[kTerms];
#pragma unroll
          for (int i = 0; i < kTerms; ++i) __builtin_memcpy(&h[i], &staged[(q * kTerms + i) * 64 + lane], 16);
          add_products<kTerms>(wt, h, units[q * 16 + j], acc[t]);
        }
    };
    L2 b[4];
    Outputs y[MT];
    int64_t n0 = n_first;
    if (n0 < n_last) load_weights<T, RANKS>(B, n0, a.N, 8 * g, a.R, j, b);
    if (n0 + 64 <= n_last) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (some[t]) y[t] = load_y(y_first + row_of[t] * a.ldy, n0);
    }
    for (; n0 < n_last; n0 += 256) {
      const bool whole = n0 + 64 <= n_last, more = n0 + 256 < n_last, next_whole = n0 + 320 <= n_last;
      v4f acc[MT][4] = {};
      Outputs y_next[MT];
      for (int c = 0; c < chunks; ++c) {
        L2 b_next[4];
        if (c + 1 < chunks) {
          load_weights<T, RANKS>(B, n0, a.N, 32 * (c + 1) + 8 * g, a.R, j, b_next);
        } else if (more) {
          load_weights<T, RANKS>(B, n0 + 256, a.N, 8 * g, a.R, j, b_next);
        }
        if (c == 0 && next_whole) {
#pragma unroll
          for (int t = 0; t < MT; ++t)
            if (some[t]) y_next[t] = load_y(y_first + row_of[t] * a.ldy, n0 + 256);
        }
        __builtin_amdgcn_sched_barrier(0);  // on their way before the products
        products(b, c, acc);
#pragma unroll
        for (int t = 0; t < 4; ++t) b[t] = b_next[t];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (!some[t]) continue;
        if (mine[t] && holds_nan(acc[t])) {
          bool number = true;
          for (int c = 0; c < chunks; ++c) {
            const float unit = units[(t * chunks + c) * 16 + j];
            number = number && unit == unit;
          }
          if (number) sum_again(a, B, a.h + (m0 + row_of[t]) * a.pitch, n0, g, acc[t]);
        }
        O* orow = out_first + row_of[t] * a.ldout;
        if (whole) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            O8 v = __builtin_bit_cast(O8, y[t].v[q]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (O)__builtin_fmaf(acc[t][2 * q + (i >> 2)][i & 3], scale, (float)v[i]);
            if (mine[t]) __builtin_memcpy(orow + n0 + 32 * q + 8 * g, &v, sizeof(v));
          }
        } else {
          const O* yrow = y_first + row_of[t] * a.ldy;
          O v[2][8];
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t n = n0 + 32 * q + 8 * g + i;
              v[q][i] = yrow[n < a.N ? n : a.N - 1];
            }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t n = n0 + 32 * q + 8 * g + i;
              const float sum = acc[t][2 * q + (i >> 2)][i & 3];
              if (mine[t] && n < a.N) orow[n] = (O)__builtin_fmaf(sum, scale, (float)v[q][i]);
            }
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) y[t] = y_next[t];
    }
    __syncthreads();  // h is read
  });
  if (worker != 0 || a.in_place) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = m0 + 16 * t + j;
    const int of = __shfl(id, 16 * t + j, 64);
    if (m >= a.M || of >= 0) continue;
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
  if (a.R <= 32) hipLaunchKernelGGL((k_expand<T, O, 1, RANKS>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_expand<T, O, 2, RANKS>), g, b, 0, a.stream, a);
}

template <typename T, typename O>
void expand(const AdapterArgs& a, dim3 g) {
  if (a.R < 4) hipLaunchKernelGGL((k_expand<T, O, 1, kTiny>), g, dim3(256), 0, a.stream, a);
  else if (a.R % 8 == 0) expand<T, O, kWhole>(a, g);
  else expand<T, O, kPart>(a, g);
}

template <typename T, typename O, int MT>
void expand_deep(const AdapterArgs& a, int64_t tiles, int64_t ranges) {
  const dim3 b(256), g = tile_grid(ranges, (tiles + MT - 1) / MT, a.workers);
  const size_t lds = (size_t)MT * ((a.R + 31) / 32) * (kTermsOf<T, O> * 1024 + 64);
  if (a.R % 8 == 0) hipLaunchKernelGGL((k_expand_deep<T, O, MT, kWhole>), g, b, lds, a.stream, a);
  else hipLaunchKernelGGL((k_expand_deep<T, O, MT, kPart>), g, b, lds, a.stream, a);
}

// Blocks of columns one after the other where there are many tokens: up to four, as long
// as 1024 workgroups are left.  A batch of 12 prompts, us, one, two, four and eight blocks
// at most: rank 16, 4096 tokens 37.4, 29.2, 26.8 and 28.3, 16384 114, 102, 101 and 106; rank 64,
// 16384 tokens 147, 138, 134 and 134.  512, 1024 and 2048 workgroups left: rank 64, 64 tokens 14.8,
// 13.4 and 13.4, 16384 134, 134 and 138; rank 128, 301 tokens 29.3, 24.9 and 24.8, 4096 68.4, 68.5
// and 74.3.
template <typename T, typename O>
void second(AdapterArgs a, int64_t tiles) {
  constexpr int MT = sizeof(O) == 4 ? 2 : 4;
  const bool wide = many_tokens(tiles, a.R) && a.R > 32 && a.L > 0;
  const int64_t blocks = ((int64_t)a.N + 255) / 256, rows = wide ? (tiles + 3) / 4 : tiles;
  int64_t per = rows * a.workers * blocks / 1024;
  per = per < 1 ? 1 : per > 4 ? 4 : per;
  a.cols = (int)per * 256;
  const int64_t ranges = (blocks + per - 1) / per;
  if (wide) expand_deep<T, O, MT>(a, tiles, ranges);
  else if (a.R > 64) expand_deep<T, O, 1>(a, tiles, ranges);
  else expand<T, O>(a, tile_grid(ranges, tiles, a.workers));
}

template <typename T, int MT>
void shrink(AdapterArgs a, int64_t tiles) {
  // Tiles of 16 ranks, over as many workgroups as take four each, evenly.
  const int ranks = (a.R + 15) / 16, chunks = (ranks + 3) / 4;
  const dim3 b(256), g = tile_grid(a.splits * chunks, (tiles + MT - 1) / MT, a.workers);
  switch ((ranks + chunks - 1) / chunks) {
    case 1: hipLaunchKernelGGL((k_shrink<T, 1, MT>), g, b, 0, a.stream, a); break;
    case 2: hipLaunchKernelGGL((k_shrink<T, 2, MT>), g, b, 0, a.stream, a); break;
    case 3: hipLaunchKernelGGL((k_shrink<T, 3, MT>), g, b, 0, a.stream, a); break;
    default: hipLaunchKernelGGL((k_shrink<T, 4, MT>), g, b, 0, a.stream, a); break;
  }
}

template <typename T>
hipError_t add(AdapterArgs a) {
  const int64_t tiles = ((int64_t)a.M + 15) / 16;
  // Few tokens: a worker for each adapter that a tile may hold.  Many: the
  // tiles cover the device, and their tokens come in runs.  us with 16 workers, 4 and 1, 8
  // prompts / requests of one token over 16 adapters:
  //   tokens  rank 16                       rank 64                       rank 128
  //       64   7.7  7.7 15.0 / 8.6 13.5 34.6  12.8 12.8 28.7 / 16.7 31.0 87  14.8 15.0 34.2 / 21.8 32.2 94
  //      512  12.2 10.3 12.8 / 25.3 23.8 43   25.0 22.0 35.9 / 38.2 55.4 174 30.5 26.3 41.8 / 57.4 66.5 207
  //     1024  15.5 14.7 15.8 / 39.6 37.6 50   32.0 23.9 36.9 / 62.9 79.5 176 40.5 31.2 49.6 / 95.8 111 208
  //     8192  72.8 52.5 53.1 / 215 190 205    84.6 82.4 77.4 / 423 408 439   113 101 107 / 680 668 708
  //    16384  144 106 101 / 403 351 361       134 123 124 / 788 763 750      189 178 180 / 1262 1254 1238
  a.workers = tiles <= 32 ? 16 : tiles <= 512 ? 4 : 1;
  while (a.workers / 2 >= a.M) a.workers /= 2;
  if (a.R > 0 && a.L > 0 && a.K > 0) {
    a.share = ((a.K + 31) / 32 + a.splits * 4 - 1) / (a.splits * 4) * 32;  // a wave's: whole steps of 32
    if (many_tokens(tiles, a.R)) shrink<T, 4>(a, tiles);
    else shrink<T, 1>(a, tiles);
  } else {
    a.L = 0;  // no adapter at all
  }
  switch (a.out_dtype) {
    case kOutBF16: second<T, __bf16>(a, tiles); break;
    case kOutFP16: second<T, _Float16>(a, tiles); break;
    default: second<T, float>(a, tiles); break;
  }
  return hipGetLastError();
}

}  // namespace

// How many workgroups split K: enough that few tokens still cover the device, up to four
// and 2048 in all.  us with one and with four: one token of rank 16 7.5 and 5.6, 64 12.0 and 7.8,
// 1024 18.6 and 15.5, 2048 20.3 and 19.1; 256 of rank 64 31.0 and 19.1 (512 in all measures
// the same in each of these).  Tokens that go 64 to a workgroup take 512 in all, 16384
// of them two where more would double h, which the second product reads: one, two and four, rank 16
// 106, 101 and 100, rank 64 140, 134 and 134, rank 128 191, 175 and 177; 4096 tokens one and four, rank 16 37.5
// and 26.7, rank 128 81.2 and 68.6.
int adapter_splits(int64_t M, int64_t K, int64_t R) {
  const int64_t tiles = (M + 15) / 16;
  const bool many = many_tokens(tiles, R);
  const int64_t groups = many ? (tiles + 3) / 4 : tiles;
  int64_t most = (K + 255) / 256;
  most = most < kMaxSplits ? most : kMaxSplits;
  const int64_t s = (many ? 512 : 2048) / (groups > 0 ? groups : 1);
  return (int)(s < 1 ? 1 : s < most ? s : most);
}

hipError_t launch_add_adapters(const AdapterArgs& a) {
  return a.dtype == kOutBF16 ? add<__bf16>(a) : add<_Float16>(a);
}

}  // namespace fbg
