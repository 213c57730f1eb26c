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

constexpr int64_t kGridX = 1 << 20;
inline dim3 wide_grid(int64_t blocks) {
  return blocks <= kGridX ? dim3((unsigned)blocks) : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t block_of_grid() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

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
  T v[8];
  load_some(row, at, n, v);
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
// Worker `first` of `count` calls pass(adapter) for its share.
template <typename F>
__device__ __forceinline__ void for_passes(int id, int first, int count, const F& pass) {
  uint64_t todo = __ballot(id >= 0) & 0xffff;
  for (int p = 0; todo; ++p) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == cur);
    if (p % count == first) pass(cur);
  }
}

// h of 16 tokens over one slice of K for one adapter of theirs, or each in
// turn; the four waves split the slice, and their sums meet in LDS.  RT tiles
// of 16 ranks at a time; the loads of U steps are in flight together.
template <typename T, int RT>
__global__ __launch_bounds__(256) void k_shrink(AdapterArgs a) {
  constexpr int U = RT == 1 ? 8 : 4;
  typedef typename Vec8<T>::type V;
  __shared__ v4f part[RT][4][64];  // [tile of 16 ranks][wave][lane]
  int64_t block = block_of_grid();
  const int split = (int)(block % a.splits);
  block /= a.splits;
  const int worker = (int)(block % a.workers);
  const int64_t m0 = block / a.workers * 16;
  if (m0 >= a.M) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
  const int id = adapter_of(a, m0 + j);
  // A wave's share: whole steps of 32.
  const int steps = (a.K + 31) / 32, per = (steps + a.splits * 4 - 1) / (a.splits * 4);
  const int first = (split * 4 + w) * per * 32;
  const int last = first + per * 32 < a.K ? first + per * 32 : a.K;
  float* h = a.h + ((int64_t)split * a.M + m0 + j) * a.pitch;
  for_passes(id, worker, a.workers, [&](int cur) {
    const bool mine = id == cur;
    // Lanes of other tokens read the row of one that is meant.
    const int64_t m = m0 + (mine ? j : __builtin_ctzll(__ballot(mine)));
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
#pragma unroll
        for (int u = 0; u < U; ++u)
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
        for (int i = 1; i < 4; ++i) s += part[w][i][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i >= a.R) s[i] = 0.0f;
        if (mine) *reinterpret_cast<v4f*>(h + r) = s;
      }
      __syncthreads();
    }
  });
}

// 16 tokens by blocks of 64 columns per wave.  Row i of the first operand's
// tile t is column 32 (t / 2) + 8 (i / 4) + 4 (t % 2) + i % 4 of the block, so that a
// lane's results are of one token and 8 columns next to one another, twice.  h stays in
// fp32: the fp32 MFMA takes it and the weights as they are.  Each token
// belongs to one pass, which alone writes its row; the first worker writes the
// rows without an adapter.  DEEP: more than 64 ranks, h read again for each
// block of columns.
template <typename T, typename O, int RT, bool DEEP>
__global__ __launch_bounds__(256) void k_expand(AdapterArgs a) {
  int64_t block = block_of_grid();
  const int64_t n_first = block % a.col_blocks * a.cols;
  block /= a.col_blocks;
  const int worker = (int)(block % a.workers);
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int64_t m0 = (block / a.workers * 4 + (threadIdx.x >> 6)) * 16;
  if (m0 >= a.M) return;  // whole waves, which meet at no barrier
  const int64_t n_last = n_first + a.cols < a.N ? n_first + a.cols : a.N;
  const int64_t m = m0 + j;
  const int id = adapter_of(a, m);
  const O* yrow = reinterpret_cast<const O*>(a.y) + m * a.ldy;
  O* orow = reinterpret_cast<O*>(a.out) + m * a.ldout;
  const auto store = [&](int64_t n, const O (&v)[8]) {
    if (n + 8 <= a.N) {
      __builtin_memcpy(orow + n, v, sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < a.N) orow[n + i] = v[i];
    }
  };
  const auto load_h = [&](int r0, float scale, v4f (&h)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      h[i] = v4f{};
      if (r0 + 16 * i < a.pitch) {
        const float* p = a.h + m * a.pitch + r0 + 16 * i + 4 * g;
        for (int s = 0; s < a.splits; ++s) h[i] += *reinterpret_cast<const v4f*>(p + (int64_t)s * a.M * a.pitch);
        h[i] *= scale;
      }
    }
  };
  for_passes(id, worker, a.workers, [&](int cur) {
    const bool mine = id == cur;
    const float scale = a.scales ? a.scales[cur] : 1.0f;
    const T* B = reinterpret_cast<const T*>(a.B) + (int64_t)cur * a.N * a.R;
    v4f h[RT] = {};
    if (!DEEP && mine) load_h(0, scale, h);
    for (int64_t n0 = n_first; n0 < n_last; n0 += 64) {
      O y[2][8];
      if (mine) {
#pragma unroll
        for (int q = 0; q < 2; ++q) load_some(yrow, (int)n0 + 32 * q + 8 * g, a.N, y[q]);
      }
      const T* row[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t n = n0 + 32 * (t >> 1) + 8 * (j >> 2) + 4 * (t & 1) + (j & 3);
        row[t] = B + (n < a.N ? n : a.N - 1) * a.R;
      }
      v4f acc[4] = {};
      for (int r0 = 0; r0 < (DEEP ? a.R : 1); r0 += 16 * RT) {
        if (DEEP && mine) load_h(r0, scale, h);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          T b[4][4];
#pragma unroll
          for (int t = 0; t < 4; ++t) load_some(row[t], r0 + 16 * i + 4 * g, a.R, b[t]);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int t = 0; t < 4; ++t)
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)b[t][u], h[i][u], acc[t], 0, 0, 0);
        }
      }
      // A lane's results are of its own token: those of the others' adapters,
      // which may hold infinities, go nowhere.
      if (mine) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t n = n0 + 32 * q + 8 * g;
          if (n >= a.N) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[q][i] = (O)((float)y[q][i] + acc[2 * q + (i >> 2)][i & 3]);
          store(n, y[q]);
        }
      }
    }
  });
  if (worker == 0 && !a.in_place && m < a.M && id < 0)
    for (int64_t n = n_first + 8 * g; n < n_last; n += 32) {
      O y[8];
      load_some(yrow, (int)n, a.N, y);
      store(n, y);
    }
}

template <typename T, typename O>
void expand(const AdapterArgs& a, dim3 g) {
  const dim3 b(256);
  if (a.R <= 16) hipLaunchKernelGGL((k_expand<T, O, 1, false>), g, b, 0, a.stream, a);
  else if (a.R <= 32) hipLaunchKernelGGL((k_expand<T, O, 2, false>), g, b, 0, a.stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL((k_expand<T, O, 4, false>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_expand<T, O, 4, true>), g, b, 0, a.stream, a);
}

template <typename T>
hipError_t add(AdapterArgs a) {
  const int64_t tiles = ((int64_t)a.M + 15) / 16;
  // Few tokens: a worker for each adapter that a tile may hold.  Many: the
  // tiles cover the device, and their tokens come in runs.
  a.workers = tiles > 64 ? 1 : a.M < 16 ? a.M : 16;
  if (a.R > 0 && a.L > 0 && a.K > 0) {
    const dim3 g = wide_grid(tiles * a.workers * a.splits), b(256);
    if (a.R <= 16) hipLaunchKernelGGL((k_shrink<T, 1>), g, b, 0, a.stream, a);
    else if (a.R <= 32) hipLaunchKernelGGL((k_shrink<T, 2>), g, b, 0, a.stream, a);
    else hipLaunchKernelGGL((k_shrink<T, 4>), g, b, 0, a.stream, a);
  } else {
    a.L = 0;  // no adapter at all
  }
  const int64_t groups = (tiles + 3) / 4 * a.workers, blocks = ((int64_t)a.N + 63) / 64;
  int64_t per = groups * blocks / 2048;
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  a.cols = (int)per * 64;
  a.col_blocks = (int)((blocks + per - 1) / per);
  const dim3 g = wide_grid(groups * a.col_blocks);
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
  const int64_t tiles = (M + 15) / 16, most = (K + 511) / 512;
  int64_t s = 512 / (tiles > 0 ? tiles : 1);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

hipError_t launch_add_adapters(const AdapterArgs& a) {
  return a.dtype == kOutBF16 ? add<__bf16>(a) : add<_Float16>(a);
}

}  // namespace fbg
