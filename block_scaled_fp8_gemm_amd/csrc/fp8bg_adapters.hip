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

// h of 16 tokens over one slice of K; the four waves split the slice, and their
// sums meet in LDS.
template <typename T>
__global__ __launch_bounds__(256) void k_shrink(AdapterArgs a) {
  __shared__ v4f part[4][4][64];  // [tile of 16 ranks][wave][lane]
  const int64_t block = block_of_grid();
  const int64_t m0 = block / a.splits * 16;
  if (m0 >= a.M) return;
  const int split = (int)(block % a.splits);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
  const int id = adapter_of(a, m0 + j);
  // A wave's share: whole steps of 32.
  const int steps = (a.K + 31) / 32, per = (steps + a.splits * 4 - 1) / (a.splits * 4);
  const int first = (split * 4 + w) * per * 32;
  const int last = first + per * 32 < a.K ? first + per * 32 : a.K;
  const int64_t m = m0 + j < a.M ? m0 + j : a.M - 1;
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
  float* h = a.h + ((int64_t)split * a.M + m0 + j) * a.pitch;
  uint64_t todo = __ballot(id >= 0) & 0xffff;
  while (todo) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == cur);
    const T* A = reinterpret_cast<const T*>(a.A) + (int64_t)cur * a.R * a.K;
    for (int r0 = 0; r0 < a.R; r0 += 64) {
      v4f acc[4] = {};
      for (int k = first; k < last; k += 32) {
        const auto xf = load8(x, k + 8 * g, a.K);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r0 + 16 * i < a.R) {
            const int r = r0 + 16 * i + j < a.R ? r0 + 16 * i + j : a.R - 1;
            acc[i] = mfma32(load8(A + (int64_t)r * a.K, k + 8 * g, a.K), xf, acc[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) part[i][w][lane] = acc[i];
      __syncthreads();
      const int r = r0 + 16 * w + 4 * g;  // wave w: ranks r0 + 16 w ..
      if (r0 + 16 * w < a.R) {
        v4f s = part[w][0][lane];
#pragma unroll
        for (int i = 1; i < 4; ++i) s += part[w][i][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i >= a.R) s[i] = 0.0f;
        if (id == cur) *reinterpret_cast<v4f*>(h + r) = s;
      }
      __syncthreads();
    }
  }
}

// 16 tokens by 32 columns per wave.  Row i of the first operand is column
// 8 * (i / 4) + i % 4 of the tile, or that plus 4, so that the two results of a
// lane are 8 columns next to one another of one token.  h stays in fp32: the
// fp32 MFMA takes it and the weights as they are.
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_expand(AdapterArgs a) {
  const int64_t block = block_of_grid();
  const int64_t m0 = block / a.col_blocks * 16;
  if (m0 >= a.M) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
  const int64_t n0 = (block % a.col_blocks) * 128 + w * 32;
  if (n0 >= a.N) return;  // whole waves, which meet at no barrier
  const int64_t m = m0 + j;
  const int id = adapter_of(a, m);
  uint64_t todo = __ballot(id >= 0) & 0xffff;
  if (todo == 0 && a.in_place) return;
  v4f delta[2] = {};
  while (todo) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == cur);
    const bool mine = id == cur;
    v4f acc[2] = {};
    const float scale = a.scales ? a.scales[cur] : 1.0f;
    const T* B[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t n = n0 + 8 * (j >> 2) + 4 * t + (j & 3);
      B[t] = reinterpret_cast<const T*>(a.B) + ((int64_t)cur * a.N + (n < a.N ? n : a.N - 1)) * a.R;
    }
    for (int r0 = 0; r0 < a.R; r0 += 16) {
      const int r = r0 + 4 * g;
      v4f h = {};
      if (mine) {
        for (int s = 0; s < a.splits; ++s)
          h += *reinterpret_cast<const v4f*>(a.h + ((int64_t)s * a.M + m) * a.pitch + r);
        h *= scale;
      }
      T b[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) load_some(B[t], r, a.R, b[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)b[t][i], h[i], acc[t], 0, 0, 0);
    }
    // A lane's results are of its own token: those of the others' adapters, which
    // may hold infinities, are dropped.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) delta[t][i] = mine ? acc[t][i] : delta[t][i];
  }
  if (m >= a.M || (id < 0 && a.in_place)) return;
  const int n = (int)n0 + 8 * g;
  if (n >= a.N) return;
  O y[8];
  load_some(reinterpret_cast<const O*>(a.y) + m * a.ldy, n, a.N, y);
  if (id >= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (O)((float)y[i] + delta[i >> 2][i & 3]);
  }
  O* out = reinterpret_cast<O*>(a.out) + m * a.ldout + n;
  if (n + 8 <= a.N) {
    __builtin_memcpy(out, y, sizeof(y));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < a.N) out[i] = y[i];
  }
}

template <typename T>
hipError_t add(AdapterArgs a) {
  if (a.R > 0 && a.L > 0 && a.K > 0) {
    const int64_t tiles = ((int64_t)a.M + 15) / 16;
    hipLaunchKernelGGL(k_shrink<T>, wide_grid(tiles * a.splits), dim3(256), 0, a.stream, a);
  } else {
    a.L = 0;  // no adapter at all
  }
  a.col_blocks = (a.N + 127) / 128;
  const dim3 g = wide_grid(((int64_t)a.M + 15) / 16 * a.col_blocks), b(256);
  switch (a.out_dtype) {
    case kOutBF16: hipLaunchKernelGGL((k_expand<T, __bf16>), g, b, 0, a.stream, a); break;
    case kOutFP16: hipLaunchKernelGGL((k_expand<T, _Float16>), g, b, 0, a.stream, a); break;
    default: hipLaunchKernelGGL((k_expand<T, float>), g, b, 0, a.stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace

// How many workgroups split K: enough that few tokens still cover the device.
int adapter_splits(int64_t M, int64_t K) {
  const int64_t tiles = (M + 15) / 16, most = (K + 511) / 512;
  int64_t s = 512 / (tiles > 0 ? tiles : 1);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

hipError_t launch_add_adapters(const AdapterArgs& a) {
  return a.dtype == kOutBF16 ? add<__bf16>(a) : add<_Float16>(a);
}

}  // namespace fbg
