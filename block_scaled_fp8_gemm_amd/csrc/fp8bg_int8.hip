// gfx950 kernels of the 8-bit-integer products: int8 activations with one fp32
// scale per token, int8 weights with one per output channel.
//
//   C[m,n] = a_s[m] * b_s[n] * sum_k A[m,k] * B[n,k]  (+ bias[n])
//
// The scales do not depend on k, so the whole sum stays in the MFMA's int32
// accumulators, exactly (|sum| <= 128 * 128 * K < 2^31 for K <= 131071, which
// the entry points check); only the epilogue works in fp32:
//   c = fl(fl(a_s * b_s) * fl(acc)) (+ bias), then one rounding to C's type.
// Integer sums do not depend on their order, so every tile shape and every
// split of K gives the same bits.
//
// Operand order as in the FP8 kernels: weight rows n on the MFMA's first
// operand, activation rows m on the second, so a lane ends with ONE row m and
// 4 consecutive columns n of each 16x16 block.
//
// The grouped (mixture-of-experts) form gives rows offsets[e] ..
// offsets[e+1]-1 of A the weight B[e]; see expert_of_slot.
#include "fp8bg_device.hpp"
#include "fp8bg_internal.h"

namespace fbg {

namespace {

// 16x16 block, 64 deep: acc[r] += sum_k X[4*(l>>4) + r][k] * Y[l & 15][k].
// Lane l holds row (l & 15) of each operand and 16 consecutive k (which 16
// does not matter as long as both operands agree).
__device__ __forceinline__ v4i mfma_i8(const v4i& x, const v4i& y, const v4i& acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, acc, 0, 0, 0);
}

// Grouped form.  Expert e owns the row-tile slots [s(e), s(e+1)) with
// s(e) = floor(offsets[e] / BM) + e.  With offsets[e] = q*BM + r and n rows,
// s(e+1) - s(e) = floor((r + n) / BM) + 1 >= ceil(n / BM): its tiles always
// fit, and s(e) needs offsets[e] alone, so every lane tests its own experts
// at once instead of a prefix sum over tile counts.  Slots past an expert's
// last tile exit.  There are floor(M / BM) + E slots.
// Returns whether slot `t` holds rows; all threads of the workgroup call it.
template <int BM>
__device__ __forceinline__ bool expert_of_slot(const int* __restrict__ offsets, int E, int M, int t, int& e_out,
                                               int& m0, int& m_end) {
  __shared__ int found[3];
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int lo = offsets[e], hi = offsets[e + 1];
    lo = lo < 0 ? 0 : (lo > M ? M : lo);  // malformed offsets never lead outside the operands
    hi = hi < lo ? lo : (hi > M ? M : hi);
    const int i = t - (lo / BM + e);
    if (i >= 0 && (int64_t)i * BM < hi - lo) {
      found[0] = e;
      found[1] = lo + i * BM;
      found[2] = hi;
    }
  }
  __syncthreads();
  e_out = found[0];
  m0 = found[1];
  m_end = found[2];
  return e_out >= 0;
}

// c = (a_s * b_s) * acc (+ bias) for 4 consecutive columns n .. n+3 of one
// row; columns at or past N are not read.
__device__ __forceinline__ v4f scale4(const v4i& acc, float as, const float* __restrict__ b_s,
                                      const float* __restrict__ bias, int n, int N) {
  v4f c;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int nn = n + r < N ? n + r : N - 1;
    c[r] = (as * b_s[nn]) * (float)acc[r];
    if (bias) c[r] = c[r] + bias[nn];
  }
  return c;
}

// 16 bytes of a row at byte k0, zeros from byte K on.  Rows start at any
// address: a whole chunk is one unaligned 16-byte load.
__device__ __forceinline__ v4i load_chunk(const uint8_t* __restrict__ row, int k0, int K) {
  v4i v = {0, 0, 0, 0};
  if (k0 + 16 <= K) {
    __builtin_memcpy(&v, row + k0, 16);
  } else if (k0 < K) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k0 + i < K) w[i >> 2] |= (uint32_t)row[k0 + i] << (8 * (i & 3));
    v = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  }
  return v;
}

// ---------------------------------------------------------------------------
// Any sizes and any alignment: BM x BN tiles, 2 x 2 waves, 128 bytes of K per
// step through registers into swizzled LDS tiles (swz_row), the next step's
// loads in flight while this one is multiplied.
// ---------------------------------------------------------------------------
template <int BM, int BN, int OUT, int GRP>
__global__ __launch_bounds__(256) void k_i8_any(I8Args a) {
  constexpr int WM = BM / 2, WN = BN / 2, IB = WM / 16, JB = WN / 16;
  constexpr int AP = BM * 8 / 256, BP = BN * 8 / 256;  // 16-byte chunks per thread
  __shared__ __attribute__((aligned(16))) uint8_t smem[(BM + BN) * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles_n = (a.N + BN - 1) / BN;
  const int lid = xcd_remap(blockIdx.x, (int)gridDim.x);
  int m0, n0, m_end = a.M, e = 0;
  if constexpr (GRP) {
    if (!expert_of_slot<BM>(a.offsets, a.E, a.M, lid / tiles_n, e, m0, m_end)) return;
    n0 = (lid % tiles_n) * BN;
  } else {
    int tm, tn;
    raster(lid, (a.M + BM - 1) / BM, tiles_n, 8, tm, tn);
    m0 = tm * BM;
    n0 = tn * BN;
  }
  const uint8_t* B = a.B + (int64_t)e * a.N * a.ldb;
  const float* b_s = a.b_s + (int64_t)e * a.N;

  // Chunk p*256 + tid of a tile: row (p*256 + tid) / 8, 16-byte chunk tid & 7.
  const uint8_t* arow[AP];
  const uint8_t* brow[BP];
#pragma unroll
  for (int p = 0; p < AP; ++p) {
    const int m = m0 + (p * 256 + tid) / 8;
    arow[p] = a.A + (int64_t)(m < m_end ? m : m_end - 1) * a.lda;
  }
#pragma unroll
  for (int p = 0; p < BP; ++p) {
    const int n = n0 + (p * 256 + tid) / 8;
    brow[p] = B + (int64_t)(n < a.N ? n : a.N - 1) * a.ldb;
  }
  v4i acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  v4i ra[AP], rb[BP];
  auto fetch = [&](int k) {
    const int c = k + 16 * (tid & 7);
#pragma unroll
    for (int p = 0; p < AP; ++p) ra[p] = load_chunk(arow[p], c, a.K);
#pragma unroll
    for (int p = 0; p < BP; ++p) rb[p] = load_chunk(brow[p], c, a.K);
  };
  fetch(0);
  for (int k = 0; k < a.K; k += 128) {
    __syncthreads();  // the previous step's reads are done
#pragma unroll
    for (int p = 0; p < AP; ++p) {
      const int r = (p * 256 + tid) / 8;
      *reinterpret_cast<v4i*>(smem + 128 * r + 16 * ((tid & 7) ^ swz_row(r))) = ra[p];
    }
#pragma unroll
    for (int p = 0; p < BP; ++p) {
      const int r = (p * 256 + tid) / 8;
      *reinterpret_cast<v4i*>(smem + BM * 128 + 128 * r + 16 * ((tid & 7) ^ swz_row(r))) = rb[p];
    }
    __syncthreads();
    if (k + 128 < a.K) fetch(k + 128);
    v8i bf[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) bf[j] = load_frag_lds_sw(smem + BM * 128, wn * WN + 16 * j, lane);
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      const v8i af = load_frag_lds_sw(smem, wm * WM + 16 * i, lane);
      const v4i alo = __builtin_shufflevector(af, af, 0, 1, 2, 3), ahi = __builtin_shufflevector(af, af, 4, 5, 6, 7);
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const v4i blo = __builtin_shufflevector(bf[j], bf[j], 0, 1, 2, 3);
        const v4i bhi = __builtin_shufflevector(bf[j], bf[j], 4, 5, 6, 7);
        acc[i][j] = mfma_i8(blo, alo, acc[i][j]);
        acc[i][j] = mfma_i8(bhi, ahi, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int m = m0 + wm * WM + 16 * i + (lane & 15);
    if (m >= m_end) continue;
    const float as = a.a_s[m];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int n = n0 + wn * WN + 16 * j + 4 * (lane >> 4);
      const int cnt = a.N - n < 4 ? a.N - n : 4;
      if (cnt > 0) store4<OUT>(a.C, (int64_t)m * a.ldc + n, scale4(acc[i][j], as, b_s, a.bias, n, a.N), cnt, a.vec);
    }
  }
}

// The empty sum: every output is its column's bias, or zero.
template <int OUT>
__global__ __launch_bounds__(256) void k_i8_no_k(I8Args a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.M * a.N) return;
  const int64_t m = i / a.N, n = i - m * a.N;
  store1<OUT>(a.C, m * a.ldc + n, a.bias ? a.bias[n] : 0.0f);
}

template <int BM, int BN, int GRP>
hipError_t launch_any(const I8Args& a, int64_t grid) {
  const dim3 g((unsigned)grid), b(256);
  switch (a.out) {
    case kOutBF16: hipLaunchKernelGGL((k_i8_any<BM, BN, kOutBF16, GRP>), g, b, 0, a.stream, a); break;
    case kOutFP16: hipLaunchKernelGGL((k_i8_any<BM, BN, kOutFP16, GRP>), g, b, 0, a.stream, a); break;
    case kOutFP32: hipLaunchKernelGGL((k_i8_any<BM, BN, kOutFP32, GRP>), g, b, 0, a.stream, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8(const I8Args& a) {
  const bool grouped = a.offsets != nullptr;
  if (a.K == 0 || (grouped && a.E == 0)) {
    const int64_t grid = ((int64_t)a.M * a.N + 255) / 256;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid), b(256);
    switch (a.out) {
      case kOutBF16: hipLaunchKernelGGL(k_i8_no_k<kOutBF16>, g, b, 0, a.stream, a); break;
      case kOutFP16: hipLaunchKernelGGL(k_i8_no_k<kOutFP16>, g, b, 0, a.stream, a); break;
      default: hipLaunchKernelGGL(k_i8_no_k<kOutFP32>, g, b, 0, a.stream, a); break;
    }
    return hipGetLastError();
  }
  const int64_t tiles_n = (a.N + 63) / 64;
  const int64_t grid = (grouped ? (int64_t)a.M / 64 + a.E : ((int64_t)a.M + 63) / 64) * tiles_n;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return grouped ? launch_any<64, 64, 1>(a, grid) : launch_any<64, 64, 0>(a, grid);
}

}  // namespace fbg
