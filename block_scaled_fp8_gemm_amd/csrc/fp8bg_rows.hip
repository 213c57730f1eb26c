// gfx950 kernels that work on one token's row at a time: the token quantiser
// of the int8 products, and the norms between two blocks.
//
//   quantise:  s = max(max_k |x[k]|, 1e-12) / 127
//              q[k] = round-to-nearest-even of clamp(x[k] / s, -127, 127)
//   norms:     u = rms(h) * (post + o),  r = alpha * x + gate * u,
//              y = rms(r) * (pre + o),   rms(v) = v / sqrt(mean(v^2) + eps)
//
// All arithmetic is fp32 whatever the tensors' type; r and y are rounded
// once, and the second norm takes r as it was before its rounding.  The
// quotients x / s are correctly rounded divisions.
#include "fp8bg_device.hpp"
#include "fp8bg_internal.h"

namespace fbg {

namespace {

template <typename T>
__device__ __forceinline__ float ld1(const void* p, int64_t i) {
  return (float)reinterpret_cast<const T*>(p)[i];
}

// Weights are of the activations' type T or fp32.
template <typename T>
__device__ __forceinline__ float ldw(const void* p, int i, bool f32) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : ld1<T>(p, i);
}

// |v| as an integer: ordered like |v|, infinities above every finite value
// and NaNs above those, so a row's maximum keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A row with a NaN or an infinity gets that as its scale; the quotients that
// are then NaN take code 0, so the products of such a row are NaN and not
// finite and wrong.
__device__ __forceinline__ int code_i8(float v, float s) {
  float t = v / s;
  t = t == t ? t : 0.0f;
  return (int)__builtin_rintf(fminf(fmaxf(t, -127.0f), 127.0f));
}

__device__ __forceinline__ float scale_of(uint32_t amax_bits, float top) {
  const float a = __uint_as_float(amax_bits);
  return (a < 1e-12f ? 1e-12f : a) / top;
}

template <int NW>
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += slots[i];
  __syncthreads();
  return v;
}

template <int NW>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* slots) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) v = max(v, slots[i]);
  __syncthreads();
  return v;
}

template <typename T>
__global__ __launch_bounds__(256) void k_quantize_tokens(QuantArgs a) {
  __shared__ uint32_t slots[4];
  const int m = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + (int64_t)m * a.ldx;
  int8_t* q = a.q + (int64_t)m * a.ldq;
  uint32_t amax = 0;
  for (int k = threadIdx.x; k < a.K; k += 256) amax = max(amax, abs_bits((float)x[k]));
  const float s = scale_of(block_max<4>(amax, slots), 127.0f);
  for (int k = threadIdx.x; k < a.K; k += 256) q[k] = (int8_t)code_i8((float)x[k], s);
  if (threadIdx.x == 0) a.scale[m] = s;
}

template <typename T>
__global__ __launch_bounds__(256) void k_block_norm(NormArgs a) {
  __shared__ float fslots[4];
  __shared__ uint32_t uslots[4];
  const int m = blockIdx.x, tid = threadIdx.x;
  const bool wf32 = a.wdtype == kOutFP32;
  const void* h = reinterpret_cast<const T*>(a.h) + (int64_t)m * a.ldh;
  const void* x = reinterpret_cast<const T*>(a.x) + (int64_t)m * a.ldx;
  float rstd_h = 1.0f;
  if (a.post) {
    float ss = 0.0f;
    for (int d = tid; d < a.D; d += 256) {
      const float v = ld1<T>(h, d);
      ss = __builtin_fmaf(v, v, ss);
    }
    rstd_h = 1.0f / __builtin_sqrtf(block_sum<4>(ss, fslots) / (float)a.D + a.eps);
  }
  auto r_at = [&](int d) {
    float u = ld1<T>(h, d);
    if (a.post) u = (u * rstd_h) * (ldw<T>(a.post, d, wf32) + a.weight_offset);
    if (a.gate) u = u * ld1<T>(a.gate, (int64_t)m * a.gate_row + (int64_t)d * a.gate_col);
    return a.x ? a.residual_scale * ld1<T>(x, d) + u : u;
  };
  float ss = 0.0f;
  T* r = reinterpret_cast<T*>(a.r) + (int64_t)m * a.ldr;
  for (int d = tid; d < a.D; d += 256) {
    const float v = r_at(d);
    r[d] = (T)v;
    ss = __builtin_fmaf(v, v, ss);
  }
  if (!a.pre) return;
  const float rstd = 1.0f / __builtin_sqrtf(block_sum<4>(ss, fslots) / (float)a.D + a.eps);
  auto y_at = [&](int d) { return (r_at(d) * rstd) * (ldw<T>(a.pre, d, wf32) + a.weight_offset); };
  if (a.quant == FBG_QUANT_NONE) {
    T* y = reinterpret_cast<T*>(a.y) + (int64_t)m * a.ldy;
    for (int d = tid; d < a.D; d += 256) y[d] = (T)y_at(d);
  } else if (a.quant == FBG_QUANT_INT8) {
    uint32_t amax = 0;
    for (int d = tid; d < a.D; d += 256) amax = max(amax, abs_bits(y_at(d)));
    const float s = scale_of(block_max<4>(amax, uslots), 127.0f);
    int8_t* y = reinterpret_cast<int8_t*>(a.y) + (int64_t)m * a.ldy;
    for (int d = tid; d < a.D; d += 256) y[d] = (int8_t)code_i8(y_at(d), s);
    if (tid == 0) a.y_scale[m] = s;
  } else {  // E4M3, one scale per 128 columns: one wave per group, two columns per lane
    uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + (int64_t)m * a.ldy;
    for (int g = tid >> 6; g < a.D / 128; g += 4) {
      const int d = g * 128 + 2 * (tid & 63);
      const float v0 = y_at(d), v1 = y_at(d + 1);
      uint32_t amax = max(abs_bits(v0), abs_bits(v1));
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, 64));
      const float s = scale_of(amax, 448.0f);
      const int c = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(v0 / s, -448.0f), 448.0f),
                                                    fminf(fmaxf(v1 / s, -448.0f), 448.0f), 0, false);
      y[d] = (uint8_t)(c & 255);
      y[d + 1] = (uint8_t)((c >> 8) & 255);
      if ((tid & 63) == 0) a.y_scale[(int64_t)m * (a.D / 128) + g] = s;
    }
  }
}

}  // namespace

hipError_t launch_quantize_tokens(const QuantArgs& a) {
  const dim3 g((unsigned)a.M), b(256);
  switch (a.dtype) {
    case kOutBF16: hipLaunchKernelGGL(k_quantize_tokens<__bf16>, g, b, 0, a.stream, a); break;
    case kOutFP16: hipLaunchKernelGGL(k_quantize_tokens<_Float16>, g, b, 0, a.stream, a); break;
    default: hipLaunchKernelGGL(k_quantize_tokens<float>, g, b, 0, a.stream, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_block_norm(const NormArgs& a) {
  const dim3 g((unsigned)a.M), b(256);
  switch (a.dtype) {
    case kOutBF16: hipLaunchKernelGGL(k_block_norm<__bf16>, g, b, 0, a.stream, a); break;
    case kOutFP16: hipLaunchKernelGGL(k_block_norm<_Float16>, g, b, 0, a.stream, a); break;
    default: hipLaunchKernelGGL(k_block_norm<float>, g, b, 0, a.stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace fbg
