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
// codes are those of correctly rounded divisions x / s.
#include <type_traits>

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

// Sums and maxima over the TPR threads of a row: a wave's butterfly, then one
// word per wave through LDS.  Every call has slots of its own, so one barrier
// is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v += slots[i];
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slots) {
  v = lanes_max<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = max(v, slots[i]);
  }
  return v;
}

// Rows are taken in chunks of 16 bytes (VE elements), chunk c starting at
// element c * VE wherever the row starts: a whole chunk is one 16-byte access
// at the elements' own alignment, the last one goes element by element, and
// elements past n read as zero.
template <typename T>
struct Chunk {
  static constexpr int VE = 16 / (int)sizeof(T);
  T v[VE];
};

//
// STREAM: the non-temporal hint, for the tensors that are read once (16384 x
// 4096: norm to int8 132 -> 113 us, quantiser 36.8 -> 35.3 us in the same
// shapes); the weights and a gate per channel, which every row reads, go without
// it (the gate with it: 16384 x 8192 202 against 185 us, 1024 x 4096 10.4 and 9.8,
// 16384 x 256 11.7 and 11.2).
template <bool STREAM, typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int at, int n) {
  Chunk<T> c;
  if (at + Chunk<T>::VE <= n) {
    typedef unsigned int U4 __attribute__((ext_vector_type(4), aligned(2)));  // rows start where they may
    const U4* p = reinterpret_cast<const U4*>(row + at);
    const U4 w = STREAM ? __builtin_nontemporal_load(p) : *p;
    __builtin_memcpy(&c, &w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < Chunk<T>::VE; ++i) c.v[i] = at + i < n ? row[at + i] : (T)0.0f;
  }
  return c;
}

// VE values of type S (of any size) to row[at ..], those before n.  STREAM: the
// non-temporal hint, for 16-byte chunks (a template flag: of two stores that
// differ only in it the compiler makes one without).
template <bool STREAM = false, typename S, int VE>
__device__ __forceinline__ void store_values(S* row, int at, int n, const S (&v)[VE]) {
  if (at + VE <= n) {
    if constexpr (STREAM) {
      static_assert(sizeof(v) == 16, "a chunk");
      typedef unsigned int U4 __attribute__((ext_vector_type(4), aligned(2)));
      U4 w;
      __builtin_memcpy(&w, v, 16);
      __builtin_nontemporal_store(w, reinterpret_cast<U4*>(row + at));
    } else {
      __builtin_memcpy(row + at, v, sizeof(v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (at + i < n) row[at + i] = v[i];
  }
}

// Weights as floats: of type T, or fp32.
template <typename T, int VE>
__device__ __forceinline__ void load_weights(const void* w, bool f32, int at, int n, float offset, float (&o)[VE]) {
  if (f32) {
    if (at + VE <= n) {
      __builtin_memcpy(o, reinterpret_cast<const float*>(w) + at, sizeof(o));
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] = at + i < n ? reinterpret_cast<const float*>(w)[at + i] : 0.0f;
    }
  } else {
    const Chunk<T> c = load_chunk<false>(reinterpret_cast<const T*>(w), at, n);
#pragma unroll
    for (int i = 0; i < VE; ++i) o[i] = (float)c.v[i];
  }
#pragma unroll
  for (int i = 0; i < VE; ++i) o[i] += offset;
}

// Int8 codes of VE values with scale s.  EXACT: by division.  Else the
// quotient is t = v * (1/s) and one correction step, t + (v - t*s) * (1/s):
// its code is that of the correctly rounded v / s for every bf16 or fp16
// value in a row with any bf16 or fp16 maximum (checked for all pairs), and for
// the fp32 values of a norm next to every boundary between two codes (checked
// for random maxima), at 3 operations where the division takes about 10.
template <bool EXACT, int VE>
__device__ __forceinline__ void int8_codes(const float (&v)[VE], float s, float y, int8_t (&q)[VE]) {
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    float t;
    if constexpr (EXACT) {
      t = v[i] / s;
    } else {
      t = v[i] * y;
      t = __builtin_fmaf(__builtin_fmaf(-t, s, v[i]), y, t);
    }
    q[i] = (int8_t)(int)__builtin_rintf(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f));
  }
}

// A scale that is a NaN or an infinity: the row (or the 128 columns) held
// one.  All its quotients are 0 or NaN, so every code is 0, and the products of
// such a row are NaN.  (E4M3's clamp makes -448 of a quotient that is NaN,
// whose products would be an infinity of the weights' sign.)
__device__ __forceinline__ bool finite(float s) { return abs_bits(s) < 0x7f800000u; }

// A launch holds less than 2^32 threads along x: many rows take a grid of two
// dimensions.
constexpr int64_t kGridX = 1 << 20;
inline dim3 row_grid(int64_t blocks) {
  return blocks <= kGridX ? dim3((unsigned)blocks) : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t block_of_grid() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// A row is held by TPR threads: half a wave or one (eight or four rows to a
// workgroup), or a workgroup of its own.
constexpr int threads(int tpr) { return tpr <= 64 ? 256 : tpr; }
constexpr int waves(int tpr) { return tpr <= 64 ? 1 : tpr / 64; }
constexpr int rows_per_block(int tpr) { return threads(tpr) / tpr; }

// ---------------------------------------------------------------------------
// Token quantiser.  A row stays in the registers of its TPR threads, ITEMS
// chunks each, so x is read once; all loads are issued before the maximum is
// taken.
// ---------------------------------------------------------------------------
template <typename T, int TPR, int ITEMS>
__global__ __launch_bounds__(threads(TPR)) void k_quantize_tokens(QuantArgs a) {
  constexpr int VE = Chunk<T>::VE;
  __shared__ uint32_t slots[waves(TPR)];
  const int t = threadIdx.x % TPR;
  const int64_t m = block_of_grid() * rows_per_block(TPR) + threadIdx.x / TPR;
  if (m >= a.M) return;  // a whole workgroup, or rows within a wave, which meet at no barrier
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
  Chunk<T> c[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) c[i] = load_chunk<true>(x, (i * TPR + t) * VE, a.K);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int j = 0; j < VE; ++j) amax = max(amax, abs_bits((float)c[i].v[j]));
  const float s = scale_of(row_max<TPR>(amax, slots), 127.0f);
  const float y = 1.0f / s;
  int8_t* q = a.q + m * a.ldq;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    float v[VE];
    int8_t o[VE] = {};
#pragma unroll
    for (int j = 0; j < VE; ++j) v[j] = (float)c[i].v[j];
    if (finite(s)) int8_codes<sizeof(T) == 4>(v, s, y, o);
    store_values(q, (i * TPR + t) * VE, a.K, o);
  }
  if (t == 0) a.scale[m] = s;
}

// Rows too long for the registers: read twice.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_long(QuantArgs a) {
  __shared__ uint32_t slots[4];
  const int64_t m = block_of_grid();
  if (m >= a.M) return;
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
  int8_t* q = a.q + m * a.ldq;
  uint32_t amax = 0;
  for (int k = threadIdx.x; k < a.K; k += 256) amax = max(amax, abs_bits((float)x[k]));
  const float s = scale_of(row_max<256>(amax, slots), 127.0f);
  for (int k = threadIdx.x; k < a.K; k += 256) q[k] = (int8_t)code_i8((float)x[k], s);
  if (threadIdx.x == 0) a.scale[m] = s;
}

// ---------------------------------------------------------------------------
// Norms.  As above a row of h, x and the gate is loaded into registers once,
// and r stays there in fp32 between the two norms.
// ---------------------------------------------------------------------------
template <typename T, int TPR, int ITEMS, bool STREAM>
__global__ __launch_bounds__(threads(TPR)) void k_block_norm(NormArgs a) {
  constexpr int VE = Chunk<T>::VE;
  __shared__ float slots[2 * waves(TPR)];
  __shared__ uint32_t uslots[waves(TPR)];
  const int t = threadIdx.x % TPR;
  const int64_t m = block_of_grid() * rows_per_block(TPR) + threadIdx.x / TPR;
  if (m >= a.M) return;
  const bool wf32 = a.wdtype == kOutFP32;
  const T* h = reinterpret_cast<const T*>(a.h) + m * a.ldh;
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
  const T* gate = reinterpret_cast<const T*>(a.gate) + m * a.gate_row;
  Chunk<T> ch[ITEMS], cx[ITEMS], cg[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) ch[i] = load_chunk<true>(h, (i * TPR + t) * VE, a.D);
  if (a.x) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) cx[i] = load_chunk<true>(x, (i * TPR + t) * VE, a.D);
  }
  if (a.gate) {
    if (a.gate_col == 1) {
      // Every row reads it.  (Few rows, one chunk per thread in a wave or more:
      // the hint says nothing there.)
      const bool shared = (ITEMS > 1 || TPR == 32) && a.gate_row == 0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        cg[i] = shared ? load_chunk<false>(gate, (i * TPR + t) * VE, a.D) : load_chunk<true>(gate, (i * TPR + t) * VE, a.D);
    } else {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const int d = (i * TPR + t) * VE + j;
          cg[i].v[j] = d < a.D ? gate[d * a.gate_col] : (T)0.0f;
        }
    }
  }
  float rstd_h = 1.0f;
  if (a.post) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j) ss = __builtin_fmaf((float)ch[i].v[j], (float)ch[i].v[j], ss);
    rstd_h = 1.0f / __builtin_sqrtf(row_sum<TPR>(ss, slots) / (float)a.D + a.eps);
  }
  float r[ITEMS][VE];
  float ss = 0.0f;
  T* ro = reinterpret_cast<T*>(a.r) + m * a.ldr;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = (i * TPR + t) * VE;
#pragma unroll
    for (int j = 0; j < VE; ++j) r[i][j] = (float)ch[i].v[j];
    if (a.post) {
      float w[VE];
      load_weights<T>(a.post, wf32, at, a.D, a.weight_offset, w);
#pragma unroll
      for (int j = 0; j < VE; ++j) r[i][j] = (r[i][j] * rstd_h) * w[j];
    }
    if (a.gate) {
#pragma unroll
      for (int j = 0; j < VE; ++j) r[i][j] *= (float)cg[i].v[j];
    }
    if (a.x) {
#pragma unroll
      for (int j = 0; j < VE; ++j) r[i][j] = a.residual_scale * (float)cx[i].v[j] + r[i][j];
    }
    T o[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      o[j] = (T)r[i][j];
      if (at + j < a.D) ss = __builtin_fmaf(r[i][j], r[i][j], ss);
    }
    store_values<STREAM>(ro, at, a.D, o);
  }
  if (!a.pre) return;
  const float rstd = 1.0f / __builtin_sqrtf(row_sum<TPR>(ss, slots + waves(TPR)) / (float)a.D + a.eps);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    float w[VE];
    load_weights<T>(a.pre, wf32, (i * TPR + t) * VE, a.D, a.weight_offset, w);
#pragma unroll
    for (int j = 0; j < VE; ++j) r[i][j] = (r[i][j] * rstd) * w[j];
  }
  if (a.quant == FBG_QUANT_NONE) {
    T* yo = reinterpret_cast<T*>(a.y) + m * a.ldy;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      T o[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) o[j] = (T)r[i][j];
      store_values(yo, (i * TPR + t) * VE, a.D, o);
    }
  } else if (a.quant == FBG_QUANT_INT8) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if ((i * TPR + t) * VE + j < a.D) amax = max(amax, abs_bits(r[i][j]));
    const float s = scale_of(row_max<TPR>(amax, uslots), 127.0f);
    const float y = 1.0f / s;
    int8_t* yo = reinterpret_cast<int8_t*>(a.y) + m * a.ldy;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      int8_t o[VE] = {};
      if (finite(s)) int8_codes<false>(r[i], s, y, o);
      store_values(yo, (i * TPR + t) * VE, a.D, o);
    }
    if (t == 0) a.y_scale[m] = s;
  } else {  // E4M3: 128 / VE neighbouring threads hold a group of 128 columns (D % 128 == 0: whole groups)
    uint8_t* yo = reinterpret_cast<uint8_t*>(a.y) + m * a.ldy;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = (i * TPR + t) * VE;
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) amax = max(amax, abs_bits(r[i][j]));
      const float s = scale_of(lanes_max<128 / VE>(amax), 448.0f);
      const float y = 1.0f / s;
      uint8_t o[VE];
#pragma unroll
      for (int j = 0; j < VE; j += 2) {
        float q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // The remainder with its sign turned: as v - e * s the step makes
          // +0 of a negative zero.
          const float v = r[i][j + k], e = v * y;
          q[k] = __builtin_amdgcn_fmed3f(__builtin_fmaf(-__builtin_fmaf(e, s, -v), y, e), -448.0f, 448.0f);
        }
        const int w = finite(s) ? __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false) : 0;
        o[j] = (uint8_t)(w & 255);
        o[j + 1] = (uint8_t)((w >> 8) & 255);
      }
      store_values(yo, at, a.D, o);
      if (t % (128 / VE) == 0 && at < a.D) a.y_scale[m * (a.D / 128) + at / 128] = s;
    }
  }
}

// Rows too long for the registers: h, x and the gate are read again for
// every pass.
template <typename T>
__global__ __launch_bounds__(256) void k_block_norm_long(NormArgs a) {
  __shared__ float fslots[8];
  __shared__ uint32_t uslots[4];
  const int64_t m = block_of_grid();
  if (m >= a.M) return;
  const int tid = threadIdx.x;
  const bool wf32 = a.wdtype == kOutFP32;
  const void* h = reinterpret_cast<const T*>(a.h) + m * a.ldh;
  const void* x = reinterpret_cast<const T*>(a.x) + m * a.ldx;
  float rstd_h = 1.0f;
  if (a.post) {
    float ss = 0.0f;
    for (int d = tid; d < a.D; d += 256) {
      const float v = ld1<T>(h, d);
      ss = __builtin_fmaf(v, v, ss);
    }
    rstd_h = 1.0f / __builtin_sqrtf(row_sum<256>(ss, fslots) / (float)a.D + a.eps);
  }
  auto r_at = [&](int d) {
    float u = ld1<T>(h, d);
    if (a.post) u = (u * rstd_h) * (ldw<T>(a.post, d, wf32) + a.weight_offset);
    if (a.gate) u = u * ld1<T>(a.gate, m * a.gate_row + (int64_t)d * a.gate_col);
    return a.x ? a.residual_scale * ld1<T>(x, d) + u : u;
  };
  float ss = 0.0f;
  T* r = reinterpret_cast<T*>(a.r) + m * a.ldr;
  for (int d = tid; d < a.D; d += 256) {
    const float v = r_at(d);
    r[d] = (T)v;
    ss = __builtin_fmaf(v, v, ss);
  }
  if (!a.pre) return;
  const float rstd = 1.0f / __builtin_sqrtf(row_sum<256>(ss, fslots + 4) / (float)a.D + a.eps);
  auto y_at = [&](int d) { return (r_at(d) * rstd) * (ldw<T>(a.pre, d, wf32) + a.weight_offset); };
  if (a.quant == FBG_QUANT_NONE) {
    T* y = reinterpret_cast<T*>(a.y) + m * a.ldy;
    for (int d = tid; d < a.D; d += 256) y[d] = (T)y_at(d);
  } else if (a.quant == FBG_QUANT_INT8) {
    uint32_t amax = 0;
    for (int d = tid; d < a.D; d += 256) amax = max(amax, abs_bits(y_at(d)));
    const float s = scale_of(row_max<256>(amax, uslots), 127.0f);
    int8_t* y = reinterpret_cast<int8_t*>(a.y) + m * a.ldy;
    for (int d = tid; d < a.D; d += 256) y[d] = (int8_t)code_i8(y_at(d), s);
    if (tid == 0) a.y_scale[m] = s;
  } else {  // E4M3, one scale per 128 columns: one wave per group, two columns per lane
    uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + m * a.ldy;
    for (int g = tid >> 6; g < a.D / 128; g += 4) {
      const int d = g * 128 + 2 * (tid & 63);
      const float v0 = y_at(d), v1 = y_at(d + 1);
      uint32_t amax = max(abs_bits(v0), abs_bits(v1));
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, 64));
      const float s = scale_of(amax, 448.0f);
      const int c = finite(s) ? __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(v0 / s, -448.0f), 448.0f),
                                                                fminf(fmaxf(v1 / s, -448.0f), 448.0f), 0, false)
                              : 0;
      y[d] = (uint8_t)(c & 255);
      y[d + 1] = (uint8_t)((c >> 8) & 255);
      if ((tid & 63) == 0) a.y_scale[m * (a.D / 128) + g] = s;
    }
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

template <typename F>
hipError_t with_items(int items, const F& f) {
  return items == 1 ? f(Int<1>{}) : items == 2 ? f(Int<2>{}) : f(Int<4>{});
}

// Calls launch(threads per row, chunks per thread).
template <typename F>
hipError_t with_shape(int tpr, int items, const F& launch) {
  return with_items(items, [&](auto it) {
    switch (tpr) {
      case 32: return launch(Int<32>{}, it);
      case 64: return launch(Int<64>{}, it);
      case 128: return launch(Int<128>{}, it);
      case 256: return launch(Int<256>{}, it);
      case 512: return launch(Int<512>{}, it);
      default: return launch(Int<1024>{}, it);
    }
  });
}

// Threads per row and chunks per thread for `rows` rows of `chunks` chunks
// (items 0: too long for the registers).  With few rows the row is spread
// over as many threads as it has chunks, since only latency counts (64 x 4096
// bf16: norm 4.5 us with 1 chunk per thread, 5.1 with 2, 6.6 with 4).  With
// many, more bytes in flight per wave win: 2 chunks (16384 x 4096 bf16: norm to
// int8 111 us then, against 144 with 1 and 119 with 4; quantiser 34.7 against 50
// and 34.2), and 4 in the long rows of `many` (2048 x 16384: norm 70 us against
// 80 with 2, quantiser 19.7 against 20.9).  A row of at most 32 chunks takes
// half a wave (16384 x 256: norm 13.2 us, 19.3 on a whole one).
struct RowShape {
  int tpr, items;
};
inline RowShape row_shape(int64_t rows, int64_t chunks, bool many) {
  int items = rows < 512 || chunks <= 32 ? 1 : many ? 4 : 2, tpr = 32;
  for (;; items *= 2) {
    while (tpr < 1024 && chunks > (int64_t)tpr * items) tpr *= 2;
    if (chunks <= (int64_t)tpr * items) return {tpr, items};
    if (items == 4) return {0, 0};
  }
}

template <typename T>
hipError_t quantize(const QuantArgs& a) {
  const int64_t chunks = ((int64_t)a.K + Chunk<T>::VE - 1) / Chunk<T>::VE;
  const RowShape s = row_shape(a.M, chunks, chunks > 512);
  if (s.items == 0) {
    hipLaunchKernelGGL(k_quantize_long<T>, row_grid(a.M), dim3(256), 0, a.stream, a);
    return hipGetLastError();
  }
  return with_shape(s.tpr, s.items, [&](auto tp, auto it) {
    constexpr int TPR = decltype(tp)::value, ITEMS = decltype(it)::value;
    const dim3 g = row_grid(((int64_t)a.M + rows_per_block(TPR) - 1) / rows_per_block(TPR)), b(threads(TPR));
    hipLaunchKernelGGL((k_quantize_tokens<T, TPR, ITEMS>), g, b, 0, a.stream, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t norm(const NormArgs& a) {
  // Four fp32 chunks hold as many values as two 16-bit ones: the fp32 rows
  // stay at 2 (8192 columns: 238 us against 243).
  const int64_t chunks = ((int64_t)a.D + Chunk<T>::VE - 1) / Chunk<T>::VE;
  const RowShape s = row_shape(a.M, chunks, sizeof(T) == 2 && chunks > 512);
  // A residual of more than 4 MB goes out with the non-temporal hint where y,
  // and not the residual, is what the next product reads: 103 us against 110 at
  // 16384 x 4096 to int8, 11.1 against 12.1 at 1024 x 4096; in a chain of norm,
  // product and quantiser of the residual 233 and 236 us at 16384 rows, 31.6 and
  // 32.3 at 1024, but 19.1 and 18.5 at 256 (2 MB).  On y, or on the quantiser's
  // codes, the hint gains up to 6 us and costs the pass that reads them next 30
  // (16384 x 4096).
  const bool stream = a.pre && (int64_t)a.M * a.D * (int64_t)sizeof(T) > ((int64_t)4 << 20);
  if (s.items == 0) {
    hipLaunchKernelGGL(k_block_norm_long<T>, row_grid(a.M), dim3(256), 0, a.stream, a);
    return hipGetLastError();
  }
  return with_shape(s.tpr, s.items, [&](auto tp, auto it) {
    constexpr int TPR = decltype(tp)::value, ITEMS = decltype(it)::value;
    const dim3 g = row_grid(((int64_t)a.M + rows_per_block(TPR) - 1) / rows_per_block(TPR)), b(threads(TPR));
    if constexpr (ITEMS > 1) {  // (rows of at most 32 chunks are left out: 512 bytes each)
      if (stream) {
        hipLaunchKernelGGL((k_block_norm<T, TPR, ITEMS, true>), g, b, 0, a.stream, a);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((k_block_norm<T, TPR, ITEMS, false>), g, b, 0, a.stream, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_quantize_tokens(const QuantArgs& a) {
  switch (a.dtype) {
    case kOutBF16: return quantize<__bf16>(a);
    case kOutFP16: return quantize<_Float16>(a);
    default: return quantize<float>(a);
  }
}

hipError_t launch_block_norm(const NormArgs& a) {
  switch (a.dtype) {
    case kOutBF16: return norm<__bf16>(a);
    case kOutFP16: return norm<_Float16>(a);
    default: return norm<float>(a);
  }
}

}  // namespace fbg
