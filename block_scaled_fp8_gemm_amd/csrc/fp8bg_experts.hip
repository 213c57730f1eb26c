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

// ---------------------------------------------------------------------------
// Routing.  One wave per token; lane l holds the experts l * VPL .. l * VPL +
// VPL - 1, so that of equal values the lowest expert is in the lowest lane and
// first in it.
// ---------------------------------------------------------------------------
template <typename T, int VPL>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
  __shared__ double shared[4][64 * VPL];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = block_of_grid() * 4 + w;
  if (t >= a.T) return;  // whole waves, which meet at no barrier
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
  // Scores in 64 bits, and what ranks them: the logits themselves without a bias.
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
    double* v = shared[w];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (allowed[i]) v[lane * VPL + i] = a.group_score == FBG_GROUP_MAX || a.bias ? c[i] : s[i];
    wave_sync();
    double best = -kInf, second = -kInf;
    if (lane < a.groups) {
      for (int i = 0; i < size; ++i) {
        const double u = v[lane * size + i];
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
  float mine = 0.0f;
  int expert = 0;
  for (int j = 0; j < a.topk; ++j) {
    double best = -kInf;
    int at = 0x7fffffff;
    float score = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (allowed[i] && (at == 0x7fffffff || c[i] > best)) best = c[i], at = lane * VPL + i, score = (float)s[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double u = __shfl_xor(best, o, 64);
      const int ua = __shfl_xor(at, o, 64);
      const float us = __shfl_xor(score, o, 64);
      if (ua != 0x7fffffff && (at == 0x7fffffff || u > best || (u == best && ua < at))) best = u, at = ua, score = us;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) allowed[i] = allowed[i] && lane * VPL + i != at;
    if (lane == j) mine = score, expert = at;
  }
  if (a.renormalize) {
    const float total = wave_sum(mine);
    mine = mine / (total < 1e-20f ? 1e-20f : total);
  }
  if (lane < a.topk) wo[lane] = mine * a.scale, eo[lane] = expert;
}

template <typename T>
hipError_t route(const RouteArgs& a) {
  const dim3 g = wide_grid(((int64_t)a.T + 3) / 4), b(256);
  if (a.E <= 64) hipLaunchKernelGGL((k_route<T, 1>), g, b, 0, a.stream, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route<T, 4>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_route<T, 16>), g, b, 0, a.stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Into expert order: a stable counting sort of the T * topk choices by expert.
// Each workgroup ranks kSortBlock choices among themselves and counts its
// experts'; one workgroup turns the counts into starts; then every choice knows
// its row, and a workgroup per token copies the token's row to all of them.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 256, kSortItems = 4, kSortBlock = kSortThreads * kSortItems;

// Where a choice's expert is held here, its number, else -1.
__device__ __forceinline__ int local_expert(int id, int64_t first, int E) {
  const int64_t e = (int64_t)id - first;
  return e >= 0 && e < E ? (int)e : -1;
}

__global__ __launch_bounds__(kSortThreads) void k_rank(DispatchArgs a) {
  extern __shared__ int counts[];  // [waves][E]
  constexpr int kWaves = kSortThreads / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (block_of_grid() >= a.blocks) return;  // a whole workgroup
  for (int i = threadIdx.x; i < kWaves * a.E; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  int* mine = counts + w * a.E;
  const int64_t base = block_of_grid() * kSortBlock + w * 64 * kSortItems;
  int expert[kSortItems], rank[kSortItems];
#pragma unroll
  for (int r = 0; r < kSortItems; ++r) {
    const int64_t i = base + r * 64 + lane;
    expert[r] = i < a.n ? local_expert(a.experts[i], a.first, a.E) : -1;
    // The lanes that hold the same expert, found bit by bit.
    uint64_t same = __ballot(expert[r] >= 0);
    for (int bit = 1; bit < a.E; bit <<= 1) {
      const uint64_t set = __ballot((expert[r] & bit) != 0);
      same &= (expert[r] & bit) ? set : ~set;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    rank[r] = 0;
    if (expert[r] >= 0) {
      const int start = mine[expert[r]];
      rank[r] = start + before;
    }
    wave_sync();
    if (expert[r] >= 0 && before == 0) mine[expert[r]] += __popcll(same);
    wave_sync();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int run = 0;
    for (int i = 0; i < kWaves; ++i) {
      const int c = counts[i * a.E + e];
      counts[i * a.E + e] = run;
      run += c;
    }
    a.counts[block_of_grid() * a.E + e] = run;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortItems; ++r) {
    const int64_t i = base + r * 64 + lane;
    if (i < a.n) a.slots[i] = expert[r] >= 0 ? mine[expert[r]] + rank[r] : -1;
  }
}

// counts[b][e] becomes the first row of block b's choices of expert e.
__global__ __launch_bounds__(1024) void k_starts(DispatchArgs a) {
  __shared__ int sums[1024];
  const int e = threadIdx.x;
  int run = 0;
  if (e < a.E)
    for (int64_t b = 0; b < a.blocks; ++b) {
      const int c = a.counts[b * a.E + e];
      a.counts[b * a.E + e] = run;
      run += c;
    }
  sums[e] = run;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int u = e >= o ? sums[e - o] : 0;
    __syncthreads();
    sums[e] += u;
    __syncthreads();
  }
  if (e < a.E) a.offsets[e + 1] = sums[e];
  if (e == 0) a.offsets[0] = 0;
}

// Copies `bytes` bytes from any address to any other, by `threads` threads.
__device__ __forceinline__ void copy_row(const uint8_t* from, uint8_t* to, int64_t bytes, int t, int threads) {
  typedef unsigned int U4 __attribute__((ext_vector_type(4), aligned(1)));
  for (int64_t at = (int64_t)t * 16; at < bytes; at += (int64_t)threads * 16) {
    if (at + 16 <= bytes) {
      *reinterpret_cast<U4*>(to + at) = *reinterpret_cast<const U4*>(from + at);
    } else {
      for (int64_t i = at; i < bytes; ++i) to[i] = from[i];
    }
  }
}

__global__ __launch_bounds__(256) void k_move(DispatchArgs a) {
  const int64_t t = block_of_grid();
  if (t >= a.T) return;
  const uint8_t* x = a.x + t * a.x_pitch;
  for (int j = 0; j < a.topk; ++j) {
    const int64_t i = t * a.topk + j;
    const int rank = a.slots[i];
    if (rank < 0) continue;
    const int e = local_expert(a.experts[i], a.first, a.E);
    const int64_t slot = (int64_t)a.offsets[e] + a.counts[i / kSortBlock * a.E + e] + rank;
    copy_row(x, a.rows + slot * a.rows_pitch, a.row_bytes, threadIdx.x, 256);
    if (a.x_scale)
      copy_row(a.x_scale + t * a.scale_bytes, a.row_scale + slot * a.scale_bytes, a.scale_bytes, threadIdx.x, 256);
  }
  __syncthreads();  // every thread has read the ranks
  for (int j = threadIdx.x; j < a.topk; j += 256) {
    const int64_t i = t * a.topk + j;
    const int rank = a.slots[i];
    if (rank < 0) continue;
    const int e = local_expert(a.experts[i], a.first, a.E);
    a.slots[i] = a.offsets[e] + a.counts[i / kSortBlock * a.E + e] + rank;
  }
}

// ---------------------------------------------------------------------------
// Back into token order: a thread sums 16 bytes' worth of a token's columns.
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
__global__ __launch_bounds__(64) void k_combine(CombineArgs a) {
  constexpr int VE = 16 / (int)sizeof(T);
  const int64_t block = block_of_grid();
  const int64_t t = block / a.splits;
  if (t >= a.T) return;
  const int at = ((int)(block % a.splits) * 64 + (int)threadIdx.x) * VE;
  if (at >= a.D) return;
  const int n = a.D - at;
  float acc[VE] = {};
  if (a.base) {
    if (a.base_is_out) load_floats<O>(a.base, t * a.ldbase + at, n, acc);
    else load_floats<T>(a.base, t * a.ldbase + at, n, acc);
  }
  for (int j = 0; j < a.topk; ++j) {
    const int slot = a.slots[t * a.topk + j];
    if (slot < 0 || slot >= a.R) continue;
    const float w = a.weights[t * a.topk + j];
    float v[VE];
    load_floats<T>(a.rows, (int64_t)slot * a.ldrows + at, n, v);
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
  }
  O* out = reinterpret_cast<O*>(a.out) + t * a.ldout + at;
  O o[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) o[i] = (O)acc[i];
  if (n >= VE) {
    __builtin_memcpy(out, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < n) out[i] = o[i];
  }
}

template <typename T, typename O>
hipError_t combine(CombineArgs a) {
  constexpr int kCols = 64 * 16 / (int)sizeof(T);
  a.splits = (a.D + kCols - 1) / kCols;
  hipLaunchKernelGGL((k_combine<T, O>), wide_grid((int64_t)a.T * a.splits), dim3(64), 0, a.stream, a);
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

int64_t dispatch_workspace(int64_t n, int64_t E) { return (n + kSortBlock - 1) / kSortBlock * E * 4; }

hipError_t launch_dispatch(DispatchArgs a) {
  a.blocks = (a.n + kSortBlock - 1) / kSortBlock;
  if (a.blocks > 0)
    hipLaunchKernelGGL(k_rank, wide_grid(a.blocks), dim3(kSortThreads), kSortThreads / 64 * a.E * sizeof(int), a.stream, a);
  hipLaunchKernelGGL(k_starts, dim3(1), dim3(1024), 0, a.stream, a);
  if (a.blocks > 0) hipLaunchKernelGGL(k_move, wide_grid(a.T), dim3(256), 0, a.stream, a);
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
