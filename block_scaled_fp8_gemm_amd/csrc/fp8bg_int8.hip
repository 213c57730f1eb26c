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
#include <stdio.h>

#include <type_traits>

#include "fp8bg_device.hpp"
#include "fp8bg_int8_configs.h"
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
// `found`: three words of LDS, free again afterwards.
//
// Malformed offsets never lead outside the operands: each is clamped, and
// where several experts claim a slot the last of them has it alone (its rows
// come from one thread).
//
// REST: slots for an expert's tiles from its second on.  They start at
// floor(offsets[e] / BM): floor((r + n) / BM) >= ceil(n / BM) - 1 of them, and
// floor(M / BM) in all.
template <int BM, bool REST = false>
__device__ __forceinline__ bool expert_of_slot(const int* __restrict__ offsets, int E, int M, int t, int& e_out,
                                               int& m0, int& m_end, int* found) {
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int mine = -1, first = 0, last = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int lo = offsets[e], hi = offsets[e + 1];
    lo = lo < 0 ? 0 : (lo > M ? M : lo);
    hi = hi < lo ? lo : (hi > M ? M : hi);
    const int s = t - (lo / BM + (REST ? 0 : e)), i = REST ? s + 1 : s;
    if (s >= 0 && (int64_t)i * BM < hi - lo) {
      mine = e;
      first = lo + i * BM;
      last = hi;
    }
  }
  if (mine >= 0) atomicMax(&found[0], mine);
  __syncthreads();
  e_out = found[0];
  if (mine >= 0 && mine == e_out) {
    found[1] = first;
    found[2] = last;
  }
  __syncthreads();
  m0 = found[1];
  m_end = found[2];
  __syncthreads();
  return e_out >= 0;
}

// This workgroup's tile: launches hold fewer workgroups than a product may
// have, each one starting at tile `first`.
__device__ __forceinline__ int logical_tile(const I8Args& a) {
  return a.first + xcd_remap(blockIdx.x, (int)gridDim.x);
}

// An fp32 value as it is rounded: a product whose conversion to fp16 follows
// becomes one instruction with one rounding otherwise, which is not what the
// other kernels and types give (it differs in about one value of 1e5).
__device__ __forceinline__ float rounded(float x) {
  asm("" : "+v"(x));
  return x;
}

// c = (a_s * b_s) * acc (+ bias) for 4 consecutive columns n .. n+3 of one
// row; columns at or past N are not read.
__device__ __forceinline__ v4f scale4(const v4i& acc, float as, const float* __restrict__ b_s,
                                      const float* __restrict__ bias, int n, int N) {
  v4f c;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int nn = n + r < N ? n + r : N - 1;
    c[r] = rounded((as * b_s[nn]) * (float)acc[r]);
    if (bias) c[r] = c[r] + bias[nn];
  }
  return c;
}

// `count` (at most 4) consecutive values of a row to C, which starts at any
// element: four go out as one store, whatever their alignment (3093 x 2707 x 100:
// 17.3 us, value by value 23.0; 301 x 1537 x 1000 5.8 and 6.1).
template <int OUT>
__device__ __forceinline__ void store_run(void* C, int64_t idx, const v4f& v, int count) {
  typedef typename Out<OUT>::T T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T4 T4U __attribute__((aligned(2)));
  T* p = reinterpret_cast<T*>(C) + idx;
  T4 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = Out<OUT>::cvt(v[r]);
  if (count >= 4) {
    *reinterpret_cast<T4U*>(p) = o;
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < count) p[r] = o[r];
  }
}

// Rows that start anywhere and end anywhere (K >= 16).  The 16-byte chunk at
// byte k0 is read at min(k0, K - 16), so that it never leaves the row and
// needs no branch; both operands read the same window, and in the activations'
// (keep_tail) the bytes before k0, which an earlier chunk holds, are zeroed.
__device__ __forceinline__ v4i load_window(const uint8_t* __restrict__ row, int k0, int K) {
  v4i v;
  __builtin_memcpy(&v, row + (k0 < K - 16 ? k0 : K - 16), 16);
  return v;
}
__device__ __forceinline__ v4i keep_tail(v4i v, int k0, int K) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int drop = k0 - (K - 16) - 4 * i;  // leading bytes of dword i to zero
    v[i] = drop <= 0 ? v[i] : drop >= 4 ? 0 : (int)((uint32_t)v[i] & (0xffffffffu << (8 * drop)));
  }
  return v;
}

// Every LDS access of the workgroup's waves before this is done after it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---------------------------------------------------------------------------
// Any sizes and any alignment: BM x BN tiles, 2 x 2 waves, 128 bytes of K per
// step through registers into two swizzled LDS tiles (swz_row).  The chunks of
// AHEAD steps are in flight in registers, since a step's arithmetic is far
// shorter than a load's latency, and with two tiles a step needs one barrier.
// ---------------------------------------------------------------------------
template <int BM, int BN, int AHEAD, int OUT, int GRP>
__global__ __launch_bounds__(256) void k_i8_any(I8Args a) {
  constexpr int WM = BM / 2, WN = BN / 2, IB = WM / 16, JB = WN / 16;
  constexpr int AP = BM * 8 / 256, BP = BN * 8 / 256;  // 16-byte chunks per thread
  constexpr int TILE = (BM + BN) * 128;
  static_assert(AHEAD % 2 == 0, "step k of an unrolled round uses tile k & 1");
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * TILE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles_n = (a.N + BN - 1) / BN;
  const int lid = logical_tile(a);
  int m0, n0, m_end = a.M, e = 0;
  if constexpr (GRP) {
    if (!expert_of_slot<BM>(a.offsets, a.E, a.M, lid / tiles_n, e, m0, m_end, reinterpret_cast<int*>(smem))) return;
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

  v4i ra[AHEAD][AP], rb[AHEAD][BP];
  auto fetch = [&](int k, v4i (&fa)[AP], v4i (&fb)[BP]) {
    const int c = k + 16 * (tid & 7);
#pragma unroll
    for (int p = 0; p < AP; ++p) fa[p] = load_window(arow[p], c, a.K);
#pragma unroll
    for (int p = 0; p < BP; ++p) fb[p] = load_window(brow[p], c, a.K);
  };
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) fetch(128 * s, ra[s], rb[s]);
  for (int k0 = 0; k0 < a.K; k0 += 128 * AHEAD) {
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      const int k = k0 + 128 * s;
      if (k >= a.K) break;
      uint8_t* tile = smem + (s & 1) * TILE;
      if (k + 128 > a.K) {
#pragma unroll
        for (int p = 0; p < AP; ++p) ra[s][p] = keep_tail(ra[s][p], k + 16 * (tid & 7), a.K);
      }
#pragma unroll
      for (int p = 0; p < AP; ++p) {
        const int r = (p * 256 + tid) / 8;
        *reinterpret_cast<v4i*>(tile + 128 * r + 16 * ((tid & 7) ^ swz_row(r))) = ra[s][p];
      }
#pragma unroll
      for (int p = 0; p < BP; ++p) {
        const int r = (p * 256 + tid) / 8;
        *reinterpret_cast<v4i*>(tile + BM * 128 + 128 * r + 16 * ((tid & 7) ^ swz_row(r))) = rb[s][p];
      }
      // The chunk's registers are free again: the step AHEAD further on.
      fetch(k + 128 * AHEAD, ra[s], rb[s]);
      lds_barrier();  // the tile's last reads were two steps ago, before the previous barrier
      v8i bf[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j) bf[j] = load_frag_lds_sw(tile + BM * 128, wn * WN + 16 * j, lane);
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        const v8i af = load_frag_lds_sw(tile, wm * WM + 16 * i, lane);
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
      if (cnt > 0) store_run<OUT>(a.C, (int64_t)m * a.ldc + n, scale4(acc[i][j], as, b_s, a.bias, n, a.N), cnt);
    }
  }
}

// ---------------------------------------------------------------------------
// The skinny kernel: few rows, so the weights' bytes and the launch's latency
// are what counts.  A workgroup takes 16*NB columns and ROWS rows; its KW
// waves split K, each loading its own fragments straight into registers in
// groups of U slices of 64 K bytes (wave w takes groups w, w + KW, ..), all of
// a group's loads in flight together and the next group's once it is
// multiplied (K = 4096 over 8 waves is two such rounds); the waves' sums meet
// in LDS.  ROWS = 8 halves a 16-row tile's activation bytes: the upper
// eight rows of the MFMA repeat the last one and are not stored.
//
// FAST: rows of whole 16-byte chunks on 16-byte boundaries; else chunks at any
// alignment (load_window).
//
// Grouped: one workgroup per (expert, column tile) takes the expert's first
// ROWS rows, and further ones (floor(M / ROWS) slots, see expert_of_slot) the
// rest: walked by the first, all rows in one expert took 137 us where they take
// 9.9 (64 experts of 128 x 4096, 512 rows), and 617 where they take 13.8 (256 of
// 128 x 1001, 3072 rows); spread evenly both ways take the same.
// ---------------------------------------------------------------------------
template <int NB, int ROWS, int KW, int U, bool FAST, int GRP>
__global__ __launch_bounds__(64 * KW) void k_i8_skinny(I8Args a) {
  static_assert(ROWS <= 16, "one row block of the MFMA");
  __shared__ v4i red[KW][NB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  int e = 0, m0, m_end, tn;
  if constexpr (GRP) {
    const int g = a.first + (int)blockIdx.x, firsts = a.E * tiles_n;
    if (g < firsts) {
      const int lid = xcd_remap(g, firsts);
      e = lid / tiles_n;
      tn = lid - e * tiles_n;
      int lo = a.offsets[e], hi = a.offsets[e + 1];
      lo = lo < 0 ? 0 : (lo > a.M ? a.M : lo);  // malformed offsets never lead outside the operands
      hi = hi < lo ? lo : (hi > a.M ? a.M : hi);
      m0 = lo;
      m_end = hi;
    } else {
      const int lid = xcd_remap(g - firsts, a.M / ROWS * tiles_n);
      if (!expert_of_slot<ROWS, true>(a.offsets, a.E, a.M, lid / tiles_n, e, m0, m_end, reinterpret_cast<int*>(red)))
        return;
      tn = lid % tiles_n;
    }
    if (m0 >= m_end) return;
    m0 = __builtin_amdgcn_readfirstlane(m0);
    m_end = __builtin_amdgcn_readfirstlane(m0 + ROWS < m_end ? m0 + ROWS : m_end);
    e = __builtin_amdgcn_readfirstlane(e);
  } else {
    const int lid = logical_tile(a), tiles_m = (a.M + ROWS - 1) / ROWS;
    tn = lid / tiles_m;
    m0 = (lid - tn * tiles_m) * ROWS;
    m_end = m0 + ROWS < a.M ? m0 + ROWS : a.M;
  }
  const int n0 = tn * 16 * NB, r = lane & 15, h = lane >> 4;
  const uint8_t* brow[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int n = n0 + 16 * j + r < a.N ? n0 + 16 * j + r : a.N - 1;
    brow[j] = a.B + ((int64_t)e * a.N + n) * a.ldb;
  }
  const int groups = (a.K + 64 * U - 1) / (64 * U);
  const uint8_t* arow = a.A + (int64_t)(m0 + r < m_end ? m0 + r : m_end - 1) * a.lda;
  v4i acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = v4i{0, 0, 0, 0};
  v4i fa[U], fb[U][NB];
  auto load = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (g * U + u) * 64 + 16 * h;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (FAST && GRP) fb[u][j] = *reinterpret_cast<const v4i*>(brow[j] + (k < a.K ? k : 0));
        else if constexpr (FAST) fb[u][j] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(brow[j] + (k < a.K ? k : 0)));
        else fb[u][j] = load_window(brow[j], k, a.K);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (g * U + u) * 64 + 16 * h;
      if constexpr (FAST) fa[u] = *reinterpret_cast<const v4i*>(arow + (k < a.K ? k : 0));
      else fa[u] = load_window(arow, k, a.K);
    }
  };
  auto multiply = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (g * U + u) * 64 + 16 * h;  // FAST: chunks past K were read from the row's start
      v4i f = fa[u];
      if constexpr (FAST) f = k < a.K ? f : v4i{0, 0, 0, 0};
      else if ((g * U + u + 1) * 64 > a.K) f = keep_tail(f, k, a.K);
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] = mfma_i8(fb[u][j], f, acc[j]);
    }
  };
  for (int g = wave; g < groups; g += KW) {
    load(g);
    __builtin_amdgcn_sched_barrier(0);  // every load of the group in flight before the first product
    multiply(g);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  for (int j = wave; j < NB; j += KW) {
    const int m = m0 + r, n = n0 + 16 * j + 4 * h;
    v4i s = red[0][j][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) s += red[w][j][lane];
    const int cnt = a.N - n < 4 ? a.N - n : 4;
    if (m < m_end && cnt > 0) {
      const v4f c = scale4(s, a.a_s[m], a.b_s + (int64_t)e * a.N, a.bias, n, a.N);
      const int64_t at = (int64_t)m * a.ldc + n;
      switch (a.out) {
        case kOutBF16: store_run<kOutBF16>(a.C, at, c, cnt); break;
        case kOutFP16: store_run<kOutFP16>(a.C, at, c, cnt); break;
        default: store_run<kOutFP32>(a.C, at, c, cnt); break;
      }
    }
  }
}

typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// The slim kernel, between the skinny one and the tiles: small tiles, so that
// a few dozen rows still give every compute unit its share of the weights to
// stream, whose four waves split K: of every 128-byte step in the ring, wave
// w multiplies slice w for the whole BM x BN.  In the tile kernel a wave of
// such a tile has one or two MFMAs between an LDS read and the next that waits
// for it, and a step takes that latency four times; here it takes it once, and
// a round of U steps shares one barrier.  The four sums meet in LDS.
//
// Rows and loads as in the tile kernel.  A round's fragments are multiplied
// while the next one's are read; the refill of a slot goes out behind those
// reads, past the barrier of the round after it.
//
// 64 x 4096 x 4096: 6.4 us, where the tile kernel's 32 x 64 takes 10.1 and the
// skinny kernel 14.7; 17 x 4096 x 4096 6.2 (9.3).  One round per step instead
// of two steps 7.4; the refill ahead of the reads 9.1.  Grouped, the weights
// take the non-temporal hint, one expert's being read by one row of tiles: 64
// tokens over 256 experts of 512 x 4096 88.8 -> 79.2 us; dense, where the row
// tiles share them, it costs (64 x 4096 x 4096 7.8 us).
// ---------------------------------------------------------------------------
template <int BM, int BN, int U, int STAGES>
struct SlimLds {
  static constexpr int STEP = (BM + BN) * 128, RING = STAGES * U * STEP;
  static constexpr int PITCH = BN * 4 + 16, SUMS = 4 * BM * PITCH;  // each wave's sums, rows padded by 16 bytes
  static constexpr int BYTES = RING > SUMS ? RING : SUMS;
};

template <int BM, int BN, int U, int STAGES, int GRP>
__global__ __launch_bounds__(256, 2) void k_i8_slim(I8Args a) {
  typedef SlimLds<BM, BN, U, STAGES> L;
  constexpr int IB = BM / 32, JB = BN / 32, SLOT = U * L::STEP;
  constexpr int LPS = U * (IB + JB);  // loads per wave and round
  static_assert((STAGES - 1) * LPS < 64 && STAGES >= 3, "vmcnt counts at most 63 outstanding loads");
  __shared__ __attribute__((aligned(16))) uint8_t smem[L::BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles_n = (a.N + BN - 1) / BN;
  int m0, n0, m_end = a.M, e = 0;
  {
    const int lid = logical_tile(a);
    if constexpr (GRP) {
      if (!expert_of_slot<BM>(a.offsets, a.E, a.M, lid / tiles_n, e, m0, m_end, reinterpret_cast<int*>(smem))) return;
      n0 = (lid % tiles_n) * BN;
    } else {  // the row tiles of a column are neighbours: they share its weights
      const int tiles_m = (a.M + BM - 1) / BM;
      n0 = lid / tiles_m * BN;
      m0 = lid % tiles_m * BM;
    }
  }
  m0 = __builtin_amdgcn_readfirstlane(m0);  // scalar registers, as the buffer resources have to be
  n0 = __builtin_amdgcn_readfirstlane(n0);
  m_end = __builtin_amdgcn_readfirstlane(m_end);
  e = __builtin_amdgcn_readfirstlane(e);
  auto upto = [](int64_t rows, int64_t ld, int64_t len) {
    const int64_t b = (rows - 1) * ld + len;
    return (uint32_t)(b < UINT32_MAX ? b : UINT32_MAX);
  };
  const buf_rsrc rA = make_rsrc_n(a.A + (int64_t)m0 * a.lda, upto(m_end - m0, a.lda, a.K));
  const buf_rsrc rB = make_rsrc_n(a.B + ((int64_t)e * a.N + n0) * a.ldb, upto(a.N - n0, a.ldb, a.K));
  const int nk = (a.K + 127) / 128, rounds = (nk + U - 1) / U;
  // Image i*4 + wave of a tile: rows 32i + 8*wave .., this lane's row and chunk.
  const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz_row(row);
  const uint32_t tail = (nk - 1) * 128 + 16 * chunk >= a.K ? 16u * (uint32_t)chunk : 0u;  // as in the tile kernel
  uint32_t aoff[IB], boff[JB];
#pragma unroll
  for (int i = 0; i < IB; ++i) aoff[i] = (uint32_t)(32 * i + row) * (uint32_t)a.lda + 16u * (uint32_t)chunk;
#pragma unroll
  for (int j = 0; j < JB; ++j) boff[j] = (uint32_t)(32 * j + row) * (uint32_t)a.ldb + 16u * (uint32_t)chunk;
  lds_u8* const lds = (lds_u8*)smem;
  // Round g: the steps g*U .. g*U + U-1 (past the last one, that one again).
  auto load_round = [&](int g, int slot) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = g * U + u < nk ? g * U + u : nk - 1;
      const uint32_t sub = k == nk - 1 ? tail : 0u;
      lds_u8* base = lds + slot * SLOT + u * L::STEP + 1024 * wave;
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        if constexpr (GRP) lds_dma16_nt(rB, boff[j] - sub, k * 128, base + BM * 128 + 4096 * j);
        else lds_dma16(rB, boff[j] - sub, k * 128, base + BM * 128 + 4096 * j);
      }
#pragma unroll
      for (int i = 0; i < IB; ++i) lds_dma16(rA, aoff[i] - sub, k * 128, base + 4096 * i);
    }
  };
#pragma unroll
  for (int p = 0; p < STAGES - 1; ++p)
    if (p < rounds) load_round(p, p);

  const int r32 = lane & 31, h = lane >> 5;
  const int off = 128 * r32 + 16 * ((2 * wave + h) ^ swz_row(r32));
  v16i acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  v4i fa[U][IB], fb[U][JB];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < IB; ++i) fa[u][i] = v4i{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < JB; ++j) fb[u][j] = v4i{0, 0, 0, 0};
  }
  auto multiply = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[u][j], fa[u][i], acc[i][j], 0, 0, 0);
  };
  int slot = 0;
  for (int g = 0; g < rounds; ++g) {
    // Round g has landed; g+1 .. g+STAGES-2 may still be on their way.
    if (g + STAGES - 2 < rounds) __builtin_amdgcn_s_waitcnt(vmcnt_only((STAGES - 2) * LPS) & ~(15 << 8));
    else __builtin_amdgcn_s_waitcnt(vmcnt_only(0) & ~(15 << 8));
    __builtin_amdgcn_s_barrier();  // and every wave has read round g - 1: its slot is free
    v4i na[U][IB], nb[U][JB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* base = smem + slot * SLOT + u * L::STEP + off;
#pragma unroll
      for (int i = 0; i < IB; ++i) na[u][i] = *reinterpret_cast<const v4i*>(base + 4096 * i);
#pragma unroll
      for (int j = 0; j < JB; ++j) nb[u][j] = *reinterpret_cast<const v4i*>(base + BM * 128 + 4096 * j);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (g + STAGES - 1 < rounds) load_round(g + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
    multiply();
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < IB; ++i) fa[u][i] = na[u][i];
#pragma unroll
      for (int j = 0; j < JB; ++j) fb[u][j] = nb[u][j];
    }
    slot = slot + 1 == STAGES ? 0 : slot + 1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool in = ((rounds - 1) * U + u) * 128 + 16 * (2 * wave + h) < a.K;
#pragma unroll
    for (int i = 0; i < IB; ++i) fa[u][i] = in ? fa[u][i] : v4i{0, 0, 0, 0};
  }
  multiply();
  lds_barrier();  // the ring is free: the waves' sums take its place, rows of BN words
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4i*>(smem + (wave * BM + 32 * i + r32) * L::PITCH + 4 * (32 * j + 8 * q + 4 * h)) =
            v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  lds_barrier();
  // Four columns per thread, neighbouring threads on neighbouring columns.
  const float* b_s = a.b_s + (int64_t)e * a.N;
#pragma unroll
  for (int t = 0; t < BM * BN / 1024; ++t) {
    const int q = t * 256 + tid, mr = q / (BN / 4), nc = 4 * (q % (BN / 4));
    const uint8_t* s0 = smem + mr * L::PITCH + 4 * nc;
    v4i s = *reinterpret_cast<const v4i*>(s0);
#pragma unroll
    for (int w = 1; w < 4; ++w) s += *reinterpret_cast<const v4i*>(s0 + w * BM * L::PITCH);
    const int m = m0 + mr, n = n0 + nc, cnt = a.N - n < 4 ? a.N - n : 4;
    if (m < m_end && cnt > 0) {
      const v4f c = scale4(s, a.a_s[m], b_s, a.bias, n, a.N);
      const int64_t at = (int64_t)m * a.ldc + n;
      switch (a.out) {
        case kOutBF16: store_run<kOutBF16>(a.C, at, c, cnt); break;
        case kOutFP16: store_run<kOutFP16>(a.C, at, c, cnt); break;
        default: store_run<kOutFP32>(a.C, at, c, cnt); break;
      }
    }
  }
}

// Scales a wave's IB x JB blocks of 32 x 32 sums and stores them.  Block
// (i, j), element 4q + r of lane l: row m = 32i + (l & 31), column
// n = 32j + 8q + 4(l >> 5) + r.  32 rows of up to 128 bytes at a time go
// through the wave's own padded slab of LDS, and from there out as whole row
// segments, 16 bytes per lane (C is written once and not read back:
// non-temporal) at any alignment of C's rows; only a row's last segment goes
// value by value (4096 x 4097 x 1024: 34.3 us, with all of it so 46; 16384 x
// 513 x 256 12.8 and 19.4).  The sums themselves pass no branch: with the
// edge's tests around each of them the epilogue was 3600 basic blocks.
//
// as_t, bs_t, bi_t: the wave's row scales, column scales and bias in LDS
// (loaded before the K loop: read from memory here, their latency would add
// to every tile's end; 16384 x 4096 x 4096 278 -> 248 us).
template <int OUT, int JB>
struct Slab {
  static constexpr int ES = (int)sizeof(typename Out<OUT>::T);
  static constexpr int JG = JB * 32 * ES <= 128 ? JB : 128 / (32 * ES);  // blocks side by side
  static constexpr int ROWB = 32 * JG * ES, ROWP = ROWB + 16, BYTES = 32 * ROWP;
  static constexpr int PER_ROW = ROWB / 16, STORES = 32 * PER_ROW / 64;
};

// Large tiles keep their sums in accumulator registers, and the compiler
// would copy all of them to vector registers before the first is used (256 of
// them: spills).  ACC_REGS: they are held there, past the last MFMA's wait
// states, and read one at a time.
template <int IB, int JB>
constexpr bool kAccRegs = IB * JB >= 8;

template <int IB, int JB>
__device__ __forceinline__ void hold_sums(v16i (&acc)[IB][JB]) {
  if constexpr (kAccRegs<IB, JB>) {
    static_assert(JB == 4, "four operands");
#pragma unroll
    for (int i = 0; i < IB; ++i)
      asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]));
  }
}

template <bool ACC_REGS>
__device__ __forceinline__ float sum_of(int v) {
  if constexpr (ACC_REGS) {
    int s;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(s) : "a"(v));
    return (float)s;
  } else {
    return (float)v;
  }
}

template <int OUT, bool BIAS, int IB, int JB>
__device__ __forceinline__ void store_tile(const I8Args& a, const v16i (&acc)[IB][JB], uint8_t* slab,
                                           const float* as_t, const float* bs_t, const float* bi_t, int lane, int m0,
                                           int m_end, int n0) {
  typedef Slab<OUT, JB> S;
  typedef typename Out<OUT>::T T;
  const int h = lane >> 5;
  const bool whole = n0 + 32 * JB <= a.N;
  typedef int v4u __attribute__((ext_vector_type(4), aligned(2)));  // at any value
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const float as = as_t[32 * i + (lane & 31)];
#pragma unroll
    for (int j0 = 0; j0 < JB; j0 += S::JG) {
      // The column scales and the bias are read again for every row block:
      // kept in registers they cost up to 128 of them, which spill, and a
      // reload from scratch waits for every store before it.
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = j0; j < j0 + S::JG; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = 32 * j + 8 * q + 4 * h;
          const v4f bs = *reinterpret_cast<const v4f*>(bs_t + col);
          v4f c;
#pragma unroll
          for (int r = 0; r < 4; ++r) c[r] = rounded((as * bs[r]) * sum_of<kAccRegs<IB, JB>>(acc[i][j][4 * q + r]));
          if constexpr (BIAS) {
            const v4f bi = *reinterpret_cast<const v4f*>(bi_t + col);
#pragma unroll
            for (int r = 0; r < 4; ++r) c[r] = c[r] + bi[r];
          }
          store4<OUT>(slab + (lane & 31) * S::ROWP, col - 32 * j0, c, 4, true);
        }
      uint8_t* base = reinterpret_cast<uint8_t*>(a.C) + ((int64_t)(m0 + 32 * i) * a.ldc + n0 + 32 * j0) * S::ES;
      if (whole) {
#pragma unroll
        for (int t = 0; t < S::STORES; ++t) {
          const int q = t * 64 + lane, row = q / S::PER_ROW, cb = (q % S::PER_ROW) * 16;
          if (m0 + 32 * i + row < m_end)
            __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(slab + row * S::ROWP + cb),
                                        reinterpret_cast<v4u*>(base + (int64_t)row * a.ldc * S::ES + cb));
        }
      } else {
        const int bytes = (a.N - (n0 + 32 * j0)) * S::ES;
#pragma unroll 1
        for (int q = lane; q < 32 * S::PER_ROW; q += 64) {
          const int row = q / S::PER_ROW, cb = (q % S::PER_ROW) * 16;
          if (m0 + 32 * i + row >= m_end) break;
          const uint8_t* from = slab + row * S::ROWP + cb;
          uint8_t* to = base + (int64_t)row * a.ldc * S::ES + cb;
          if (cb + 16 <= bytes) {
            __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(from), reinterpret_cast<v4u*>(to));
          } else {
#pragma unroll 1
            for (int c = 0; c < bytes - cb; c += S::ES) *reinterpret_cast<T*>(to + c) = *reinterpret_cast<const T*>(from + c);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The tile kernel: BM x BN outputs per workgroup, WAVES_M x WAVES_N waves, a
// STAGES-deep ring of 128-byte K steps in LDS filled by direct-to-LDS loads
// (16 bytes per lane, so rows start on 16-byte boundaries and K is a multiple
// of 16).
//
// The accumulators stay in the MFMA's own registers for all of K, so a wave
// can hold 128 x 128 outputs (256 accumulator registers, one wave per SIMD),
// which halves the LDS reads per product against the 128 x 64 of the FP8
// kernel: 128 KB of fragments and 64 KB of fills per 2048 MFMA cycles, three
// quarters of what LDS delivers.
//
// A step is 4 slices of 32 K bytes: slice s of a row block is chunk 2s + h of
// its 32 rows (h = lane >> 5), one 16-byte read per lane.  The fragments of
// slice s + 1 are read while slice s is multiplied; at the start of the last
// slice the wave has read all of the step, so that is where it waits for the
// next step's loads, meets the others, refills the slot with the step STAGES
// ahead and reads the next step's first fragments.
// ---------------------------------------------------------------------------
template <int BM, int BN, int STAGES>
struct TileLds {
  static constexpr int SLOT = (BM + BN) * 128;
  static constexpr int AI = (BM + 63) / 64, BI = BN / 64;   // 64-value images of the row and the column scales
  static constexpr int BYTES = STAGES * SLOT + (AI + 2 * BI) * 256;
  static constexpr int PER_CU = 160 * 1024 / BYTES;
};

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, int GRP>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, (TileLds<BM, BN, STAGES>::PER_CU > 1 ? 2 : 1)) void k_i8_tile(I8Args a) {
  constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, IB = WM / 32, JB = WN / 32;
  constexpr int BK = 128, CH = BK / 16, RI = 64 / CH, SL = BK / 32;  // bytes of K and chunks per row, rows per load image, slices
  constexpr int AP = BM * CH / NT, BP = BN * CH / NT, LPS = AP + BP;  // loads per thread per step
  constexpr int A_BYTES = BM * BK, SLOT = (BM + BN) * BK;
  static_assert(BM * CH % NT == 0 && BN * CH % NT == 0, "whole load images per wave");
  static_assert((NW * RI) % 16 == 0, "a lane's chunk is the same in all its images");
  static_assert((STAGES - 1) * LPS < 64, "vmcnt counts at most 63 outstanding loads");
  typedef TileLds<BM, BN, STAGES> L;
  __shared__ __attribute__((aligned(16))) uint8_t smem[L::BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int tiles_n = (a.N + BN - 1) / BN;
  int m0, n0, m_end = a.M, e = 0;
  {
    const int lid = logical_tile(a);
    if constexpr (GRP) {
      if (!expert_of_slot<BM>(a.offsets, a.E, a.M, lid / tiles_n, e, m0, m_end, reinterpret_cast<int*>(smem))) return;
      n0 = (lid % tiles_n) * BN;
    } else {
      int tm, tn;
      raster(lid, (a.M + BM - 1) / BM, tiles_n, 8, tm, tn);
      m0 = tm * BM;
      n0 = tn * BN;
    }
  }
  // Uniform over the workgroup: in scalar registers, as the buffer resources
  // have to be.
  m0 = __builtin_amdgcn_readfirstlane(m0);
  n0 = __builtin_amdgcn_readfirstlane(n0);
  m_end = __builtin_amdgcn_readfirstlane(m_end);
  e = __builtin_amdgcn_readfirstlane(e);
  // The resources end with the last row that the tile may use: lanes of rows
  // past it read zeros and touch no memory (their outputs are never stored).
  auto upto = [](int64_t rows, int64_t ld, int64_t len) {
    const int64_t b = (rows - 1) * ld + len;
    return (uint32_t)(b < UINT32_MAX ? b : UINT32_MAX);
  };
  const buf_rsrc rA = make_rsrc_n(a.A + (int64_t)m0 * a.lda, upto(m_end - m0, a.lda, a.K));
  const buf_rsrc rB = make_rsrc_n(a.B + ((int64_t)e * a.N + n0) * a.ldb, upto(a.N - n0, a.ldb, a.K));
  const int nk = (a.K + BK - 1) / BK;

  // Load image q (q = i*NW + wave) fills RI LDS rows of a tile; lane l writes
  // row q*RI + l / CH, slot l % CH, so it reads the row's chunk
  // (l % CH) ^ swz(row).
  uint32_t aoff[AP], boff[BP];
  const int chunk = (lane % CH) ^ swz_row(RI * wave + lane / CH);
#pragma unroll
  for (int i = 0; i < AP; ++i) {
    const int r = RI * (i * NW + wave) + lane / CH;
    aoff[i] = (uint32_t)r * (uint32_t)a.lda + 16u * (uint32_t)chunk;
  }
#pragma unroll
  for (int i = 0; i < BP; ++i) {
    const int r = RI * (i * NW + wave) + lane / CH;
    boff[i] = (uint32_t)r * (uint32_t)a.ldb + 16u * (uint32_t)chunk;
  }
  // In the last step, lanes whose chunk lies past K read the step's first
  // chunk instead (K % 16 == 0: a chunk is wholly in or out); the fragments'
  // mask keeps it out of the sums.
  const uint32_t tail = (nk - 1) * BK + 16 * chunk >= a.K ? 16u * (uint32_t)chunk : 0u;
  lds_u8* const lds = (lds_u8*)smem;
  auto load_one = [&](int k, int slot, int i, uint32_t sub) {
    lds_u8* base = lds + slot * SLOT;
    if (i < AP) lds_dma16(rA, aoff[i < AP ? i : 0] - sub, k * BK, base + 1024 * (i * NW + wave));
    else lds_dma16(rB, boff[i < AP ? 0 : i - AP] - sub, k * BK, base + A_BYTES + 1024 * ((i - AP) * NW + wave));
  };
  // A step's refill is spread over two slices, the last one of the step that
  // frees the slot and the first one of the step after it, LPS0 loads behind
  // the MFMAs of the one and LPS - LPS0 behind those of the other.
  constexpr int NM = IB * JB;
  constexpr int LPS0 = (LPS + 1) / 2;
  // Slice s of row block b: this lane's 16 bytes.
  const int frow = lane & 31, fh = lane >> 5, fsw = swz_row(frow);
  auto frag = [&](int slot, int off, int row0, int s) {
    return *reinterpret_cast<const v4i*>(smem + slot * SLOT + off + BK * (row0 + frow) + 16 * ((2 * s + fh) ^ fsw));
  };

  v16i acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  // The scales go straight to LDS too, 64 values per load and as many loads in
  // every wave (the last ones repeat the last image; without a bias its images
  // hold column scales that no one reads).
  {
    constexpr int IMAGES = L::AI + 2 * L::BI;
    const float* b_s = a.b_s + (int64_t)e * a.N + n0;
    const buf_rsrc ra = make_rsrc_n(a.a_s + m0, upto(m_end - m0, 4, 4)), rb = make_rsrc_n(b_s, upto(a.N - n0, 4, 4));
    const buf_rsrc ri = make_rsrc_n(a.bias ? a.bias + n0 : b_s, upto(a.N - n0, 4, 4));
#pragma unroll
    for (int i = 0; i < (IMAGES + NW - 1) / NW; ++i) {
      const int q = i * NW + wave < IMAGES ? i * NW + wave : IMAGES - 1;
      const int first = q < L::AI ? 0 : q < L::AI + L::BI ? L::AI : L::AI + L::BI;
      lds_dma4(q < L::AI ? ra : q < L::AI + L::BI ? rb : ri, 256u * (uint32_t)(q - first) + 4u * (uint32_t)lane, 0,
               lds + STAGES * SLOT + 256 * q);
    }
  }
#pragma unroll
  for (int p = 0; p < STAGES; ++p)
    if (p < nk) {
      const uint32_t sub = p == nk - 1 ? tail : 0u;
#pragma unroll
      for (int i = 0; i < (p < STAGES - 1 ? LPS : LPS0); ++i) load_one(p, p, i, sub);
    }
  if (nk >= STAGES) __builtin_amdgcn_s_waitcnt(vmcnt_only((STAGES - 2) * LPS + LPS0));
  else __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  __builtin_amdgcn_s_barrier();
  v4i fa[2][IB], fb[2][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i) fa[0][i] = frag(0, 0, wm * WM + 32 * i, 0);
#pragma unroll
  for (int j = 0; j < JB; ++j) fb[0][j] = frag(0, A_BYTES, wn * WN + 32 * j, 0);

  // One step.  kPrev: the rest of the refill that the step before began;
  // kRefill: the first part of this slot's, with the step STAGES ahead; kNext:
  // another step follows (the last one masks its tail instead).  The order of
  // MFMAs, fragment reads and loads is pinned, a read or load behind an MFMA,
  // so that none of them holds up the MFMA after it for long.
  auto step = [&](int k, int slot, auto prev, auto refill, auto more) {
    constexpr bool kPrev = decltype(prev)::value, kRefill = decltype(refill)::value, kNext = decltype(more)::value;
    const int next = slot + 1 == STAGES ? 0 : slot + 1, before = slot == 0 ? STAGES - 1 : slot - 1;
    uint32_t sub = 0, sub_prev = 0;
    if constexpr (kRefill) sub = k + STAGES == nk - 1 ? tail : 0u;
    if constexpr (kPrev) sub_prev = k - 1 + STAGES == nk - 1 ? tail : 0u;
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const int cur = s & 1, nxt = cur ^ 1;
      if (s == SL - 1 && kNext) {
        // Every LDS read of this step has been issued: past the barrier the
        // slot is free and the next step's tile is visible.
        __builtin_amdgcn_s_waitcnt(vmcnt_only(kPrev ? (STAGES - 2) * LPS : 0) & ~(15 << 8));
        __builtin_amdgcn_s_barrier();
      }
      if constexpr (!kNext) {
        if (a.K % BK != 0) {
          const bool in = k * BK + 16 * (2 * s + fh) < a.K;
#pragma unroll
          for (int i = 0; i < IB; ++i) fa[cur][i] = in ? fa[cur][i] : v4i{0, 0, 0, 0};
        }
      }
      const int rs = s == SL - 1 ? next : slot, ss = (s + 1) % SL;
      const bool reads = s < SL - 1 || kNext;
#pragma unroll
      for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          const int t = i * JB + j;
          __builtin_amdgcn_sched_barrier(0);
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if (reads) {  // A 0, B 0 .., A 1 ..: the order the next slice needs them in
            constexpr int R = (IB + JB + NM - 1) / NM;
#pragma unroll
            for (int q = t * R; q < t * R + R && q < IB + JB; ++q) {
              if (q == 0) fa[nxt][0] = frag(rs, 0, wm * WM, ss);
              else if (q <= JB) fb[nxt][q - 1 < JB ? q - 1 : 0] = frag(rs, A_BYTES, wn * WN + 32 * (q - 1), ss);
              else fa[nxt][q - JB < IB ? q - JB : 0] = frag(rs, 0, wm * WM + 32 * (q - JB), ss);
            }
          }
#pragma unroll
          for (int q = 0; q < LPS; ++q) {
            const int at = q < LPS0 ? q * NM / LPS0 : (q - LPS0) * NM / (LPS - LPS0);
            if (kRefill && s == SL - 1 && q < LPS0 && at == t) load_one(k + STAGES, slot, q, sub);
            if (kPrev && s == 0 && q >= LPS0 && at == t) load_one(k - 1 + STAGES, before, q, sub_prev);
          }
        }
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  int slot = 0, k = 0;
  auto advance = [&] {
    ++k;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
  };
  while (k + STAGES < nk) {
    step(k, slot, yes, yes, yes);
    advance();
  }
  if (k + STAGES == nk) {
    step(k, slot, yes, no, yes);
    advance();
  }
  if constexpr (STAGES > 2) {
    while (k + 1 < nk) {
      step(k, slot, no, no, yes);
      advance();
    }
  }
  step(k, slot, no, no, no);
  lds_barrier();  // the ring is free: the slabs take its place
  hold_sums(acc);
  const float* as_w = reinterpret_cast<const float*>(smem + STAGES * SLOT) + wm * WM;
  const float* bs_w = reinterpret_cast<const float*>(smem + STAGES * SLOT) + 64 * L::AI + wn * WN;
  const float* bi_w = bs_w + BN;
  auto store = [&](auto out, auto bias) {
    typedef Slab<decltype(out)::value, JB> S;
    static_assert(NW * S::BYTES <= STAGES * SLOT, "room for the slabs");
    store_tile<decltype(out)::value, decltype(bias)::value, IB, JB>(a, acc, smem + wave * S::BYTES, as_w, bs_w, bi_w, lane,
                                                                    m0 + wm * WM, m_end, n0 + wn * WN);
  };
  auto store_as = [&](auto out) {
    if (a.bias) store(out, yes);
    else store(out, no);
  };
  if (a.out == kOutBF16) store_as(std::integral_constant<int, kOutBF16>{});
  else if (a.out == kOutFP16) store_as(std::integral_constant<int, kOutFP16>{});
  else store_as(std::integral_constant<int, kOutFP32>{});
}

// Whether every row of A and B starts on a 16-byte boundary and holds whole
// 16-byte chunks, as the direct-to-LDS loads want it.
inline bool fast_rows(const I8Args& a) {
  return ((uintptr_t)a.A | (uintptr_t)a.B | (uintptr_t)a.lda | (uintptr_t)a.ldb | (uintptr_t)a.K) % 16 == 0;
}

// K < 16: rows shorter than a chunk, one output at a time.  K == 0 is the
// empty sum: the column's bias, or zero, in every row (also of no expert).
template <int OUT>
__device__ __forceinline__ void short_output(const I8Args& a, int64_t m, int64_t n) {
  if (a.K == 0) {
    store1<OUT>(a.C, m * a.ldc + n, a.bias ? a.bias[n] : 0.0f);
    return;
  }
  int lo = 0, hi = a.offsets ? a.E : 1;  // the experts whose offset is at most m end before `hi`
  if (a.offsets) {
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (a.offsets[mid] <= m) lo = mid;
      else hi = mid;
    }
    if (m < a.offsets[lo] || m >= a.offsets[lo + 1]) return;
  }
  const int8_t* x = reinterpret_cast<const int8_t*>(a.A) + m * a.lda;
  const int8_t* w = reinterpret_cast<const int8_t*>(a.B) + ((int64_t)lo * a.N + n) * a.ldb;
  int sum = 0;
  for (int k = 0; k < a.K; ++k) sum += (int)x[k] * (int)w[k];
  float c = rounded((a.a_s[m] * a.b_s[(int64_t)lo * a.N + n]) * (float)sum);
  if (a.bias) c = c + a.bias[n];
  store1<OUT>(a.C, m * a.ldc + n, c);
}

template <int OUT>
__global__ __launch_bounds__(256) void k_i8_short(I8Args a) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.M * a.N; i += (int64_t)gridDim.x * 256)
    short_output<OUT>(a, i / a.N, i % a.N);
}

template <int BM, int BN, int AHEAD, int GRP>
void start_any(const I8Args& a, dim3 g) {
  switch (a.out) {
    case kOutBF16: hipLaunchKernelGGL((k_i8_any<BM, BN, AHEAD, kOutBF16, GRP>), g, dim3(256), 0, a.stream, a); break;
    case kOutFP16: hipLaunchKernelGGL((k_i8_any<BM, BN, AHEAD, kOutFP16, GRP>), g, dim3(256), 0, a.stream, a); break;
    default: hipLaunchKernelGGL((k_i8_any<BM, BN, AHEAD, kOutFP32, GRP>), g, dim3(256), 0, a.stream, a); break;
  }
}

template <int BM, int BN, int AHEAD>
hipError_t launch_ANY(const I8Args& a, unsigned grid) {
  const dim3 g(grid);
  if (a.offsets) start_any<BM, BN, AHEAD, 1>(a, g);
  else start_any<BM, BN, AHEAD, 0>(a, g);
  return hipGetLastError();
}

template <int BM, int BN, int WM_, int WN_, int ST>
hipError_t launch_TILE(const I8Args& a, unsigned grid) {
  if (!fast_rows(a)) return hipErrorInvalidValue;
  const dim3 g(grid), b(64 * WM_ * WN_);
  if (a.offsets) hipLaunchKernelGGL((k_i8_tile<BM, BN, WM_, WN_, ST, 1>), g, b, 0, a.stream, a);
  else hipLaunchKernelGGL((k_i8_tile<BM, BN, WM_, WN_, ST, 0>), g, b, 0, a.stream, a);
  return hipGetLastError();
}

template <int BM, int BN, int U, int STAGES>
hipError_t launch_SLIM(const I8Args& a, unsigned grid) {
  if (!fast_rows(a)) return hipErrorInvalidValue;
  if (a.offsets) hipLaunchKernelGGL((k_i8_slim<BM, BN, U, STAGES, 1>), dim3(grid), dim3(256), 0, a.stream, a);
  else hipLaunchKernelGGL((k_i8_slim<BM, BN, U, STAGES, 0>), dim3(grid), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

template <int ROWS, int COLS, int KW, int U, bool FORM>
hipError_t launch_SKINNY(const I8Args& a, unsigned grid) {
  constexpr int NB = COLS / 16;
  const dim3 g(grid), b(64 * KW);
  if constexpr (FORM) {
    if (fast_rows(a)) {
      if (a.offsets) hipLaunchKernelGGL((k_i8_skinny<NB, ROWS, KW, U, true, 1>), g, b, 0, a.stream, a);
      else hipLaunchKernelGGL((k_i8_skinny<NB, ROWS, KW, U, true, 0>), g, b, 0, a.stream, a);
      return hipGetLastError();
    }
    if (a.offsets) return hipErrorInvalidValue;  // experts of such rows take the 32-column form
    hipLaunchKernelGGL((k_i8_skinny<NB, ROWS, KW, U, false, 0>), g, b, 0, a.stream, a);
  } else {
    if (a.offsets) hipLaunchKernelGGL((k_i8_skinny<NB, ROWS, KW, U, false, 1>), g, b, 0, a.stream, a);
    else hipLaunchKernelGGL((k_i8_skinny<NB, ROWS, KW, U, false, 0>), g, b, 0, a.stream, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8(const I8Args& a, int cus, int force_cfg, bool log) {
  const int64_t E = a.offsets ? a.E : 0;
  auto report = [&](int cfg, int64_t grid) {
    if (log)
      fprintf(stderr, "fp8bg int8: E=%lld M=%d N=%d K=%d out=%d -> cfg=%d grid=%lld\n", (long long)E, a.M, a.N, a.K, a.out,
              cfg, (long long)grid);
  };
  if (a.K < 16) {
    if (a.K > 0 && force_cfg >= 0) return hipErrorInvalidValue;
    report(-1, 0);
    const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
    const dim3 g((unsigned)(blocks < 65536 ? blocks : 65536)), b(256);
    switch (a.out) {
      case kOutBF16: hipLaunchKernelGGL(k_i8_short<kOutBF16>, g, b, 0, a.stream, a); break;
      case kOutFP16: hipLaunchKernelGGL(k_i8_short<kOutFP16>, g, b, 0, a.stream, a); break;
      default: hipLaunchKernelGGL(k_i8_short<kOutFP32>, g, b, 0, a.stream, a); break;
    }
    return hipGetLastError();
  }
  const int cfg = force_cfg >= 0 ? force_cfg : int8_cfg_for(E, a.M, a.N, a.K, fast_rows(a), cus);
  if (cfg >= kNumI8Cfgs) return hipErrorInvalidValue;
  const int64_t grid = int8_grid(cfg, E, a.M, a.N);
  if (grid > kMaxI8Grid) return hipErrorInvalidValue;
  report(cfg, grid);
  // A launch holds less than 2^32 threads, and a workgroup up to 512.
  constexpr int64_t kPerLaunch = ((int64_t)1 << 23) - kXcds;
  for (int64_t first = 0; first < grid; first += kPerLaunch) {
    I8Args part = a;
    part.first = (int)first;
    const unsigned n = (unsigned)(grid - first < kPerLaunch ? grid - first : kPerLaunch);
    hipError_t e = hipErrorInvalidValue;
    switch (cfg) {
#define X(id, kind, ...) \
  case id: e = launch_##kind<__VA_ARGS__>(part, n); break;
      FBG_I8_CFGS(X)
#undef X
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fbg
