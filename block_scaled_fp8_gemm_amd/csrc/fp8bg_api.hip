// C-ABI entry points: argument validation, the dispatcher's plan, split-K
// workspace handling and kernel launch.  See include/fp8bg.h for the
// contract of each function.
#include <atomic>
#include <mutex>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "fp8bg.h"
#include "fp8bg_int8_configs.h"
#include "fp8bg_internal.h"
#include "fp8bg_tokens.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_cu_count[kMaxDevices];  // 0 = not yet queried

int device_cu_count(int* status) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    *status = FBG_ERROR_HIP;
    return 0;
  }
  if (dev < kMaxDevices) {
    const int cached = g_cu_count[dev].load(std::memory_order_relaxed);
    if (cached > 0) return cached;
  }
  int cu = 0;
  if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cu <= 0) {
    *status = FBG_ERROR_HIP;
    return 0;
  }
  if (dev < kMaxDevices) g_cu_count[dev].store(cu, std::memory_order_relaxed);
  return cu;
}

bool env_flag(const char* name) {
  const char* v = getenv(name);
  return v && v[0] && strcmp(v, "0") != 0;
}

int elem_size(int out_dtype) { return out_dtype == FBG_OUT_FP32 ? 4 : 2; }

// Largest K: the kernels address a tile's rows (up to 256 of K bytes each)
// through a buffer resource based at the tile's first row, whose 32-bit
// record count reaches 2^32 - 1 bytes: 256 rows of K bytes must end before
// that, so K <= 2^24 - 128 (at K = 2^24 the last dword of a 256-row tile
// read as zero).
constexpr int64_t kMaxK = ((int64_t)1 << 24) - 128;

bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// FBG_FORCE_CONFIG=<index>: tests and benchmarks pin the tile configuration
// of the chosen variant (read on every call so a test can change it).
int forced_config() {
  const char* v = getenv("FBG_FORCE_CONFIG");
  return (v && v[0]) ? atoi(v) : -1;
}

// Pure host checks, made before any HIP call.
int validate(const void* A, const float* a_s, const void* B, const float* b_s, const void* C, int64_t M,
             int64_t N, int64_t K, int out_dtype) {
  if (M < 0 || N < 0 || K < 0) return FBG_ERROR_INVALID_VALUE;
  if (out_dtype != FBG_OUT_BF16 && out_dtype != FBG_OUT_FP16 && out_dtype != FBG_OUT_FP32)
    return FBG_ERROR_INVALID_VALUE;
  if (K % 128 != 0) return FBG_ERROR_UNSUPPORTED;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return FBG_ERROR_UNSUPPORTED;
  // The kernels address a tile's rows (up to 256 of them) with 32-bit offsets.
  if (K > kMaxK) return FBG_ERROR_UNSUPPORTED;
  const int64_t G = K / 128, NB = (N + 127) / 128;
  const int64_t bytesA = M * K, bytesB = N * K, bytesAs = M * G * 4, bytesBs = NB * G * 4;
  const int64_t bytesC = M * N * elem_size(out_dtype);
  // The generic kernel addresses the scale arrays with 32-bit buffer offsets.
  if (bytesAs > (int64_t)UINT32_MAX || bytesBs > (int64_t)UINT32_MAX) return FBG_ERROR_UNSUPPORTED;
  if ((bytesA > 0 && !A) || (bytesB > 0 && !B) || (bytesAs > 0 && !a_s) || (bytesBs > 0 && !b_s) ||
      (bytesC > 0 && !C))
    return FBG_ERROR_INVALID_VALUE;
  if (overlaps(C, bytesC, A, bytesA) || overlaps(C, bytesC, B, bytesB) || overlaps(C, bytesC, a_s, bytesAs) ||
      overlaps(C, bytesC, b_s, bytesBs))
    return FBG_ERROR_INVALID_VALUE;
  if ((bytesA > 0 && !aligned(A, 16)) || (bytesB > 0 && !aligned(B, 16)) || (bytesAs > 0 && !aligned(a_s, 4)) ||
      (bytesBs > 0 && !aligned(b_s, 4)) || (bytesC > 0 && !aligned(C, (uintptr_t)elem_size(out_dtype))))
    return FBG_ERROR_UNSUPPORTED;
  return FBG_SUCCESS;
}

// FBG_RASTER_BAND=<rows>: benchmarks try other raster band heights for the
// generic kernel (default 8 tile-rows).
int raster_band() {
  const char* v = getenv("FBG_RASTER_BAND");
  const int b = (v && v[0]) ? atoi(v) : 0;
  return b > 0 ? b : 8;
}

// Launches the plan's kernel.  partial / counters: the split-K workspace's
// FP32 partials and arrival counters (unused unless the plan splits K).
int launch_plan(const fbg_plan& p, const fbg::GemmArgs& args, float* partial, unsigned* counters) {
  hipError_t e = hipSuccess;
  switch (p.variant) {
    case FBG_VARIANT_GENERIC:
      e = fbg::launch_generic(args, p.config, p.grid, raster_band());
      break;
    case FBG_VARIANT_SHORT_K256:
      e = fbg::launch_short_k256(args, p.config, p.grid);
      break;
    case FBG_VARIANT_SWAP_AB:
    case FBG_VARIANT_SWAP_AB_SPLITK:
      if (p.split_k <= 1) partial = nullptr, counters = nullptr;
      e = fbg::launch_swap(args, p.config, p.grid, p.split_k, partial, counters);
      break;
    default:
      return FBG_ERROR_INVALID_VALUE;
  }
  return e == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

// A workspace laid out as fp8_block_gemm_workspace_size describes: the
// partials first, the counters at workspace_counter_offset.
int launch_with_workspace(const fbg_plan& p, const fbg::GemmArgs& args, void* ws, int64_t M, int64_t N) {
  return launch_plan(p, args, static_cast<float*>(ws),
                     reinterpret_cast<unsigned*>(static_cast<char*>(ws) + fbg::workspace_counter_offset(p, M, N)));
}

// ---------------------------------------------------------------------------
// The no-allocation entry point's scratch: split-K arrival counters in the
// first kScratchCounterBytes, FP32 partials after them.  Every GPU the library
// runs on holds its own copy for the life of the process.  In host code the
// array's name is not a device address: the kernels get the per-device address
// that hipGetSymbolAddress returns (scratch_address).  The counters are zero
// when the code object is loaded, are cleared once more by the first call on
// each device, and every completed call leaves them zero.
// ---------------------------------------------------------------------------
constexpr int64_t kScratchBytes = (int64_t)4 << 20;
constexpr int64_t kScratchCounterBytes = (int64_t)16 << 10;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

std::mutex g_scratch_mu;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

// This device's scratch address (set up on the device's first call: the
// symbol's address, then a kernel on `stream` clearing the counters), or
// nullptr with *status set.
void* scratch_address(hipStream_t stream, int* status) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    *status = FBG_ERROR_HIP;
    return nullptr;
  }
  void* ptr = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (ptr) return ptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  ptr = g_scratch_ptr[dev].load(std::memory_order_relaxed);
  if (ptr) return ptr;
  if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) {
    (void)hipGetLastError();
    *status = FBG_ERROR_HIP;
    return nullptr;
  }
  if (fbg::launch_zero_words(ptr, kScratchCounterBytes / 4, stream) != hipSuccess) {
    *status = FBG_ERROR_HIP;
    return nullptr;
  }
  g_scratch_ptr[dev].store(ptr, std::memory_order_release);
  return ptr;
}

enum WorkspaceMode { kCallerOrLibrary, kStaticScratch };

int gemm_call(const void* A, const float* a_s, const void* B, const float* b_s, void* C, int64_t M, int64_t N,
              int64_t K, int out_dtype, void* stream_, int variant, int split_k, void* workspace,
              size_t workspace_size, WorkspaceMode mode) {
  int st = validate(A, a_s, B, b_s, C, M, N, K, out_dtype);
  if (st != FBG_SUCCESS) return st;
  if (variant < FBG_VARIANT_AUTO || variant > FBG_VARIANT_SWAP_AB_SPLITK || split_k < 0)
    return FBG_ERROR_INVALID_VALUE;
  hipStream_t stream = static_cast<hipStream_t>(stream_);
  // No caller workspace and the dispatcher's choice: plan without a K split,
  // so the call never allocates (a stream-ordered allocation and free cost
  // more than splitting saves).  A split forced without a workspace still
  // gets a stream-ordered one below.  The static scratch keeps the split.
  if (mode == kCallerOrLibrary && !workspace && variant == FBG_VARIANT_AUTO && split_k == 0) split_k = 1;
  if (M == 0 || N == 0) return FBG_SUCCESS;
  if (K == 0) {
    // Still honour a forced variant's guard before filling.
    fbg_plan p;
    st = fbg::make_plan(M, N, K, out_dtype, 256, variant, split_k, &p, -1);
    if (st != FBG_SUCCESS) return st;
    return fbg::launch_fill_zero(C, M * N, out_dtype, stream) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
  }
  const int cu = device_cu_count(&st);
  if (st != FBG_SUCCESS) return st;
  fbg_plan p;
  st = fbg::make_plan(M, N, K, out_dtype, cu, variant, split_k, &p, forced_config());
  if (st != FBG_SUCCESS) return st;

  fbg::GemmArgs args;
  args.A = static_cast<const uint8_t*>(A);
  args.a_s = a_s;
  args.B = static_cast<const uint8_t*>(B);
  args.b_s = b_s;
  args.C = C;
  args.M = (int)M;
  args.N = (int)N;
  args.K = (int)K;
  args.out = out_dtype;
  args.vec = (N % 4 == 0) && aligned(C, (uintptr_t)(4 * elem_size(out_dtype)));
  if (args.vec && (N * elem_size(out_dtype)) % 16 == 0 && aligned(C, 16)) args.vec |= 2;  // 16-byte rows
  args.stream = stream;

  if (env_flag("FBG_LOG"))
    fprintf(stderr, "fp8bg: M=%lld N=%lld K=%lld out=%d -> variant=%d cfg=%d tile=%dx%d S=%d grid=%lld ws=%lld\n",
            (long long)M, (long long)N, (long long)K, out_dtype, p.variant, p.config, p.tile_m, p.tile_n, p.split_k,
            (long long)p.grid, (long long)p.workspace_bytes);

  if (p.workspace_bytes == 0) return launch_plan(p, args, nullptr, nullptr);

  if (mode == kStaticScratch) {
    const int64_t tiles = p.grid / p.split_k;
    const int64_t partial = fbg::workspace_counter_offset(p, M, N);
    if (tiles * 4 > kScratchCounterBytes || partial > kScratchBytes - kScratchCounterBytes)
      return FBG_ERROR_SCRATCH_LIMIT;
    char* base = static_cast<char*>(scratch_address(stream, &st));
    if (!base) return st;
    return launch_plan(p, args, reinterpret_cast<float*>(base + kScratchCounterBytes),
                       reinterpret_cast<unsigned*>(base));
  }
  if (workspace) {
    if (workspace_size < (size_t)p.workspace_bytes) return FBG_ERROR_OUT_OF_MEMORY;
    if (!aligned(workspace, 16)) return FBG_ERROR_UNSUPPORTED;
    return launch_with_workspace(p, args, workspace, M, N);
  }
  // Library-owned workspace: stream-ordered, so concurrent streams never share one.
  if (env_flag("FBG_TEST_FAIL_ALLOC")) return FBG_ERROR_OUT_OF_MEMORY;
  void* ws = nullptr;
  if (hipMallocAsync(&ws, (size_t)p.workspace_bytes, stream) != hipSuccess || !ws) {
    (void)hipGetLastError();
    return FBG_ERROR_OUT_OF_MEMORY;
  }
  const int64_t coff = fbg::workspace_counter_offset(p, M, N);
  if (fbg::launch_zero_words(static_cast<char*>(ws) + coff, (p.workspace_bytes - coff) / 4, stream) != hipSuccess) {
    (void)hipFreeAsync(ws, stream);
    return FBG_ERROR_HIP;
  }
  st = launch_with_workspace(p, args, ws, M, N);
  if (hipFreeAsync(ws, stream) != hipSuccess && st == FBG_SUCCESS) st = FBG_ERROR_HIP;
  return st;
}

}  // namespace

extern "C" int fp8_block_gemm_ex(const void* A, const float* a_s, const void* B, const float* b_s, void* C, int64_t M,
                                 int64_t N, int64_t K, int out_dtype, void* stream, int variant, int split_k,
                                 void* workspace, size_t workspace_size) {
  return gemm_call(A, a_s, B, b_s, C, M, N, K, out_dtype, stream, variant, split_k, workspace, workspace_size,
                   kCallerOrLibrary);
}

extern "C" int fp8_block_gemm(const void* A, const float* a_s, const void* B, const float* b_s, void* C, int64_t M,
                              int64_t N, int64_t K, int out_dtype, void* stream) {
  return fp8_block_gemm_ex(A, a_s, B, b_s, C, M, N, K, out_dtype, stream, FBG_VARIANT_AUTO, 0, nullptr, 0);
}

extern "C" int fp8_block_gemm_noalloc(const void* A, const float* a_s, const void* B, const float* b_s, void* C,
                                      int64_t M, int64_t N, int64_t K, int out_dtype, void* stream, int variant,
                                      int split_k) {
  return gemm_call(A, a_s, B, b_s, C, M, N, K, out_dtype, stream, variant, split_k, nullptr, 0, kStaticScratch);
}

extern "C" size_t fp8_block_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int variant, int split_k) {
  int cu = 256;
  if (variant == FBG_VARIANT_AUTO || split_k == 0) {
    int st = FBG_SUCCESS;
    cu = device_cu_count(&st);
    if (st != FBG_SUCCESS) return (size_t)-1;
  }
  fbg_plan p;
  if (fbg::make_plan(M, N, K, FBG_OUT_BF16, cu, variant, split_k, &p, forced_config()) != FBG_SUCCESS)
    return (size_t)-1;
  return (size_t)p.workspace_bytes;
}

extern "C" int fp8_block_gemm_quantize_rows(const void* x, int64_t M, int64_t K, void* A, float* a_s, void* stream_) {
  if (M < 0 || K < 0) return FBG_ERROR_INVALID_VALUE;
  if (K % 128 != 0) return FBG_ERROR_UNSUPPORTED;
  if (M > INT32_MAX || K > INT32_MAX) return FBG_ERROR_UNSUPPORTED;
  const int64_t G = K / 128, bytesX = M * K * 2, bytesA = M * K, bytesAs = M * G * 4;
  if ((bytesX > 0 && !x) || (bytesA > 0 && !A) || (bytesAs > 0 && !a_s)) return FBG_ERROR_INVALID_VALUE;
  if (overlaps(A, bytesA, x, bytesX) || overlaps(a_s, bytesAs, x, bytesX) || overlaps(A, bytesA, a_s, bytesAs))
    return FBG_ERROR_INVALID_VALUE;
  if ((bytesX > 0 && !aligned(x, 16)) || (bytesA > 0 && !aligned(A, 8)) || (bytesAs > 0 && !aligned(a_s, 4)))
    return FBG_ERROR_UNSUPPORTED;
  if (M == 0 || K == 0) return FBG_SUCCESS;
  const hipError_t e = fbg::launch_quantize_rows(static_cast<const uint16_t*>(x), static_cast<uint8_t*>(A), a_s,
                                                 M * G, static_cast<hipStream_t>(stream_));
  return e == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

extern "C" int fp8_block_gemm_quantize_blocks(const void* w, int64_t N, int64_t K, void* B, float* b_s,
                                              void* stream_) {
  if (N < 0 || K < 0) return FBG_ERROR_INVALID_VALUE;
  if (K % 128 != 0) return FBG_ERROR_UNSUPPORTED;
  if (N > INT32_MAX || K > INT32_MAX) return FBG_ERROR_UNSUPPORTED;
  const int64_t G = K / 128, NB = (N + 127) / 128;
  const int64_t bytesW = N * K * 2, bytesB = N * K, bytesBs = NB * G * 4;
  if ((bytesW > 0 && !w) || (bytesB > 0 && !B) || (bytesBs > 0 && !b_s)) return FBG_ERROR_INVALID_VALUE;
  if (overlaps(B, bytesB, w, bytesW) || overlaps(b_s, bytesBs, w, bytesW) || overlaps(B, bytesB, b_s, bytesBs))
    return FBG_ERROR_INVALID_VALUE;
  if ((bytesW > 0 && !aligned(w, 16)) || (bytesB > 0 && !aligned(B, 8)) || (bytesBs > 0 && !aligned(b_s, 4)))
    return FBG_ERROR_UNSUPPORTED;
  if (N == 0 || K == 0) return FBG_SUCCESS;
  const hipError_t e = fbg::launch_quantize_blocks(static_cast<const uint16_t*>(w), static_cast<uint8_t*>(B), b_s,
                                                   (int)N, (int)K, static_cast<hipStream_t>(stream_));
  return e == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

extern "C" int fp8_block_gemm_grouped(const void* A, const float* a_s, const void* B, const float* b_s, void* C,
                                      const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t K,
                                      int out_dtype, void* stream_) {
  if (E < 0 || M < 0 || N < 0 || K < 0) return FBG_ERROR_INVALID_VALUE;
  if (out_dtype != FBG_OUT_BF16 && out_dtype != FBG_OUT_FP16 && out_dtype != FBG_OUT_FP32)
    return FBG_ERROR_INVALID_VALUE;
  if (K % 128 != 0) return FBG_ERROR_UNSUPPORTED;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || E > INT32_MAX - 1) return FBG_ERROR_UNSUPPORTED;
  if (K > kMaxK) return FBG_ERROR_UNSUPPORTED;  // 32-bit offsets inside a tile's rows
  const int64_t G = K / 128, NB = (N + 127) / 128;
  int64_t bytesB = 0, bytesBs = 0;
  if (__builtin_mul_overflow(E, N * K, &bytesB) || __builtin_mul_overflow(E, NB * G * 4, &bytesBs))
    return FBG_ERROR_UNSUPPORTED;  // B or b_s larger than any address space
  const int64_t bytesA = M * K, bytesAs = M * G * 4;
  const int64_t bytesC = M * N * elem_size(out_dtype), bytesOff = (E + 1) * 4;
  // The generic kernel addresses the scale arrays (one expert's b_s) with 32-bit buffer offsets.
  if (bytesAs > (int64_t)UINT32_MAX || NB * G * 4 > (int64_t)UINT32_MAX) return FBG_ERROR_UNSUPPORTED;
  if ((bytesA > 0 && !A) || (bytesAs > 0 && !a_s) || (bytesB > 0 && !B) || (bytesBs > 0 && !b_s) ||
      (bytesC > 0 && !C) || (E > 0 && !offsets))
    return FBG_ERROR_INVALID_VALUE;
  if (overlaps(C, bytesC, A, bytesA) || overlaps(C, bytesC, B, bytesB) || overlaps(C, bytesC, a_s, bytesAs) ||
      overlaps(C, bytesC, b_s, bytesBs) || overlaps(C, bytesC, offsets, bytesOff))
    return FBG_ERROR_INVALID_VALUE;
  if ((bytesA > 0 && !aligned(A, 16)) || (bytesB > 0 && !aligned(B, 16)) || (bytesAs > 0 && !aligned(a_s, 4)) ||
      (bytesBs > 0 && !aligned(b_s, 4)) || (bytesC > 0 && !aligned(C, (uintptr_t)elem_size(out_dtype))) ||
      (E > 0 && !aligned(offsets, 4)))
    return FBG_ERROR_UNSUPPORTED;
  hipStream_t stream = static_cast<hipStream_t>(stream_);
  if (M == 0 || N == 0) return FBG_SUCCESS;
  if (K == 0 || E == 0)  // the empty sum (no groups, or no expert to hold a row)
    return fbg::launch_fill_zero(C, M * N, out_dtype, stream) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
  const int cfg = fbg::grouped_cfg_for(M, E, N, K, forced_config());
  if (cfg < 0) return FBG_ERROR_UNSUPPORTED;
  const int64_t grid = fbg::grouped_grid(cfg, E, M, N);
  if (grid > INT32_MAX) return FBG_ERROR_UNSUPPORTED;

  fbg::GemmArgs args;
  args.A = static_cast<const uint8_t*>(A);
  args.a_s = a_s;
  args.B = static_cast<const uint8_t*>(B);
  args.b_s = b_s;
  args.C = C;
  args.M = (int)M;
  args.N = (int)N;
  args.K = (int)K;
  args.out = out_dtype;
  args.vec = (N % 4 == 0) && aligned(C, (uintptr_t)(4 * elem_size(out_dtype)));
  if (args.vec && (N * elem_size(out_dtype)) % 16 == 0 && aligned(C, 16)) args.vec |= 2;  // 16-byte rows
  args.stream = stream;
  if (env_flag("FBG_LOG"))
    fprintf(stderr, "fp8bg grouped: E=%lld M=%lld N=%lld K=%lld out=%d -> cfg=%d grid=%lld\n", (long long)E,
            (long long)M, (long long)N, (long long)K, out_dtype, cfg, (long long)grid);
  const hipError_t e = cfg < fbg::grouped_num_skinny_cfgs()
                           ? fbg::launch_grouped(args, cfg, grid, offsets, (int)E)
                           : fbg::launch_generic_grouped(args, cfg - fbg::grouped_num_skinny_cfgs(), grid, offsets,
                                                         (int)E);
  return e == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

// ---------------------------------------------------------------------------
// 8-bit integers, and the row operators that feed them.
// ---------------------------------------------------------------------------
namespace {

using fbg::kMaxExtent;
using fbg::kMaxInt8K;

// Bytes from the first element of `rows` rows of `cols` elements, `ld` apart,
// to the end of the last one; false if that overflows.
bool extent(int64_t rows, int64_t cols, int64_t ld, int64_t size, int64_t* bytes) {
  *bytes = 0;
  if (rows <= 0 || cols <= 0) return true;
  int64_t n = 0;
  return !__builtin_mul_overflow(rows - 1, ld, &n) && !__builtin_add_overflow(n, cols, &n) &&
         !__builtin_mul_overflow(n, size, bytes);
}

bool known_dtype(int d) { return d == FBG_OUT_BF16 || d == FBG_OUT_FP16 || d == FBG_OUT_FP32; }

int int8_call(const void* A, int64_t lda, const float* a_s, const void* B, int64_t ldb, const float* b_s,
              const float* bias, void* C, int64_t ldc, const int32_t* offsets, int64_t E, int64_t M, int64_t N,
              int64_t K, int out_dtype, bool grouped, void* stream) {
  if (E < 0 || M < 0 || N < 0 || K < 0 || !known_dtype(out_dtype)) return FBG_ERROR_INVALID_VALUE;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxInt8K || E > kMaxExtent) return FBG_ERROR_UNSUPPORTED;
  const bool many_b = N > 1 || (grouped && E > 1);
  if ((M > 1 && lda < K) || (many_b && ldb < K) || (M > 1 && ldc < N)) return FBG_ERROR_INVALID_VALUE;
  if (M <= 1) lda = K, ldc = N;  // the pitch of a single row says nothing
  if (!many_b) ldb = K;
  if (lda > kMaxK || ldb > kMaxK) return FBG_ERROR_UNSUPPORTED;  // 32-bit offsets inside a tile's rows
  const int64_t es = elem_size(out_dtype);
  int64_t rows_b = 0, bytesA = 0, bytesB = 0, bytesC = 0, bytesBs = 0;
  if (__builtin_mul_overflow(E, N, &rows_b) || !extent(M, K, lda, 1, &bytesA) || !extent(rows_b, K, ldb, 1, &bytesB) ||
      !extent(M, N, ldc, es, &bytesC) || __builtin_mul_overflow(rows_b, (int64_t)4, &bytesBs))
    return FBG_ERROR_UNSUPPORTED;
  const int64_t bytesAs = M * 4, bytesOff = grouped ? (E + 1) * 4 : 0;
  if (M == 0 || N == 0) return FBG_SUCCESS;
  if ((bytesA > 0 && !A) || (bytesB > 0 && !B) || !a_s || (bytesBs > 0 && !b_s) || !C || (grouped && E > 0 && !offsets))
    return FBG_ERROR_INVALID_VALUE;
  if (overlaps(C, bytesC, A, bytesA) || overlaps(C, bytesC, B, bytesB) || overlaps(C, bytesC, a_s, bytesAs) ||
      overlaps(C, bytesC, b_s, bytesBs) || overlaps(C, bytesC, bias, N * 4) || overlaps(C, bytesC, offsets, bytesOff))
    return FBG_ERROR_INVALID_VALUE;
  if (!aligned(a_s, 4) || !aligned(b_s, 4) || !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(C, (uintptr_t)es))
    return FBG_ERROR_UNSUPPORTED;

  fbg::I8Args args;
  args.A = static_cast<const uint8_t*>(A);
  args.a_s = a_s;
  args.B = static_cast<const uint8_t*>(B);
  args.b_s = b_s;
  args.bias = bias;
  args.C = C;
  args.offsets = grouped ? offsets : nullptr;
  args.lda = lda;
  args.ldb = ldb;
  args.ldc = ldc;
  args.M = (int)M;
  args.N = (int)N;
  args.K = grouped && E == 0 ? 0 : (int)K;
  args.E = (int)E;
  args.out = out_dtype;
  args.first = 0;
  args.stream = static_cast<hipStream_t>(stream);
  int st = FBG_SUCCESS;
  const int cus = device_cu_count(&st);
  if (st != FBG_SUCCESS) return st;
  const hipError_t err = fbg::launch_i8(args, cus, forced_config(), env_flag("FBG_LOG"));
  if (err == hipErrorInvalidValue) return FBG_ERROR_UNSUPPORTED;  // more tiles than 32 bits hold, or a forced configuration
  return err == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

}  // namespace

extern "C" int fbg_int8_gemm(const void* A, int64_t lda, const float* a_s, const void* B, int64_t ldb,
                             const float* b_s, const float* bias, void* C, int64_t ldc, int64_t M, int64_t N,
                             int64_t K, int out_dtype, void* stream) {
  return int8_call(A, lda, a_s, B, ldb, b_s, bias, C, ldc, nullptr, 1, M, N, K, out_dtype, false, stream);
}

extern "C" int fbg_int8_grouped_gemm(const void* A, int64_t lda, const float* a_s, const void* B, const float* b_s,
                                     void* C, int64_t ldc, const int32_t* offsets, int64_t E, int64_t M, int64_t N,
                                     int64_t K, int out_dtype, void* stream) {
  return int8_call(A, lda, a_s, B, K, b_s, nullptr, C, ldc, offsets, E, M, N, K, out_dtype, true, stream);
}

int fbg::int8_grouped_gemm(const void* A, int64_t lda, const float* a_s, const void* B, int64_t ldb, const float* b_s,
                           void* C, int64_t ldc, const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t K,
                           int out_dtype, void* stream) {
  return int8_call(A, lda, a_s, B, ldb, b_s, nullptr, C, ldc, offsets, E, M, N, K, out_dtype, true, stream);
}

extern "C" int fbg_quantize_tokens(const void* x, int64_t ldx, int in_dtype, int64_t M, int64_t K, void* q,
                                   int64_t ldq, float* scale, void* stream) {
  if (M < 0 || K < 0 || !known_dtype(in_dtype)) return FBG_ERROR_INVALID_VALUE;
  if (M > kMaxExtent || K > kMaxExtent) return FBG_ERROR_UNSUPPORTED;
  if (M > 1 && (ldx < K || ldq < K)) return FBG_ERROR_INVALID_VALUE;
  if (M <= 1) ldx = K, ldq = K;
  const int64_t es = elem_size(in_dtype);
  int64_t bytesX = 0, bytesQ = 0;
  if (!extent(M, K, ldx, es, &bytesX) || !extent(M, K, ldq, 1, &bytesQ)) return FBG_ERROR_UNSUPPORTED;
  if (M == 0) return FBG_SUCCESS;
  if ((bytesX > 0 && !x) || (bytesQ > 0 && !q) || !scale) return FBG_ERROR_INVALID_VALUE;
  if (overlaps(q, bytesQ, x, bytesX) || overlaps(scale, M * 4, x, bytesX) || overlaps(scale, M * 4, q, bytesQ))
    return FBG_ERROR_INVALID_VALUE;
  if (!aligned(x, (uintptr_t)es) || !aligned(scale, 4)) return FBG_ERROR_UNSUPPORTED;
  fbg::QuantArgs args;
  args.x = x;
  args.q = static_cast<int8_t*>(q);
  args.scale = scale;
  args.ldx = ldx;
  args.ldq = ldq;
  args.M = (int)M;
  args.K = (int)K;
  args.dtype = in_dtype;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_quantize_tokens(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

extern "C" int fbg_block_norm(const void* h, int64_t ldh, const void* x, int64_t ldx, const void* gate,
                              int64_t gate_row, int64_t gate_col, const void* post, const void* pre, int dtype,
                              int weight_dtype, int64_t M, int64_t D, float residual_scale, float eps,
                              float weight_offset, void* r, int64_t ldr, void* y, int64_t ldy, float* y_scale,
                              int quantize, void* stream) {
  if (M < 0 || D < 0 || gate_row < 0 || gate_col < 0 || !known_dtype(dtype) ||
      (weight_dtype != dtype && weight_dtype != FBG_OUT_FP32) || quantize < FBG_QUANT_NONE || quantize > FBG_QUANT_FP8)
    return FBG_ERROR_INVALID_VALUE;
  if (M > kMaxExtent || D > kMaxExtent) return FBG_ERROR_UNSUPPORTED;
  if (pre && quantize == FBG_QUANT_FP8 && D % 128 != 0) return FBG_ERROR_UNSUPPORTED;
  if (M > 1 && (ldh < D || (x && ldx < D) || ldr < D || (pre && ldy < D))) return FBG_ERROR_INVALID_VALUE;
  if (M <= 1) ldh = ldx = ldr = ldy = D;
  if (M == 0) return FBG_SUCCESS;
  if (D == 0)  // no pointer to an empty row says anything: y_scale alone asks for the scales
    return quantize == FBG_QUANT_INT8 && y_scale
               ? fbg_quantize_tokens(nullptr, 0, dtype, M, 0, nullptr, 0, y_scale, stream)
               : FBG_SUCCESS;
  const int64_t es = elem_size(dtype), ws = elem_size(weight_dtype), ys = quantize == FBG_QUANT_NONE ? es : 1;
  const int64_t bytesS = quantize == FBG_QUANT_NONE ? 0 : quantize == FBG_QUANT_INT8 ? M * 4 : M * (D / 128) * 4;
  int64_t bytesH = 0, bytesX = 0, bytesR = 0, bytesY = 0, bytesG = 0, g0 = 0, g1 = 0;
  if (!extent(M, D, ldh, es, &bytesH) || !extent(M, D, ldx, es, &bytesX) || !extent(M, D, ldr, es, &bytesR) ||
      !extent(M, D, ldy, ys, &bytesY) || __builtin_mul_overflow(M - 1, gate_row, &g0) ||
      __builtin_mul_overflow(D - 1, gate_col, &g1) || __builtin_add_overflow(g0, g1, &g0) ||
      __builtin_add_overflow(g0, (int64_t)1, &g0) || __builtin_mul_overflow(g0, es, &bytesG))
    return FBG_ERROR_UNSUPPORTED;
  if (!h || !r || (pre && !y) || (pre && bytesS > 0 && !y_scale)) return FBG_ERROR_INVALID_VALUE;
  if (!pre) y = nullptr, y_scale = nullptr;
  struct Range {
    const void* p;
    int64_t bytes;
  };
  const Range in[] = {{h, bytesH}, {x, bytesX}, {gate, bytesG}, {post, D * ws}, {pre, D * ws}};
  const Range out[] = {{r, bytesR}, {y, bytesY}, {y_scale, bytesS}};
  for (int i = 0; i < 3; ++i) {
    for (const Range& b : in)
      if (overlaps(out[i].p, out[i].bytes, b.p, b.bytes)) return FBG_ERROR_INVALID_VALUE;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return FBG_ERROR_INVALID_VALUE;
  }
  const uintptr_t ea = (uintptr_t)es;
  if (!aligned(h, ea) || !aligned(x, ea) || !aligned(gate, ea) || !aligned(r, ea) || !aligned(y, (uintptr_t)ys) ||
      !aligned(post, (uintptr_t)ws) || !aligned(pre, (uintptr_t)ws) || !aligned(y_scale, 4))
    return FBG_ERROR_UNSUPPORTED;
  fbg::NormArgs args;
  args.h = h;
  args.x = x;
  args.gate = gate;
  args.post = post;
  args.pre = pre;
  args.r = r;
  args.y = y;
  args.y_scale = y_scale;
  args.ldh = ldh;
  args.ldx = ldx;
  args.ldr = ldr;
  args.ldy = ldy;
  args.gate_row = gate_row;
  args.gate_col = gate_col;
  args.M = (int)M;
  args.D = (int)D;
  args.dtype = dtype;
  args.wdtype = weight_dtype;
  args.quant = quantize;
  args.residual_scale = residual_scale;
  args.eps = eps;
  args.weight_offset = weight_offset;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_block_norm(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

// ---------------------------------------------------------------------------
// Operators by which every token picks its weights (fp8bg_tokens.h).
// ---------------------------------------------------------------------------
namespace {

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether an output overlaps an input or another output.
template <int O, int I>
bool any_overlap(const Range (&out)[O], const Range (&in)[I]) {
  for (int i = 0; i < O; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i].p, out[i].bytes, r.p, r.bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

using fbg::kMaxRouted;
constexpr int64_t kMaxTopk = 64;
constexpr int64_t kMaxRank = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 35;  // workgroups of a grid of two dimensions

}  // namespace

extern "C" int fbg_route_experts(const void* logits, int64_t ld, int dtype, int64_t T, int64_t E, int64_t topk,
                                 int score, const float* bias, int64_t groups, int64_t topk_groups, int group_score,
                                 int renormalize, float scale, const uint8_t* mask, float* weights, int32_t* experts,
                                 void* stream) {
  if (T < 0 || E < 0 || topk < 0 || !known_dtype(dtype) || (score != FBG_SCORE_SOFTMAX && score != FBG_SCORE_SIGMOID) ||
      (group_score != FBG_GROUP_MAX && group_score != FBG_GROUP_TOP2) || groups < 1 || topk_groups < 1 ||
      topk_groups > groups || E % groups != 0)
    return FBG_ERROR_INVALID_VALUE;
  if (T > kMaxExtent || E > kMaxRouted || topk > kMaxTopk || groups > kMaxTopk) return FBG_ERROR_UNSUPPORTED;
  if (topk > E / groups * topk_groups || (T > 1 && ld < E)) return FBG_ERROR_INVALID_VALUE;
  if (T <= 1) ld = E;
  const int64_t es = elem_size(dtype);
  int64_t bytesL = 0;
  if (!extent(T, E, ld, es, &bytesL)) return FBG_ERROR_UNSUPPORTED;
  if (T == 0 || topk == 0) return FBG_SUCCESS;
  if (!logits || !weights || !experts) return FBG_ERROR_INVALID_VALUE;
  const Range out[] = {{weights, T * topk * 4}, {experts, T * topk * 4}};
  const Range in[] = {{logits, bytesL}, {bias, E * 4}, {mask, T}};
  if (any_overlap(out, in)) return FBG_ERROR_INVALID_VALUE;
  if (!aligned(logits, (uintptr_t)es) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(experts, 4))
    return FBG_ERROR_UNSUPPORTED;
  fbg::RouteArgs args;
  args.logits = logits;
  args.bias = bias;
  args.mask = mask;
  args.weights = weights;
  args.experts = experts;
  args.ld = ld;
  args.T = (int)T;
  args.E = (int)E;
  args.topk = (int)topk;
  args.groups = topk_groups == groups ? 1 : (int)groups;  // all groups stay: none to choose
  args.topk_groups = (int)topk_groups;
  args.group_lanes = 0;
  args.group_inverse = 0;
  args.dtype = dtype;
  args.score = score;
  args.group_score = group_score;
  args.renormalize = renormalize != 0;
  args.scale = scale;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_route(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

extern "C" int fbg_dispatch_tokens(const int32_t* experts, int64_t T, int64_t topk, int64_t first_expert, int64_t E,
                                   const void* x, int64_t ldx, int64_t K, int size, const float* x_scale, int64_t S,
                                   void* rows, int64_t ldrows, float* row_scale, int32_t* offsets, int32_t* slots,
                                   void* stream) {
  if (!x_scale) S = 0, row_scale = nullptr;
  if (T < 0 || topk < 0 || E < 0 || first_expert < 0 || K < 0 || S < 0 || (size != 1 && size != 2 && size != 4))
    return FBG_ERROR_INVALID_VALUE;
  if (T > kMaxExtent || topk > kMaxTopk || E > kMaxRouted || K > kMaxExtent || S > kMaxExtent || T * topk > kMaxExtent ||
      first_expert > kMaxExtent)
    return FBG_ERROR_UNSUPPORTED;
  const int64_t n = T * topk;
  if ((T > 1 && ldx < K) || (n > 1 && ldrows < K)) return FBG_ERROR_INVALID_VALUE;
  if (T <= 1) ldx = K;
  if (n <= 1) ldrows = K;
  int64_t bytesX = 0, bytesR = 0, bytesXs = 0, bytesRs = 0;
  if (!extent(T, K, ldx, size, &bytesX) || !extent(n, K, ldrows, size, &bytesR) || !extent(T, S, S, 4, &bytesXs) ||
      !extent(n, S, S, 4, &bytesRs))
    return FBG_ERROR_UNSUPPORTED;
  if (!offsets || (n > 0 && (!experts || !slots)) || (n > 0 && bytesX > 0 && (!x || !rows)) || (bytesRs > 0 && !row_scale))
    return FBG_ERROR_INVALID_VALUE;
  if (n == 0) x = nullptr, rows = nullptr;
  const Range out[] = {{rows, bytesR}, {row_scale, bytesRs}, {offsets, (E + 1) * 4}, {slots, n * 4}};
  const Range in[] = {{experts, n * 4}, {x, bytesX}, {x_scale, bytesXs}};
  if (any_overlap(out, in)) return FBG_ERROR_INVALID_VALUE;
  if (!aligned(experts, 4) || !aligned(x, (uintptr_t)size) || !aligned(x_scale, 4) || !aligned(rows, (uintptr_t)size) ||
      !aligned(row_scale, 4) || !aligned(offsets, 4) || !aligned(slots, 4))
    return FBG_ERROR_UNSUPPORTED;
  fbg::DispatchArgs args;
  args.experts = experts;
  args.x = static_cast<const uint8_t*>(x);
  args.x_scale = bytesXs > 0 ? reinterpret_cast<const uint8_t*>(x_scale) : nullptr;
  args.rows = static_cast<uint8_t*>(rows);
  args.row_scale = reinterpret_cast<uint8_t*>(row_scale);
  args.offsets = offsets;
  args.slots = slots;
  args.x_pitch = ldx * size;
  args.row_bytes = K * size;
  args.rows_pitch = ldrows * size;
  args.scale_bytes = S * 4;
  args.first = (int)first_expert;
  args.own = 0;
  args.T = (int)T;
  args.topk = (int)topk;
  args.n = (int)n;
  args.E = (int)E;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_dispatch(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

extern "C" int fbg_combine_experts(const void* rows, int64_t ldrows, int dtype, int64_t R, const int32_t* slots,
                                   const float* weights, const void* base, int64_t ldbase, int base_dtype, void* out,
                                   int64_t ldout, int out_dtype, int64_t T, int64_t topk, int64_t D, void* stream) {
  if (R < 0 || T < 0 || topk < 0 || D < 0 || !known_dtype(dtype) || !known_dtype(out_dtype) ||
      (base && base_dtype != dtype && base_dtype != out_dtype))
    return FBG_ERROR_INVALID_VALUE;
  if (R > kMaxExtent || T > kMaxExtent || topk > kMaxTopk || D > kMaxExtent) return FBG_ERROR_UNSUPPORTED;
  if ((R > 1 && ldrows < D) || (T > 1 && (ldout < D || (base && ldbase < D)))) return FBG_ERROR_INVALID_VALUE;
  if (R <= 1) ldrows = D;
  if (T <= 1) ldbase = ldout = D;
  const int64_t es = elem_size(dtype), os = elem_size(out_dtype), bs = elem_size(base ? base_dtype : dtype);
  int64_t bytesR = 0, bytesB = 0, bytesO = 0;
  if (!extent(R, D, ldrows, es, &bytesR) || !extent(T, D, base ? ldbase : D, bs, &bytesB) ||
      !extent(T, D, ldout, os, &bytesO))
    return FBG_ERROR_UNSUPPORTED;
  if (T == 0 || D == 0) return FBG_SUCCESS;
  if ((bytesR > 0 && !rows) || !out || (topk > 0 && (!slots || !weights))) return FBG_ERROR_INVALID_VALUE;
  const bool in_place = base == out && ldbase == ldout && base_dtype == out_dtype;
  const Range o[] = {{out, bytesO}};
  const Range in[] = {{rows, bytesR}, {slots, T * topk * 4}, {weights, T * topk * 4}, {in_place ? nullptr : base, bytesB}};
  if (any_overlap(o, in)) return FBG_ERROR_INVALID_VALUE;
  if (!aligned(rows, (uintptr_t)es) || !aligned(slots, 4) || !aligned(weights, 4) || !aligned(base, (uintptr_t)bs) ||
      !aligned(out, (uintptr_t)os))
    return FBG_ERROR_UNSUPPORTED;
  fbg::CombineArgs args;
  args.rows = rows;
  args.slots = slots;
  args.weights = weights;
  args.base = base;
  args.out = out;
  args.ldrows = ldrows;
  args.ldbase = ldbase;
  args.ldout = ldout;
  args.R = (int)R;
  args.T = (int)T;
  args.topk = (int)topk;
  args.D = (int)D;
  args.dtype = dtype;
  args.out_dtype = out_dtype;
  args.base_is_out = base && base_dtype == out_dtype;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_combine(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}

namespace {

int adapter_pitch(int64_t R) { return (int)((R + 15) / 16 * 16); }

// Bytes of h; false if that overflows.
bool adapter_workspace(int64_t M, int64_t K, int64_t R, int64_t* bytes) {
  return !__builtin_mul_overflow(M * fbg::adapter_splits(M, K, R), (int64_t)adapter_pitch(R) * 4, bytes);
}

}  // namespace

extern "C" size_t fbg_add_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R) {
  int64_t bytes = 0;
  if (M < 0 || N < 0 || K < 0 || R < 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxK || R > kMaxRank ||
      !adapter_workspace(M, K, R, &bytes))
    return (size_t)-1;
  return M == 0 || N == 0 || K == 0 || R == 0 ? 0 : (size_t)bytes;
}

extern "C" int fbg_add_adapters(const void* y, int64_t ldy, const void* x, int64_t ldx, const void* A, const void* B,
                                const int32_t* adapters, const float* scales, void* out, int64_t ldout, int64_t M,
                                int64_t N, int64_t K, int64_t R, int64_t L, int dtype, int out_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || L < 0 || (dtype != FBG_OUT_BF16 && dtype != FBG_OUT_FP16) ||
      !known_dtype(out_dtype))
    return FBG_ERROR_INVALID_VALUE;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxK || R > kMaxRank || L > kMaxExtent) return FBG_ERROR_UNSUPPORTED;
  if (M > 1 && (ldy < N || ldx < K || ldout < N)) return FBG_ERROR_INVALID_VALUE;
  if (M <= 1) ldy = ldout = N, ldx = K;
  const int64_t os = elem_size(out_dtype);
  int64_t bytesX = 0, bytesY = 0, bytesO = 0, bytesA = 0, bytesB = 0, need = 0;
  if (!extent(M, K, ldx, 2, &bytesX) || !extent(M, N, ldy, os, &bytesY) || !extent(M, N, ldout, os, &bytesO) ||
      __builtin_mul_overflow(L * R, K * 2, &bytesA) || __builtin_mul_overflow(L * R, N * 2, &bytesB) ||
      !adapter_workspace(M, K, R, &need) || (M + 15) / 16 * ((N + 63) / 64) > kMaxBlocks)
    return FBG_ERROR_UNSUPPORTED;
  if (M == 0 || N == 0) return FBG_SUCCESS;
  const bool any = K > 0 && R > 0 && L > 0;
  if (!y || !out || (any && (!x || !A || !B || !adapters))) return FBG_ERROR_INVALID_VALUE;
  if (!any) x = A = B = nullptr, adapters = nullptr, scales = nullptr, need = 0, L = 0;
  if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return FBG_ERROR_OUT_OF_MEMORY;
  const bool in_place = y == out && ldy == ldout;
  const Range o[] = {{out, bytesO}, {workspace, need}};
  const Range in[] = {{in_place ? nullptr : y, bytesY}, {x, bytesX}, {A, bytesA}, {B, bytesB}, {adapters, M * 4},
                      {scales, L * 4}};
  if (any_overlap(o, in)) return FBG_ERROR_INVALID_VALUE;
  if (!aligned(y, (uintptr_t)os) || !aligned(out, (uintptr_t)os) || !aligned(x, 2) || !aligned(A, 2) || !aligned(B, 2) ||
      !aligned(adapters, 4) || !aligned(scales, 4) || (need > 0 && !aligned(workspace, 16)))
    return FBG_ERROR_UNSUPPORTED;
  if (!any && in_place) return FBG_SUCCESS;
  fbg::AdapterArgs args;
  args.y = y;
  args.x = x;
  args.A = A;
  args.B = B;
  args.adapters = adapters;
  args.scales = scales;
  args.out = out;
  args.h = static_cast<float*>(workspace);
  args.ldy = ldy;
  args.ldx = ldx;
  args.ldout = ldout;
  args.M = (int)M;
  args.N = (int)N;
  args.K = (int)K;
  args.R = (int)R;
  args.L = (int)L;
  args.pitch = adapter_pitch(R);
  args.splits = fbg::adapter_splits(M, K, R);
  args.in_place = in_place;
  args.dtype = dtype;
  args.out_dtype = out_dtype;
  args.workers = args.share = args.cols = 0;
  args.stream = static_cast<hipStream_t>(stream);
  return fbg::launch_add_adapters(args) == hipSuccess ? FBG_SUCCESS : FBG_ERROR_HIP;
}
