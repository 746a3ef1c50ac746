// C ABI of libcider (declared in include/cider.h): argument validation,
// device gate and kernel dispatch. Every argument check runs before the first
// HIP call, so a bad call returns CIDER_ERROR_INVALID_VALUE with nothing
// enqueued, also on a machine without a GPU.
#include "../../include/cider.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "cider_internal.h"

namespace {

constexpr int kVersion = 100;   // 0.1.0

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_gs(int32_t gs) { return gs == 0 || gs == 64 || gs == 128; }

// K must be a positive multiple of `mult` (1 for int8 codes, 2 for packed
// int4, 16 where a kernel family needs aligned rows), at most CIDER_MAX_K,
// and a multiple of the group size.
bool valid_k(int64_t K, int64_t mult, int32_t gs) {
  if (K <= 0 || K > CIDER_MAX_K || K % mult) return false;
  return gs == 0 || K % gs == 0;
}

// Per-device architecture flag: 1 = gfx950, 0 = other, -1 = not yet queried.
constexpr int kMaxDevices = 64;
struct ArchCache {
  std::atomic<int> ok[kMaxDevices];
  ArchCache() {
    for (auto& a : ok) a.store(-1);
  }
};

ArchCache& arch_cache() {
  static ArchCache cache;   // thread-safe one-time construction
  return cache;
}

bool device_is_gfx950() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return false;
  if (dev < kMaxDevices) {
    const int cached = arch_cache().ok[dev].load();
    if (cached >= 0) return cached == 1;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return false;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) arch_cache().ok[dev].store(ok ? 1 : 0);
  return ok;
}

cider_status_t from_hip(hipError_t e) { return e == hipSuccess ? CIDER_SUCCESS : CIDER_ERROR_LAUNCH; }

// Split-K scratch of cider_w8a8_gemm_noalloc (for callers that cannot
// allocate). Every GPU that loads the library holds its own copy of this
// array until the process ends; in host code its name is only a stand-in, so
// the kernels get the device address looked up below, never the name.
static __device__ __align__(256) int8_t scratch[CIDER_NOALLOC_SCRATCH_BYTES];

// This device's address of `scratch`, looked up on the device's first
// no-allocation call (with the device current) and kept; null if the lookup
// fails.
std::atomic<void*> g_scratch[kMaxDevices];
std::atomic<int> g_scratch_state[kMaxDevices];   // 0 = not looked up, 1 = ok, 2 = failed
std::mutex g_scratch_mu;

void* scratch_address() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  if (g_scratch_state[dev].load(std::memory_order_acquire) == 0) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (g_scratch_state[dev].load(std::memory_order_relaxed) == 0) {
      void* ptr = nullptr;
      const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
      g_scratch[dev].store(e == hipSuccess ? ptr : nullptr, std::memory_order_relaxed);
      g_scratch_state[dev].store(e == hipSuccess && ptr ? 1 : 2, std::memory_order_release);
    }
  }
  return g_scratch_state[dev].load(std::memory_order_acquire) == 1 ? g_scratch[dev].load() : nullptr;
}

}  // namespace

extern "C" {

int cider_version(void) { return kVersion; }

const char* cider_status_string(cider_status_t s) {
  switch (s) {
    case CIDER_SUCCESS: return "success";
    case CIDER_ERROR_INVALID_VALUE: return "invalid argument (null/misaligned pointer, bad size or group size)";
    case CIDER_ERROR_NOT_SUPPORTED: return "not supported (no gfx950 device is current)";
    case CIDER_ERROR_LAUNCH: return "kernel launch failed";
    case CIDER_ERROR_SCRATCH_LIMIT:
      return "the shape's split-K plan needs more scratch than cider_w8a8_gemm_noalloc holds "
             "(CIDER_NOALLOC_SCRATCH_BYTES = 48 MiB)";
  }
  return "unknown status";
}

int cider_is_available(void) {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) return 0;
  return device_is_gfx950() ? 1 : 0;
}

static bool valid_dtype(int32_t d) { return d == CIDER_DTYPE_F16 || d == CIDER_DTYPE_BF16; }

cider_status_t cider_quant_act_dt(const void* x, int32_t x_dtype, int64_t M, int64_t K, int32_t group_size,
                                  int8_t* x_q, float* x_scale, void* stream) {
  if (!valid_dtype(x_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (M < 0 || !valid_gs(group_size) || !valid_k(K, 1, group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0) return CIDER_SUCCESS;
  if (!x || !x_q || !x_scale || !aligned16(x) || !aligned16(x_q) || !aligned16(x_scale))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_quant_rows(x, M, K, group_size, 127, x_q, x_scale, static_cast<hipStream_t>(stream),
                                           x_dtype == CIDER_DTYPE_BF16));
}

cider_status_t cider_quant_act(const void* x_f16, int64_t M, int64_t K, int32_t group_size, int8_t* x_q,
                               float* x_scale, void* stream) {
  return cider_quant_act_dt(x_f16, CIDER_DTYPE_F16, M, K, group_size, x_q, x_scale, stream);
}

cider_status_t cider_quant_weight(const void* w_f16, int64_t N, int64_t K, int32_t bits, int32_t group_size,
                                  void* w_q, float* w_scale, void* stream) {
  return cider_quant_weight_dt(w_f16, CIDER_DTYPE_F16, N, K, bits, group_size, w_q, w_scale, stream);
}

cider_status_t cider_quant_weight_dt(const void* w, int32_t w_dtype, int64_t N, int64_t K, int32_t bits,
                                     int32_t group_size, void* w_q, float* w_scale, void* stream) {
  if (!valid_dtype(w_dtype)) return CIDER_ERROR_INVALID_VALUE;
  const void* w_f16 = w;
  if (N < 0 || !valid_gs(group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (bits == 8) {
    if (!valid_k(K, 1, group_size)) return CIDER_ERROR_INVALID_VALUE;
  } else if (bits == 4) {
    if (group_size != 0 || !valid_k(K, 2, 0)) return CIDER_ERROR_INVALID_VALUE;
  } else {
    return CIDER_ERROR_INVALID_VALUE;
  }
  if (N == 0) return CIDER_SUCCESS;
  if (!w_f16 || !w_q || !w_scale || !aligned16(w_f16) || !aligned16(w_q) || !aligned16(w_scale))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_quant_rows(w_f16, N, K, group_size, bits == 8 ? 127 : 7, w_q, w_scale,
                                           static_cast<hipStream_t>(stream), w_dtype == CIDER_DTYPE_BF16));
}

cider_status_t cider_quant_weight_clip(const void* w_f16, int32_t w_dtype, int64_t N, int64_t K, int32_t bits,
                                       int32_t group_size, double percentile, void* w_q, float* w_scale,
                                       void* stream) {
  if (!valid_dtype(w_dtype) || N < 0 || !valid_gs(group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (!(percentile >= 0.0 && percentile <= 100.0)) return CIDER_ERROR_INVALID_VALUE;   // NaN fails too
  if (bits == 8) {
    if (!valid_k(K, 16, group_size)) return CIDER_ERROR_INVALID_VALUE;
  } else if (bits == 4) {
    if (group_size != 0 || !valid_k(K, 32, 0)) return CIDER_ERROR_INVALID_VALUE;
  } else {
    return CIDER_ERROR_INVALID_VALUE;
  }
  const int64_t G = group_size ? K / group_size : 1;
  if (N * G >= (int64_t(1) << 31)) return CIDER_ERROR_INVALID_VALUE;
  if (N == 0) return CIDER_SUCCESS;
  if (!w_f16 || !w_q || !w_scale || !aligned16(w_f16) || !aligned16(w_q) || !aligned16(w_scale))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_quant_rows_clip(w_f16, N, K, group_size, bits == 8 ? 127 : 7, percentile, w_q,
                                                w_scale, static_cast<hipStream_t>(stream),
                                                w_dtype == CIDER_DTYPE_BF16));
}

static cider_status_t gemm_common(cider::GemmArgs& g, cider::WeightKind wk, cider::Epilogue epi,
                                  void* stream) {
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_gemm(g, wk, epi, static_cast<hipStream_t>(stream)));
}

static bool gemm_sizes_ok(int64_t M, int64_t N) {
  return M >= 0 && N >= 0 && M < (int64_t(1) << 31) && N < (int64_t(1) << 31);
}

cider_status_t cider_w8a8_gemm(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                               const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t group_size,
                               void* y_f16, void* stream) {
  return cider_w8a8_gemm_dt(x_q, x_scale, w_q, w_scale, M, N, K, group_size, y_f16, CIDER_DTYPE_F16, stream);
}

int64_t cider_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t bits, int32_t group_size) {
  if (!gemm_sizes_ok(M, N) || !valid_gs(group_size) || (bits != 8 && bits != 4)) return -1;
  if (bits == 4 && (group_size != 0 || !valid_k(K, 2, 0))) return -1;
  if (bits == 8 && !valid_k(K, 1, group_size)) return -1;
  if (M == 0 || N == 0) return 0;
  return cider::gemm_split_workspace_bytes(M, N, K, bits == 4 ? cider::kWeightI4 : cider::kWeightI8, group_size);
}

// A caller workspace, when given, must hold the size query's bytes.
static bool workspace_ok(const void* ws, int64_t ws_bytes, int64_t need) {
  if (!ws) return true;
  return aligned16(ws) && ws_bytes >= need;
}

cider_status_t cider_w8a8_gemm_dt(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                  const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                  void* y_f16, int32_t y_dtype, void* stream) {
  return cider_w8a8_gemm_ex(x_q, x_scale, w_q, w_scale, M, N, K, group_size, y_f16, y_dtype, nullptr, 0, stream);
}

cider_status_t cider_w8a8_gemm_ex(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                  const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                  void* y_f16, int32_t y_dtype, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (!gemm_sizes_ok(M, N) || !valid_gs(group_size) || !valid_k(K, 1, group_size))
    return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !w_q || !w_scale || !y_f16) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w_q) || !aligned16(w_scale) || !aligned16(y_f16))
    return CIDER_ERROR_INVALID_VALUE;
  if (!workspace_ok(workspace, workspace_bytes, cider_gemm_workspace_size(M, N, K, 8, group_size)))
    return CIDER_ERROR_INVALID_VALUE;
  cider::GemmArgs g{x_q, x_scale, w_q, w_scale, M, N, K, group_size, y_f16, nullptr};
  g.ws = workspace;
  g.ws_bytes = workspace ? workspace_bytes : 0;
  return gemm_common(g, cider::kWeightI8, y_dtype == CIDER_DTYPE_BF16 ? cider::kEpiBF16 : cider::kEpiF16, stream);
}

cider_status_t cider_w8a8_gemm_noalloc(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                       const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                       void* y, int32_t y_dtype, void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (!gemm_sizes_ok(M, N) || !valid_gs(group_size) || !valid_k(K, 1, group_size))
    return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !w_q || !w_scale || !y) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w_q) || !aligned16(w_scale) || !aligned16(y))
    return CIDER_ERROR_INVALID_VALUE;
  const int64_t need = cider_gemm_workspace_size(M, N, K, 8, group_size);
  if (need > CIDER_NOALLOC_SCRATCH_BYTES) return CIDER_ERROR_SCRATCH_LIMIT;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  cider::GemmArgs g{x_q, x_scale, w_q, w_scale, M, N, K, group_size, y, nullptr};
  if (need > 0) {
    // every slab element the reduction reads is written first by the same
    // call's split kernel, so nothing in the scratch needs clearing
    g.ws = scratch_address();
    if (!g.ws) return CIDER_ERROR_LAUNCH;
    g.ws_bytes = CIDER_NOALLOC_SCRATCH_BYTES;
  }
  return from_hip(cider::launch_gemm(g, cider::kWeightI8,
                                     y_dtype == CIDER_DTYPE_BF16 ? cider::kEpiBF16 : cider::kEpiF16,
                                     static_cast<hipStream_t>(stream)));
}

cider_status_t cider_w4a8_gemm(const int8_t* x_q, const float* x_scale, const uint8_t* w_packed,
                               const float* w_scale, int64_t M, int64_t N, int64_t K, void* y_f16,
                               void* stream) {
  return cider_w4a8_gemm_dt(x_q, x_scale, w_packed, w_scale, M, N, K, y_f16, CIDER_DTYPE_F16, stream);
}

cider_status_t cider_w4a8_gemm_dt(const int8_t* x_q, const float* x_scale, const uint8_t* w_packed,
                                  const float* w_scale, int64_t M, int64_t N, int64_t K, void* y_f16,
                                  int32_t y_dtype, void* stream) {
  return cider_w4a8_gemm_ex(x_q, x_scale, w_packed, w_scale, M, N, K, y_f16, y_dtype, nullptr, 0, stream);
}

cider_status_t cider_w4a8_gemm_ex(const int8_t* x_q, const float* x_scale, const uint8_t* w_packed,
                                  const float* w_scale, int64_t M, int64_t N, int64_t K, void* y_f16,
                                  int32_t y_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (!gemm_sizes_ok(M, N) || !valid_k(K, 2, 0)) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !w_packed || !w_scale || !y_f16) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w_packed) || !aligned16(w_scale) ||
      !aligned16(y_f16))
    return CIDER_ERROR_INVALID_VALUE;
  if (!workspace_ok(workspace, workspace_bytes, cider_gemm_workspace_size(M, N, K, 4, 0)))
    return CIDER_ERROR_INVALID_VALUE;
  cider::GemmArgs g{x_q, x_scale, w_packed, w_scale, M, N, K, 0, y_f16, nullptr};
  g.ws = workspace;
  g.ws_bytes = workspace ? workspace_bytes : 0;
  return gemm_common(g, cider::kWeightI4, y_dtype == CIDER_DTYPE_BF16 ? cider::kEpiBF16 : cider::kEpiF16, stream);
}

cider_status_t cider_w8a8_gemm_token_group_dt(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                              const float* w_scale, int64_t M, int64_t N, int64_t K,
                                              int32_t group_size, void* y, int32_t y_dtype, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (!gemm_sizes_ok(M, N) || (group_size != 64 && group_size != 128) || !valid_k(K, 16, group_size))
    return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !w_q || !w_scale || !y) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w_q) || !aligned16(w_scale) || !aligned16(y))
    return CIDER_ERROR_INVALID_VALUE;
  if (!workspace_ok(workspace, workspace_bytes, cider_gemm_workspace_size(M, N, K, 8, group_size)))
    return CIDER_ERROR_INVALID_VALUE;
  cider::GemmArgs g{x_q, x_scale, w_q, w_scale, M, N, K, group_size, y, nullptr};
  g.ws = workspace;
  g.ws_bytes = workspace ? workspace_bytes : 0;
  return gemm_common(g, cider::kWeightI8, y_dtype == CIDER_DTYPE_BF16 ? cider::kEpiBF16Tok : cider::kEpiF16Tok,
                     stream);
}

cider_status_t cider_w8a8_gemm_token_group(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                           const float* w_scale, int64_t M, int64_t N, int64_t K,
                                           int32_t group_size, void* y_f16, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  return cider_w8a8_gemm_token_group_dt(x_q, x_scale, w_q, w_scale, M, N, K, group_size, y_f16, CIDER_DTYPE_F16,
                                        workspace, workspace_bytes, stream);
}

cider_status_t cider_w8a8_gemm_split_dt(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                        const float* w_scale, int64_t M, int64_t K, int32_t n_parts,
                                        const int64_t* part_n, void* const* y_parts, int32_t y_dtype,
                                        void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (M < 0 || M >= (int64_t(1) << 31) || !valid_k(K, 16, 0)) return CIDER_ERROR_INVALID_VALUE;
  if (n_parts < 1 || n_parts > CIDER_SPLIT_MAX_PARTS || !part_n || !y_parts) return CIDER_ERROR_INVALID_VALUE;
  cider::OutSplit sp{};
  int64_t N = 0;
  for (int32_t i = 0; i < n_parts; ++i) {
    if (part_n[i] <= 0 || part_n[i] % 16 != 0) return CIDER_ERROR_INVALID_VALUE;
    N += part_n[i];
    if (N >= (int64_t(1) << 31)) return CIDER_ERROR_INVALID_VALUE;
    sp.y[i] = static_cast<_Float16*>(y_parts[i]);
    sp.end[i] = (int)N;
  }
  for (int32_t i = n_parts; i < CIDER_SPLIT_MAX_PARTS; ++i) {
    sp.y[i] = sp.y[n_parts - 1];
    sp.end[i] = (int)N;
  }
  if (M == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !w_q || !w_scale) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w_q) || !aligned16(w_scale)) return CIDER_ERROR_INVALID_VALUE;
  for (int32_t i = 0; i < n_parts; ++i)
    if (!y_parts[i] || !aligned16(y_parts[i])) return CIDER_ERROR_INVALID_VALUE;
  cider::GemmArgs g{x_q, x_scale, w_q, w_scale, M, N, K, 0, sp.y[0], nullptr};
  g.split = sp;
  return gemm_common(g, cider::kWeightI8, y_dtype == CIDER_DTYPE_BF16 ? cider::kEpiBF16Split : cider::kEpiF16Split,
                     stream);
}

cider_status_t cider_w8a8_gemm_split(const int8_t* x_q, const float* x_scale, const int8_t* w_q,
                                     const float* w_scale, int64_t M, int64_t K, int32_t n_parts,
                                     const int64_t* part_n, void* const* y_parts, void* stream) {
  return cider_w8a8_gemm_split_dt(x_q, x_scale, w_q, w_scale, M, K, n_parts, part_n, y_parts, CIDER_DTYPE_F16,
                                  stream);
}

// The one-call linear's workspace: the activation codes and scales (each
// 256-byte aligned), then room for the GEMM's split-K slabs.
static int64_t linear_quant_bytes(int64_t M, int64_t K, int32_t group_size) {
  const int64_t G = group_size ? K / group_size : 1;
  return (M * K + 255) / 256 * 256 + (4 * M * G + 255) / 256 * 256;
}

int64_t cider_linear_workspace_size(int64_t M, int64_t N, int64_t K, int32_t bits, int32_t group_size) {
  if (!gemm_sizes_ok(M, N) || !valid_gs(group_size) || (bits != 8 && bits != 4)) return -1;
  if (bits == 4 && group_size != 0) return -1;
  if (!valid_k(K, bits == 4 ? 2 : 1, group_size)) return -1;
  if (M == 0 || N == 0 || cider::linear_is_one_launch(M, K, group_size, bits == 4 ? cider::kWeightI4 : cider::kWeightI8)) return 0;
  return linear_quant_bytes(M, K, group_size) + cider_gemm_workspace_size(M, N, K, bits, group_size);
}

cider_status_t cider_linear_dt(const void* x_f16, int32_t dtype, const void* w, const float* w_scale, int64_t M,
                               int64_t N, int64_t K, int32_t bits, int32_t group_size, void* workspace,
                               int64_t workspace_bytes, void* y_f16, void* stream) {
  if (!valid_dtype(dtype)) return CIDER_ERROR_INVALID_VALUE;
  const bool bf = dtype == CIDER_DTYPE_BF16;
  const int64_t need = cider_linear_workspace_size(M, N, K, bits, group_size);
  if (need < 0) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_f16 || !w || !w_scale || !y_f16) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_f16) || !aligned16(w) || !aligned16(w_scale) || !aligned16(y_f16)) return CIDER_ERROR_INVALID_VALUE;
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  const cider::WeightKind wk = bits == 4 ? cider::kWeightI4 : cider::kWeightI8;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (need == 0) {   // one launch: the GEMV kernel quantizes its activations itself
    cider::GemmArgs g{static_cast<const int8_t*>(x_f16), nullptr, w, w_scale, M, N, K, 0, y_f16, nullptr};
    return from_hip(cider::launch_gemm(g, wk, bf ? cider::kEpiBF16Linear : cider::kEpiF16Linear, st));
  }
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* sa = reinterpret_cast<float*>(static_cast<char*>(workspace) + (M * K + 255) / 256 * 256);
  hipError_t e = cider::launch_quant_rows(x_f16, M, K, group_size, 127, xq, sa, st, bf);
  if (e != hipSuccess) return from_hip(e);
  cider::GemmArgs g{xq, sa, w, w_scale, M, N, K, group_size, y_f16, nullptr};
  const int64_t qb = linear_quant_bytes(M, K, group_size);
  if (need > qb) {   // the split-K slabs follow the codes and scales
    g.ws = static_cast<char*>(workspace) + qb;
    g.ws_bytes = workspace_bytes - qb;
  }
  return from_hip(cider::launch_gemm(g, wk, bf ? cider::kEpiBF16 : cider::kEpiF16, st));
}

cider_status_t cider_linear(const void* x_f16, const void* w, const float* w_scale, int64_t M, int64_t N,
                            int64_t K, int32_t bits, int32_t group_size, void* workspace,
                            int64_t workspace_bytes, void* y_f16, void* stream) {
  return cider_linear_dt(x_f16, CIDER_DTYPE_F16, w, w_scale, M, N, K, bits, group_size, workspace, workspace_bytes,
                         y_f16, stream);
}

cider_status_t cider_int8_mv(const void* x_f16, const int8_t* w_q, const float* w_scale, int64_t M, int64_t N,
                             int64_t K, int32_t group_size, void* y_f16, void* stream) {
  if (M < 0 || M > CIDER_MV_MAX_M || !gemm_sizes_ok(M, N) || !valid_gs(group_size) || !valid_k(K, 16, group_size))
    return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_f16 || !w_q || !w_scale || !y_f16) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_f16) || !aligned16(w_q) || !aligned16(w_scale) || !aligned16(y_f16))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  cider::MvArgs a{x_f16, w_q, w_scale, M, N, K, group_size, y_f16};
  return from_hip(cider::launch_mv(a, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_read_probe(const void* buf, int64_t bytes, int32_t* sink, void* stream) {
  if (bytes < 0 || bytes % 16) return CIDER_ERROR_INVALID_VALUE;
  if (bytes == 0) return CIDER_SUCCESS;
  if (!buf || !sink || !aligned16(buf) || !aligned16(sink)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_read_probe(buf, bytes, sink, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_gemm_acc_i32(int32_t mode, const int8_t* x_q, const void* w, int64_t M, int64_t N,
                                  int64_t K, int32_t group_size, int32_t* acc, void* stream) {
  if (mode != 0 && mode != 1) return CIDER_ERROR_INVALID_VALUE;
  if (!gemm_sizes_ok(M, N) || !valid_gs(group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (mode == 1 && (group_size != 0 || !valid_k(K, 2, 0))) return CIDER_ERROR_INVALID_VALUE;
  if (mode == 0 && !valid_k(K, 1, group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || N == 0) return CIDER_SUCCESS;
  if (!x_q || !w || !acc || !aligned16(x_q) || !aligned16(w) || !aligned16(acc)) return CIDER_ERROR_INVALID_VALUE;
  cider::GemmArgs g{x_q, nullptr, w, nullptr, M, N, K, group_size, nullptr, acc};
  return gemm_common(g, mode == 1 ? cider::kWeightI4 : cider::kWeightI8, cider::kEpiAccI32, stream);
}

}  // extern "C"

// Stack workspace regions 0..8 (see include/cider.h) plus region 9: the int32
// partial sums of a split-K GEMM (the largest the stack's per-projection GEMMs
// need; 0 bytes when none splits). Returns the total, 0 for invalid dims.
static int64_t stack_layout(int64_t M, int64_t hidden, int64_t q_dim, int64_t kv_dim, int64_t mlp_dim,
                            int64_t off[10]) {
  if (M < 0 || hidden <= 0 || q_dim <= 0 || kv_dim <= 0 || mlp_dim <= 0) return 0;
  if (hidden % 16 || q_dim % 16 || kv_dim % 16 || mlp_dim % 16) return 0;
  const int64_t kmax = std::max(hidden, std::max(q_dim, mlp_dim));
  int64_t split = 0;
  if (M > 0) {
    const int64_t nk[4][2] = {{q_dim, hidden}, {kv_dim, hidden}, {hidden, q_dim}, {mlp_dim, hidden}};
    for (const auto& p : nk)
      split = std::max(split, cider::gemm_split_workspace_bytes(M, p[0], p[1], cider::kWeightI8, 0));
    split = std::max(split, cider::gemm_split_workspace_bytes(M, hidden, mlp_dim, cider::kWeightI8, 0));
  }
  const int64_t sizes[10] = {M * kmax, 4 * M, 2 * M * q_dim, 2 * M * kv_dim, 2 * M * kv_dim,
                             2 * M * hidden, 2 * M * mlp_dim, 2 * M * mlp_dim, 2 * M * hidden, split};
  int64_t o = 0;
  for (int i = 0; i < 10; ++i) {
    off[i] = o;
    o += (sizes[i] + 255) / 256 * 256;
  }
  return o;
}

extern "C" {

int64_t cider_stack_workspace_layout(int64_t M, int64_t hidden, int64_t q_dim, int64_t kv_dim, int64_t mlp_dim,
                                     int64_t* offsets) {
  int64_t off[10];
  const int64_t total = stack_layout(M, hidden, q_dim, kv_dim, mlp_dim, off);
  if (total && offsets)
    for (int i = 0; i < 9; ++i) offsets[i] = off[i];
  return total;
}

cider_status_t cider_stack_forward_dt(const void* x_f16, int32_t dtype, int64_t M, int64_t hidden, int64_t q_dim,
                                      int64_t kv_dim, int64_t mlp_dim, int32_t n_layers,
                                      const cider_stack_layer_t* layers, void* workspace, int64_t workspace_bytes,
                                      void* y_f16, void* stream) {
  if (!valid_dtype(dtype)) return CIDER_ERROR_INVALID_VALUE;
  const bool bf = dtype == CIDER_DTYPE_BF16;
  int64_t off[10];
  const int64_t need = stack_layout(M, hidden, q_dim, kv_dim, mlp_dim, off);
  if (need == 0 || n_layers < 0 || M >= (int64_t(1) << 31)) return CIDER_ERROR_INVALID_VALUE;
  if (std::max(hidden, std::max(q_dim, mlp_dim)) > CIDER_MAX_K) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0 || n_layers == 0) return CIDER_SUCCESS;
  if (!x_f16 || !layers || !workspace || !y_f16 || workspace_bytes < need) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_f16) || !aligned16(workspace) || !aligned16(y_f16)) return CIDER_ERROR_INVALID_VALUE;
  for (int32_t l = 0; l < n_layers; ++l)
    for (int j = 0; j < 7; ++j)
      if (!layers[l].w[j] || !layers[l].s[j] || !aligned16(layers[l].w[j]) || !aligned16(layers[l].s[j]))
        return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;

  char* ws = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(ws + off[0]);
  float* sa = reinterpret_cast<float*>(ws + off[1]);
  void* q = ws + off[2];
  void* k = ws + off[3];
  void* v = ws + off[4];
  void* o = ws + off[5];
  void* g = ws + off[6];
  void* u = ws + off[7];
  void* h = ws + off[8];
  hipStream_t st = static_cast<hipStream_t>(stream);

  auto quant = [&](const void* in, int64_t K) { return cider::launch_quant_rows(in, M, K, 0, 127, xq, sa, st, bf); };
  auto gemm = [&](const cider_stack_layer_t& L, int j, int64_t N, int64_t K, void* out) {
    cider::GemmArgs a{xq, sa, L.w[j], L.s[j], M, N, K, 0, out, nullptr};
    // split-K partials (e.g. the long-K down projection); stream order keeps
    // one GEMM's partials from overlapping the next one's
    if (need > off[9]) {
      a.ws = ws + off[9];
      a.ws_bytes = need - off[9];
    }
    return cider::launch_gemm(a, cider::kWeightI8, bf ? cider::kEpiBF16 : cider::kEpiF16, st);
  };
  // Projections j, j+1[, j+2] of one input as one GEMM when their codes and
  // scales are adjacent in memory, in that order (columns split to `outs`).
  auto adjacent = [&](const cider_stack_layer_t& L, int j, int parts, const int64_t* n) {
    for (int i = 1; i < parts; ++i) {
      if (L.w[j + i] != L.w[j + i - 1] + n[i - 1] * hidden) return false;
      if (L.s[j + i] != L.s[j + i - 1] + n[i - 1]) return false;
    }
    return true;
  };
  auto gemm_fused = [&](const cider_stack_layer_t& L, int j, int parts, const int64_t* n, void* const* outs) {
    cider::GemmArgs a{xq, sa, L.w[j], L.s[j], M, 0, hidden, 0, outs[0], nullptr};
    int64_t end = 0;
    for (int i = 0; i < cider::kMaxSplitParts; ++i) {
      if (i < parts) end += n[i];
      a.split.y[i] = static_cast<_Float16*>(outs[i < parts ? i : parts - 1]);
      a.split.end[i] = (int)end;
    }
    a.N = end;
    return cider::launch_gemm(a, cider::kWeightI8, bf ? cider::kEpiBF16Split : cider::kEpiF16Split, st);
  };
  const int64_t n_qkv[3] = {q_dim, kv_dim, kv_dim}, n_gu[2] = {mlp_dim, mlp_dim};
  const void* in = x_f16;
  for (int32_t l = 0; l < n_layers; ++l) {
    const cider_stack_layer_t& L = layers[l];
    void* out = l + 1 == n_layers ? y_f16 : h;
    void* const qkv_out[3] = {q, k, v};
    void* const gu_out[2] = {g, u};
    hipError_t e = quant(in, hidden);
    if (adjacent(L, 0, 3, n_qkv)) {
      if (e == hipSuccess) e = gemm_fused(L, 0, 3, n_qkv, qkv_out);
    } else {
      if (e == hipSuccess) e = gemm(L, 0, q_dim, hidden, q);
      if (e == hipSuccess) e = gemm(L, 1, kv_dim, hidden, k);
      if (e == hipSuccess) e = gemm(L, 2, kv_dim, hidden, v);
    }
    if (e == hipSuccess) e = quant(q, q_dim);
    if (e == hipSuccess) e = gemm(L, 3, hidden, q_dim, o);
    if (e == hipSuccess) e = quant(o, hidden);
    if (adjacent(L, 4, 2, n_gu)) {
      if (e == hipSuccess) e = gemm_fused(L, 4, 2, n_gu, gu_out);
    } else {
      if (e == hipSuccess) e = gemm(L, 4, mlp_dim, hidden, g);
      if (e == hipSuccess) e = gemm(L, 5, mlp_dim, hidden, u);
    }
    if (e == hipSuccess) e = quant(u, mlp_dim);
    if (e == hipSuccess) e = gemm(L, 6, hidden, mlp_dim, out);
    if (e != hipSuccess) return CIDER_ERROR_LAUNCH;
    in = out;   // stream order: the next layer's first quant reads h before h is rewritten
  }
  return CIDER_SUCCESS;
}

cider_status_t cider_stack_forward(const void* x_f16, int64_t M, int64_t hidden, int64_t q_dim, int64_t kv_dim,
                                   int64_t mlp_dim, int32_t n_layers, const cider_stack_layer_t* layers,
                                   void* workspace, int64_t workspace_bytes, void* y_f16, void* stream) {
  return cider_stack_forward_dt(x_f16, CIDER_DTYPE_F16, M, hidden, q_dim, kv_dim, mlp_dim, n_layers, layers,
                                workspace, workspace_bytes, y_f16, stream);
}

// ---- expert blocks ----------------------------------------------------------

static bool moe_sizes_ok(int64_t T, int32_t top_k, int32_t n_experts) {
  return T >= 0 && T < (int64_t(1) << 31) && top_k >= 1 && T * top_k < (int64_t(1) << 31) && n_experts >= 1 &&
         n_experts <= CIDER_MOE_MAX_EXPERTS;
}

int64_t cider_moe_plan_workspace_size(int64_t T, int32_t top_k, int32_t n_experts) {
  if (!moe_sizes_ok(T, top_k, n_experts)) return -1;
  return cider::moe_plan_workspace_bytes(T * top_k, n_experts);
}

cider_status_t cider_moe_plan(const int32_t* expert_ids, int64_t T, int32_t top_k, int32_t n_experts,
                              int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  if (!moe_sizes_ok(T, top_k, n_experts)) return CIDER_ERROR_INVALID_VALUE;
  if (!offsets || !aligned16(offsets)) return CIDER_ERROR_INVALID_VALUE;
  if (T > 0 && (!expert_ids || !rows || !slots)) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(expert_ids) || !aligned16(rows) || !aligned16(slots)) return CIDER_ERROR_INVALID_VALUE;
  const int64_t need = cider::moe_plan_workspace_bytes(T * top_k, n_experts);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_moe_plan(expert_ids, T * top_k, n_experts, offsets, rows, slots, workspace,
                                         static_cast<hipStream_t>(stream)));
}

static cider_status_t grouped_common(const int8_t* x_q, const float* x_scale, int64_t x_rows, const void* w,
                                     const float* w_scale, const int32_t* offsets, const int32_t* row_index,
                                     int32_t row_div, int64_t P, int64_t N, int64_t K, int32_t n_experts, void* y,
                                     int32_t y_dtype, void* stream, cider::WeightKind wk, bool gated) {
  const bool i4 = wk == cider::kWeightI4;
  constexpr int64_t kLimit = int64_t(1) << 31;
  if (!valid_dtype(y_dtype) || !gemm_sizes_ok(P, N) || !valid_k(K, i4 ? 32 : 16, 0)) return CIDER_ERROR_INVALID_VALUE;
  if (i4 && K > CIDER_MOE_MAX_K_PACKED) return CIDER_ERROR_INVALID_VALUE;   // their sums are of 16 * code
  if (x_rows < 0 || x_rows >= kLimit || row_div < 1 || n_experts < 1 || n_experts > CIDER_MOE_MAX_EXPERTS ||
      (gated && N % 2 != 0))
    return CIDER_ERROR_INVALID_VALUE;
  if (N * (i4 ? K / 2 : K) >= kLimit || (row_index ? x_rows * K >= kLimit : x_rows < P))
    return CIDER_ERROR_INVALID_VALUE;
  if (P == 0 || N == 0) return CIDER_SUCCESS;
  if (!w || !w_scale || !offsets || !y || (x_rows > 0 && (!x_q || !x_scale))) return CIDER_ERROR_INVALID_VALUE;
  if (!aligned16(x_q) || !aligned16(x_scale) || !aligned16(w) || !aligned16(w_scale) || !aligned16(offsets) ||
      !aligned16(row_index) || !aligned16(y))
    return CIDER_ERROR_INVALID_VALUE;
  const cider::GroupedArgs g{x_q, x_scale, w, w_scale, offsets, row_index, x_rows, P, N, K, row_div, n_experts, y};
  if (!cider::grouped_launch_fits(g, gated)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_grouped(g, wk, y_dtype == CIDER_DTYPE_BF16, gated, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_w8a8_grouped_gemm(const int8_t* x_q, const float* x_scale, int64_t x_rows, const int8_t* w_q,
                                       const float* w_scale, const int32_t* offsets, const int32_t* row_index,
                                       int32_t row_div, int64_t P, int64_t N, int64_t K, int32_t n_experts, void* y,
                                       int32_t y_dtype, void* stream) {
  return grouped_common(x_q, x_scale, x_rows, w_q, w_scale, offsets, row_index, row_div, P, N, K, n_experts, y,
                        y_dtype, stream, cider::kWeightI8, false);
}

cider_status_t cider_w4a8_grouped_gemm(const int8_t* x_q, const float* x_scale, int64_t x_rows,
                                       const uint8_t* w_packed, const float* w_scale, const int32_t* offsets,
                                       const int32_t* row_index, int32_t row_div, int64_t P, int64_t N, int64_t K,
                                       int32_t n_experts, void* y, int32_t y_dtype, void* stream) {
  return grouped_common(x_q, x_scale, x_rows, w_packed, w_scale, offsets, row_index, row_div, P, N, K, n_experts, y,
                        y_dtype, stream, cider::kWeightI4, false);
}

cider_status_t cider_w8a8_grouped_swiglu(const int8_t* x_q, const float* x_scale, int64_t x_rows, const int8_t* w_q,
                                         const float* w_scale, const int32_t* offsets, const int32_t* row_index,
                                         int32_t row_div, int64_t P, int64_t N, int64_t K, int32_t n_experts, void* y,
                                         int32_t y_dtype, void* stream) {
  return grouped_common(x_q, x_scale, x_rows, w_q, w_scale, offsets, row_index, row_div, P, N, K, n_experts, y,
                        y_dtype, stream, cider::kWeightI8, true);
}

cider_status_t cider_w4a8_grouped_swiglu(const int8_t* x_q, const float* x_scale, int64_t x_rows,
                                         const uint8_t* w_packed, const float* w_scale, const int32_t* offsets,
                                         const int32_t* row_index, int32_t row_div, int64_t P, int64_t N, int64_t K,
                                         int32_t n_experts, void* y, int32_t y_dtype, void* stream) {
  return grouped_common(x_q, x_scale, x_rows, w_packed, w_scale, offsets, row_index, row_div, P, N, K, n_experts, y,
                        y_dtype, stream, cider::kWeightI4, true);
}

cider_status_t cider_norm_quant(const cider_norm_quant_t* args, void* stream) {
  if (!args) return CIDER_ERROR_INVALID_VALUE;
  const cider_norm_quant_t& a = *args;
  // one workgroup of 256 threads per row: the grid stays below 2^31 threads
  if (!valid_dtype(a.dtype) || a.M < 0 || a.M >= (int64_t(1) << 23) || !valid_gs(a.group_size) ||
      !valid_k(a.K, 1, a.group_size))
    return CIDER_ERROR_INVALID_VALUE;
  if (!std::isfinite(a.alpha) || !std::isfinite(a.eps) || !(a.eps > 0.0f) || a.rows_per_gate < 0)
    return CIDER_ERROR_INVALID_VALUE;
  if ((a.slots != nullptr) != (a.weights != nullptr) || (a.x_q != nullptr) != (a.x_scale != nullptr))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.slots && (a.top_k < 1 || a.top_k > CIDER_MOE_MAX_TOP_K || a.block_rows < 0 ||
                  a.block_rows >= (int64_t(1) << 31)))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.M == 0) return CIDER_SUCCESS;
  if (a.block ? !a.h : (!a.x || a.slots || a.post_weight || a.gate)) return CIDER_ERROR_INVALID_VALUE;
  if ((a.x_q || a.normed) && !a.norm_weight) return CIDER_ERROR_INVALID_VALUE;
  if (!a.h && !a.x_q && !a.normed) return CIDER_ERROR_INVALID_VALUE;
  for (const void* p : {a.x, a.block, static_cast<const void*>(a.slots), static_cast<const void*>(a.weights),
                        a.post_weight, a.gate, a.norm_weight, static_cast<const void*>(a.h),
                        static_cast<const void*>(a.normed), static_cast<const void*>(a.x_q),
                        static_cast<const void*>(a.x_scale)})
    if (!aligned16(p)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  const cider::NormArgs n{a.x,      a.block,  a.slots,   a.weights, a.post_weight, a.gate,          a.norm_weight,
                          a.h,      a.normed, a.x_q,     a.x_scale, a.M,           a.K,             a.block_rows,
                          a.rows_per_gate,    a.top_k,   a.group_size, a.alpha,    a.eps};
  return from_hip(cider::launch_norm(n, a.dtype == CIDER_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_dequant_act(const int8_t* x_q, const float* x_scale, int64_t M, int64_t K, int32_t group_size,
                                 void* y, int32_t y_dtype, void* stream) {
  if (!valid_dtype(y_dtype)) return CIDER_ERROR_INVALID_VALUE;
  if (M < 0 || !valid_gs(group_size) || !valid_k(K, 1, group_size)) return CIDER_ERROR_INVALID_VALUE;
  if (M == 0) return CIDER_SUCCESS;
  if (!x_q || !x_scale || !y || !aligned16(x_q) || !aligned16(x_scale) || !aligned16(y))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_dequant_rows(x_q, x_scale, M, K, group_size, y, y_dtype == CIDER_DTYPE_BF16,
                                             static_cast<hipStream_t>(stream)));
}

// ---- attention blocks -------------------------------------------------------

static bool kv4_cache_ok(const cider_kv4_cache_t& c) {
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return false;
  const int32_t gs = c.group_size ? c.group_size : c.head_dim;
  if (gs < 32 || (gs != c.head_dim && 2 * gs != c.head_dim && 4 * gs != c.head_dim)) return false;
  if (c.page_size < 16 || c.page_size > CIDER_KV4_MAX_PAGE_SIZE || (c.page_size & (c.page_size - 1))) return false;
  if (c.kv_heads < 1 || c.kv_heads > CIDER_KV4_MAX_HEADS || c.n_pages < 1) return false;
  return c.n_pages < (int64_t(1) << 31) / c.page_size;   // slots are int32
}

static bool kv4_cache_there(const cider_kv4_cache_t& c) {
  return c.k_codes && c.k_scale && c.v_codes && c.v_scale && aligned16(c.k_codes) && aligned16(c.k_scale) &&
         aligned16(c.v_codes) && aligned16(c.v_scale);
}

static cider::Kv4Cache kv4_cache_of(const cider_kv4_cache_t& c) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return cider::Kv4Cache{c.k_codes,   c.k_scale, c.v_codes,  c.v_scale,  c.n_pages,
                         c.page_size, shift,     c.kv_heads, c.head_dim, c.group_size ? c.head_dim / c.group_size : 1};
}

// Strides of a [T, heads, D] array that is written: no two elements in one place.
static bool rows_apart(int64_t T, int64_t heads, int64_t D, int64_t row, int64_t head) {
  constexpr int64_t kMost = int64_t(1) << 40;
  if (row < 0 || head < 0 || row > kMost || head > kMost) return false;
  return ((heads == 1 || head >= D) && (T == 1 || row >= (heads - 1) * head + D)) ||
         ((T == 1 || row >= D) && (heads == 1 || head >= (T - 1) * row + D));
}

static bool strides_ok(int64_t row, int64_t head) {   // of an array that is read
  constexpr int64_t kMost = int64_t(1) << 40;
  return row >= 0 && head >= 0 && row <= kMost && head <= kMost;
}

cider_status_t cider_rope(const cider_rope_t* args, void* stream) {
  if (!args) return CIDER_ERROR_INVALID_VALUE;
  const cider_rope_t& a = *args;
  // one workgroup of 256 threads per token and slice of heads: the grid stays below 2^31 threads
  if (!valid_dtype(a.dtype) || a.T < 0 || a.T >= (int64_t(1) << 23) || a.heads < 0 || a.head_dim < 2 ||
      a.head_dim > CIDER_ROPE_MAX_HEAD_DIM || a.heads > CIDER_ROPE_MAX_HEADS)
    return CIDER_ERROR_INVALID_VALUE;
  if (a.rotary_dim < 2 || a.rotary_dim % 2 || a.rotary_dim > a.head_dim || a.rotary_dim > CIDER_ROPE_MAX_ROTARY_DIM ||
      (a.interleaved != 0 && a.interleaved != 1) || !std::isfinite(a.scale))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.T == 0 || a.heads == 0) return CIDER_SUCCESS;
  if (!a.x || !a.y || !a.positions || !a.inv_freq) return CIDER_ERROR_INVALID_VALUE;
  if (!strides_ok(a.x_row_stride, a.x_head_stride) ||
      !rows_apart(a.T, a.heads, a.head_dim, a.y_row_stride, a.y_head_stride) ||
      (a.x == a.y && (a.x_row_stride != a.y_row_stride || a.x_head_stride != a.y_head_stride)))
    return CIDER_ERROR_INVALID_VALUE;
  for (const void* p : {a.x, static_cast<const void*>(a.y), static_cast<const void*>(a.positions),
                        static_cast<const void*>(a.inv_freq)})
    if (!aligned16(p)) return CIDER_ERROR_INVALID_VALUE;
  const cider::RopeArgs r{a.x,      a.y,     a.positions, a.inv_freq, a.T,          a.x_row_stride, a.x_head_stride,
                          a.y_row_stride, a.y_head_stride, a.heads,   a.head_dim,   a.rotary_dim,   a.interleaved,
                          a.scale};
  if (!cider::rope_fits(r)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_rope(r, a.dtype == CIDER_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_kv4_append(const cider_kv4_append_t* args, void* stream) {
  if (!args) return CIDER_ERROR_INVALID_VALUE;
  const cider_kv4_append_t& a = *args;
  const cider_kv4_cache_t& c = a.cache;
  if (!kv4_cache_ok(c) || !valid_dtype(a.dtype) || a.T < 0 || a.T >= (int64_t(1) << 23) || a.q_heads < 0 ||
      a.q_heads > CIDER_KV4_MAX_Q_HEADS)
    return CIDER_ERROR_INVALID_VALUE;
  if (a.T == 0) return CIDER_SUCCESS;
  if ((a.q != nullptr) != (a.q_out != nullptr) || (a.q == nullptr && a.q_norm != nullptr) ||
      (a.positions != nullptr) != (a.inv_freq != nullptr))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.positions && (a.rotary_dim < 16 || a.rotary_dim % 16 || a.rotary_dim > c.head_dim ||
                      (a.interleaved != 0 && a.interleaved != 1) || !std::isfinite(a.rope_scale)))
    return CIDER_ERROR_INVALID_VALUE;
  if ((a.q_norm || a.k_norm) && (!std::isfinite(a.eps) || !(a.eps >= 0x1p-126f))) return CIDER_ERROR_INVALID_VALUE;
  if (!kv4_cache_there(c) || !a.k || !a.v || !a.slots || (a.q && a.q_heads < 1)) return CIDER_ERROR_INVALID_VALUE;
  for (const int64_t s : {a.q_row_stride, a.q_head_stride, a.k_row_stride, a.k_head_stride, a.v_row_stride,
                          a.v_head_stride, a.out_row_stride, a.out_head_stride})
    if (s % 8) return CIDER_ERROR_INVALID_VALUE;
  if (!strides_ok(a.k_row_stride, a.k_head_stride) || !strides_ok(a.v_row_stride, a.v_head_stride))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.q && (!strides_ok(a.q_row_stride, a.q_head_stride) ||
              !rows_apart(a.T, a.q_heads, c.head_dim, a.out_row_stride, a.out_head_stride) ||
              (a.q == a.q_out && (a.q_row_stride != a.out_row_stride || a.q_head_stride != a.out_head_stride))))
    return CIDER_ERROR_INVALID_VALUE;
  for (const void* p : {a.q, a.k, a.v, a.q_norm, a.k_norm, static_cast<const void*>(a.positions),
                        static_cast<const void*>(a.inv_freq), static_cast<const void*>(a.slots),
                        static_cast<const void*>(a.q_out)})
    if (!aligned16(p)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  const cider::Kv4AppendArgs k{kv4_cache_of(c), a.q, a.k, a.v, a.q_norm, a.k_norm, a.positions, a.inv_freq, a.slots,
                               a.q_out, a.T, a.q_row_stride, a.q_head_stride, a.k_row_stride, a.k_head_stride,
                               a.v_row_stride, a.v_head_stride, a.out_row_stride, a.out_head_stride,
                               a.q ? a.q_heads : 0, a.rotary_dim, a.interleaved, a.rope_scale, a.eps};
  return from_hip(cider::launch_kv4_append(k, a.dtype == CIDER_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

cider_status_t cider_kv4_read(const cider_kv4_cache_t* cache, const int32_t* slots, int64_t n, void* k, void* v,
                              int32_t dtype, void* stream) {
  if (!cache || !kv4_cache_ok(*cache) || !valid_dtype(dtype) || n < 0 || n >= (int64_t(1) << 31))
    return CIDER_ERROR_INVALID_VALUE;
  if (n == 0) return CIDER_SUCCESS;
  if (!kv4_cache_there(*cache) || !slots || !k || !v || !aligned16(slots) || !aligned16(k) || !aligned16(v))
    return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  return from_hip(cider::launch_kv4_read(kv4_cache_of(*cache), slots, n, k, v, dtype == CIDER_DTYPE_BF16,
                                         static_cast<hipStream_t>(stream)));
}

static bool kv4_attention_sizes_ok(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                   int64_t capacity) {
  // (tokens and positions are int32 with some steps of a loop past them, window and queries before them)
  constexpr int64_t kLimit = int64_t(1) << 31, kMost = int64_t(1) << 30;
  if (T < 0 || T > kMost || B < 1 || B >= kLimit || capacity < 0 || capacity > kMost || kv_heads < 1 ||
      kv_heads > CIDER_KV4_MAX_HEADS || q_heads < 1 || q_heads > CIDER_KV4_MAX_Q_HEADS || q_heads % kv_heads)
    return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
  return T == 0 || (T * q_heads <= kMost && cider::kv4_attention_fits(T, B, q_heads, kv_heads, head_dim, capacity));
}

int64_t cider_kv4_attention_workspace_size(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                           int64_t capacity) {
  if (!kv4_attention_sizes_ok(T, B, q_heads, kv_heads, head_dim, capacity)) return -1;
  return T == 0 ? 0 : cider::kv4_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, capacity);
}

cider_status_t cider_kv4_attention(const cider_kv4_attention_t* args, void* stream) {
  if (!args) return CIDER_ERROR_INVALID_VALUE;
  const cider_kv4_attention_t& a = *args;
  const cider_kv4_cache_t& c = a.cache;
  if (!kv4_cache_ok(c) || !valid_dtype(a.dtype) || a.max_pages < 0 || a.max_pages >= (int64_t(1) << 31))
    return CIDER_ERROR_INVALID_VALUE;
  const int64_t capacity = a.max_pages * c.page_size;
  if (!kv4_attention_sizes_ok(a.T, a.B, a.q_heads, c.kv_heads, c.head_dim, capacity)) return CIDER_ERROR_INVALID_VALUE;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || !std::isfinite(a.softmax_scale) ||
      (!a.query_offsets && a.T % a.B))
    return CIDER_ERROR_INVALID_VALUE;
  if (a.T == 0) return CIDER_SUCCESS;
  if (!kv4_cache_there(c) || !a.q || !a.y || !a.lengths || (a.max_pages && !a.page_table)) return CIDER_ERROR_INVALID_VALUE;
  if (!strides_ok(a.q_row_stride, a.q_head_stride) || a.q_row_stride % 8 || a.q_head_stride % 8)
    return CIDER_ERROR_INVALID_VALUE;
  for (const void* p : {a.q, static_cast<const void*>(a.page_table), static_cast<const void*>(a.lengths),
                        static_cast<const void*>(a.query_offsets), static_cast<const void*>(a.y),
                        static_cast<const void*>(a.workspace)})
    if (!aligned16(p)) return CIDER_ERROR_INVALID_VALUE;
  const int64_t need = cider::kv4_attention_workspace_bytes(a.T, a.B, a.q_heads, c.kv_heads, c.head_dim, capacity);
  if (need > 0 && (!a.workspace || a.workspace_bytes < need)) return CIDER_ERROR_INVALID_VALUE;
  if (!device_is_gfx950()) return CIDER_ERROR_NOT_SUPPORTED;
  // a window that reaches over the whole capacity hides nothing
  const cider::Kv4AttentionArgs k{kv4_cache_of(c), a.q, a.page_table, a.lengths, a.query_offsets, a.y,
                                  need > 0 ? static_cast<float*>(a.workspace) : nullptr, a.T, a.B, a.max_pages, a.q_row_stride,
                                  a.q_head_stride, a.q_heads, a.causal, a.window < capacity ? a.window : 0,
                                  a.softmax_scale};
  return from_hip(cider::launch_kv4_attention(k, a.dtype == CIDER_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
