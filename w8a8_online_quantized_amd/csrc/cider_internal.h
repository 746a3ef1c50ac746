// Internal declarations shared by the HIP translation units of libcider.
// Nothing here is part of the public ABI (include/cider.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cider {

// Launches the activation / weight quantization kernel.
//   x: fp16 [R, K]; qmax 127 (int8 codes into q8 [R, K]) or 7 (packed int4
//   codes into q4 [R, K/2]); s: fp32 [R, G].
//   bf16: the rows are bfloat16 instead of fp16.
hipError_t launch_quant_rows(const void* x, int64_t R, int64_t K, int group_size, int qmax,
                             void* q, float* s, hipStream_t stream, bool bf16 = false);

// The same with percentile-clipped scales: s = t / qmax, t = the percentile
// (0..100) of the group's magnitudes (linear interpolation between order
// statistics, fp64, rounded to fp32). R * K / group size groups, one
// workgroup each.
hipError_t launch_quant_rows_clip(const void* x, int64_t R, int64_t K, int group_size, int qmax,
                                  double percentile, void* q, float* s, hipStream_t stream, bool bf16 = false);

// Epilogue kinds of the GEMM kernels. kEpiF16Tok: per-group weight scales
// [N, G] with per-token activation scales [M] (int8 weights, gs 64 / 128).
// kEpiF16Split: per-channel fp16 output whose columns go to up to 4 separate
// matrices (GemmArgs::split).
// kEpiF16Linear: the GEMV kernel takes fp16 activations and quantizes them
// itself (per token), then dequantizes as kEpiF16.
// kEpiBF16: as kEpiF16 with a bfloat16 output; kEpiBF16Tok: as kEpiF16Tok
// with a bfloat16 output; kEpiBF16Linear: as kEpiF16Linear with bfloat16
// activations and output; kEpiBF16Split: as kEpiF16Split with bfloat16
// output matrices.
enum Epilogue {
  kEpiF16 = 0, kEpiAccI32 = 1, kEpiF16Tok = 2, kEpiF16Split = 3, kEpiF16Linear = 4, kEpiBF16 = 5, kEpiBF16Tok = 6,
  kEpiBF16Linear = 7, kEpiBF16Split = 8
};

// Column split of a GEMM's output: columns [end[i-1], end[i]) (end[-1] = 0)
// go to y[i], a row-major fp16 (bf16 for kEpiBF16Split) matrix of
// end[i] - end[i-1] columns. Unused
// trailing parts repeat the last end and are never selected.
constexpr int kMaxSplitParts = 4;
struct OutSplit {
  _Float16* y[kMaxSplitParts];
  int end[kMaxSplitParts];
};

// Weight encodings of the GEMM kernels.
enum WeightKind { kWeightI8 = 0, kWeightI4 = 1 };

struct GemmArgs {
  const int8_t* a;   // activation codes [M, K]
  const float* sa;   // activation scales [M] or [M, G] ([M] for kEpiF16Tok)
  const void* w;     // weight codes [N, K] int8 or packed [N, K/2]
  const float* sw;   // weight scales [N] or [N, G]
  int64_t M, N, K;
  int group_size;    // 0, 64, 128
  void* y;           // fp16 [M, N]
  int32_t* acc;      // int32 [M, N] or [G, M, N] (accumulator test hook)
  void* ws = nullptr;     // split-K workspace (counters zero on entry), or null
  int64_t ws_bytes = 0;
  OutSplit split{};       // kEpiF16Split only
};

hipError_t launch_gemm(const GemmArgs& args, WeightKind wk, Epilogue epi, hipStream_t stream);

// True when the one-launch linear applies: per-channel, M <= 2, K a multiple
// of 16 (32 for int4 weights) and the activation codes fit the GEMV kernel's
// LDS staging. (From M = 3 on, the activation quantization that every block
// repeats costs more than the separate quantization launch it saves.)
bool linear_is_one_launch(int64_t M, int64_t K, int group_size, WeightKind wk);

// Workspace bytes the GEMM dispatch uses for split-K at this shape (0: none).
int64_t gemm_split_workspace_bytes(int64_t M, int64_t N, int64_t K, WeightKind wk, int group_size);

struct MvArgs {
  const void* x;     // fp16 activations [M, K], 1 <= M <= 4
  const int8_t* w;   // int8 weight codes [N, K]
  const float* sw;   // weight scales [N] or [N, K / group_size]
  int64_t M, N, K;
  int group_size;    // 0, 64, 128
  void* y;           // fp16 [M, N]
};

// Decode matrix-vector product (no activation quantization).
hipError_t launch_mv(const MvArgs& args, hipStream_t stream);

// One pass over bytes (a multiple of 16) of buf; sink receives nothing
// (written only for an impossible data pattern).
hipError_t launch_read_probe(const void* buf, int64_t bytes, int32_t* sink, hipStream_t stream);

// Products grouped by expert (int8 or packed int4 weights, per-channel).
struct GroupedArgs {
  const int8_t* a;          // activation codes [x_rows, K]
  const float* sa;          // activation scales [x_rows]
  const void* w;            // weight codes [E, N, K] int8 or packed [E, N, K/2]
  const float* sw;          // weight scales [E, N]
  const int32_t* offsets;   // [E + 1], device
  const int32_t* row_index; // [P], device, or null: output row p reads activation row row_index[p] / row_div (p)
  int64_t x_rows, P, N, K;
  int row_div, E;
  void* y;                  // [P, N], gated [P, N / 2]
  uint32_t div_mul = 0;     // row_div as a multiplication (launch_grouped sets it; 0: row_div is 1)
  int div_shift = 0;
};

// gated: weight rows 0 .. N/2 - 1 are gates, the others ups. grouped_launch_fits:
// whether the grid of the output's tiles stays below 2^31 threads.
bool grouped_launch_fits(const GroupedArgs& args, bool gated);
hipError_t launch_grouped(const GroupedArgs& args, WeightKind wk, bool bf16, bool gated, hipStream_t stream);

// The routing plan of P = T * top_k expert ids; ws holds moe_plan_workspace_bytes.
int64_t moe_plan_workspace_bytes(int64_t P, int E);
hipError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* rows, int32_t* slots,
                           void* ws, hipStream_t stream);

// The boundary between two blocks (null pointers leave a part out).
struct NormArgs {
  const void* x;            // residual [M, K]
  const void* block;        // block output [M, K], or expert rows [block_rows, K] with slots
  const int32_t* slots;     // [M, top_k]
  const float* weights;     // [M, top_k]
  const void* post_weight;  // [K]
  const void* gate;         // [ceil(M / rows_per_gate), K], [K] with rows_per_gate 0
  const void* norm_weight;  // [K]
  void* h;                  // [M, K]
  void* normed;             // [M, K]
  int8_t* x_q;              // [M, K]
  float* x_scale;           // [M] or [M, K / group_size]
  int64_t M, K, block_rows, rows_per_gate;
  int top_k, group_size;
  float alpha, eps;
};
hipError_t launch_norm(const NormArgs& args, bool bf16, hipStream_t stream);

// y [M, K] = codes [M, K] times their scales (group_size as for quantizing).
hipError_t launch_dequant_rows(const int8_t* q, const float* s, int64_t M, int64_t K, int group_size, void* y,
                               bool bf16, hipStream_t stream);

}  // namespace cider
