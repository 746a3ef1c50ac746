// The boundary between two blocks of a decoder, and the way back from codes:
//
//   norm_rows_*      p = post_norm(block), h = x + alpha * gate * p,
//                    n = norm(h), then the int8 codes of n - one pass over
//                    the row instead of the five (combine, norm, add, norm,
//                    quantize) that the parts take
//   dequant_rows     codes and scales -> fp16 / bf16 rows
//
// Mathematics, per row (all in fp32):
//   p0 = block row, or sum_j weight_j * block[slot_j] (one fma per term, in
//        j order)
//   p  = p0 * (1 / sqrt(mean(p0^2) + eps)) * w_post       (with w_post)
//   h  = round(x + alpha * (gate * p))    to the rows' 16-bit type: the
//        residual stream is stored in it, and the norm below reads the
//        stored value, as a program that norms the residual later does
//   n  = (h * w) * (1 / sqrt(mean(h^2) + eps))
//   s  = max|n| / 127, codes = clamp(rint(n / s)) by cider_quant_rule.h;
//        n itself is not rounded to 16 bits before it is quantized.
// The max over |n| needs no pass of its own: rounding is monotone, so
// max|fl(t * r)| = fl(max|t| * r) with t = h * w, and max|t| is reduced
// together with the sum of h^2.
//
// HBM-bound: each of x and the block's rows is read once, h and the codes are
// written once. The row stays in registers from the first load to the codes.
// Kernel times (HIP events): 4096 rows of 2560 fp16 with both norms and a gate
// 16.6 us (73 MB, 4.4 TB/s), 4096 rows of 2048 bf16 each summing 8 expert rows
// 31.1 us (177 MB, 5.7 TB/s; six in seven of them reads, which a plain read
// stream takes at 6.2 and a copy at 5.1), one row 4.1 us (an empty launch takes
// 3.5). Rows that take norm_rows_loop are far from this (see there). Loads as
// address-space-1 vectors took these from 29.4 and 38.9 us to 17.8 and 37.1: the
// compiler had made flat one-dword loads of them; past-the-cache loads and stores
// did the rest (load16_once).
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rows.h"

namespace cider {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The same past the caches' retention, for what is read or written once here:
// a token's expert rows, and 16-bit rows whose reader comes a block later. The
// inputs then stay in the last-level cache: 4096 rows of 4096 with both norms
// 28.2 -> 21.4 us and, with the GEMM before it, 87.2 -> 83.5; expert rows
// 36 -> 31. Not for x, a block in place, or the codes, which the next or last
// launch also touches (codes: GEMM and norm of 4096 x 2560 45.4 -> 49.4).
__device__ __forceinline__ u4 load16_once(const void* base, int64_t c) {
  return __builtin_nontemporal_load((const global_u4*)base + c);
}
__device__ __forceinline__ void store16_once(void* base, int64_t c, u4 v) {
  __builtin_nontemporal_store(v, (global_u4*)base + c);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = __builtin_elementwise_maximum(v, __shfl_xor(v, off));
  return v;
}

// Sum (and max) over the row's lanes: a wave, or the row's WPR waves through
// `red` (2 * kWaves floats of its own for each call).
template <int WPR>
__device__ __forceinline__ void row_reduce(float& sum, float& mx, float* red, int wave, int lane) {
  sum = wave_sum(sum);
  mx = wave_max(mx);
  if constexpr (WPR > 1) {
    if (lane == 0) {
      red[wave] = sum;
      red[kWaves + wave] = mx;
    }
    __syncthreads();
    const int w0 = wave / WPR * WPR;
    sum = red[w0];
    mx = red[kWaves + w0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      sum += red[w0 + w];
      mx = __builtin_elementwise_maximum(mx, red[kWaves + w0 + w]);
    }
  }
}

// NaN for a row that is not finite or whose squares overflow: 1 / sqrt(inf)
// would turn its finite values into zeros. With it, and maxima that keep a NaN
// (v_maximum3_f32), every scale of the row is NaN, per row or per group.
__device__ __forceinline__ float inv_rms(float sum, int64_t K, float eps) {
  const float v = sum / (float)K + eps;
  return __builtin_isfinite(v) ? 1.0f / __builtin_sqrtf(v) : __builtin_nanf("");
}

// Rows of K % 8 == 0 that fit the registers of WPR waves (4 / WPR rows per
// workgroup): CPL 16-byte chunks per lane, chunk L + 64 * WPR * i, so that a
// wave's loads are contiguous and the 8 or 16 chunks of a scale group are
// neighbouring lanes.
template <int CPL, int WPR, bool BF>
__global__ void __launch_bounds__(kThreads) norm_rows_reg(const NormArgs a) {
  static_assert(WPR == 1 || WPR == 2 || WPR == kWaves, "rows per workgroup");
  __shared__ float red[2][2 * kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t row = (int64_t)blockIdx.x * (kWaves / WPR) + wave / WPR;
  if constexpr (WPR == 1) {
    if (row >= a.M) return;
  }
  // a workgroup's second row may not exist: its waves keep the barriers, as a
  // row of no chunks
  const int C0 = (int)(a.K / 8), C = row < a.M ? C0 : 0;
  if (row >= a.M) row = a.M - 1;
  constexpr int kStride = 64 * WPR;
  const int cl = (wave % WPR) * 64 + lane;

  // every load that depends on nothing goes out first
  const u4 z{0, 0, 0, 0};
  u4 xv[CPL], nw[CPL], pw[CPL], gv[CPL];
  const int64_t grow = a.gate && a.rows_per_gate ? row / a.rows_per_gate : 0;
#pragma unroll
  for (int i = 0; i < CPL; ++i) xv[i] = nw[i] = pw[i] = gv[i] = z;
  auto load_row = [&](u4 (&v)[CPL], const void* base, int64_t r) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = cl + kStride * i;
      if (c < C) v[i] = load16(base, r * C0 + c);
    }
  };
  if (a.x) load_row(xv, a.x, row);
  if (a.norm_weight) load_row(nw, a.norm_weight, 0);
  if (a.post_weight) load_row(pw, a.post_weight, 0);
  if (a.gate) load_row(gv, a.gate, grow);

  u4 hv[CPL];
  float sum = 0.0f, mx = 0.0f;
  if (a.block) {
    float p[CPL][8];
    if (a.slots) {
#pragma unroll
      for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[i][e] = 0.0f;
      constexpr int kAhead = CPL == 1 ? 8 : CPL == 2 ? 4 : 2;   // expert rows in flight
      for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
        u4 v[kAhead][CPL];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool in = j0 + j < a.top_k;
          const int64_t at = row * a.top_k + j0 + j;
          const int slot = in ? a.slots[at] : -1;
          const bool ok = slot >= 0 && slot < a.block_rows;
          w[j] = ok ? a.weights[at] : 0.0f;
#pragma unroll
          for (int i = 0; i < CPL; ++i) v[j][i] = z;
          if (ok) {
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
              const int c = cl + kStride * i;
              if (c < C) v[j][i] = load16_once(a.block, (int64_t)slot * C0 + c);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < CPL; ++i) {
            float t[8];
            unpack8<BF>(v[j][i], t);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] = __builtin_fmaf(w[j], t[e], p[i][e]);
          }
      }
    } else {
      u4 v[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) v[i] = z;
      load_row(v, a.block, row);
#pragma unroll
      for (int i = 0; i < CPL; ++i) unpack8<BF>(v[i], p[i]);
    }
    if (a.post_weight) {
      float s2 = 0.0f, unused = 0.0f;
#pragma unroll
      for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s2 = __builtin_fmaf(p[i][e], p[i][e], s2);
      row_reduce<WPR>(s2, unused, red[0], wave, lane);
      const float r = inv_rms(s2, a.K, a.eps);
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float w[8];
        unpack8<BF>(pw[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[i][e] = p[i][e] * r * w[e];
      }
    }
    if (a.gate) {
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float g[8];
        unpack8<BF>(gv[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[i][e] *= g[e];
      }
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      float x[8], h[8];
      unpack8<BF>(xv[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = __builtin_fmaf(a.alpha, p[i][e], x[e]);
      hv[i] = pack8<BF>(h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPL; ++i) hv[i] = xv[i];
  }
  if (a.h) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = cl + kStride * i;
      if (c < C) store16_once(a.h, row * C0 + c, hv[i]);
    }
  }
  if (!a.norm_weight) return;                    // uniform: the residual only

  float t[CPL][8];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    float h[8], w[8];
    unpack8<BF>(hv[i], h);
    unpack8<BF>(nw[i], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {                // chunks past the row are zeros
      sum = __builtin_fmaf(h[e], h[e], sum);
      t[i][e] = h[e] * w[e];
      mx = __builtin_elementwise_maximum(mx, __builtin_fabsf(t[i][e]));
    }
  }
  row_reduce<WPR>(sum, mx, red[1], wave, lane);
  const float r = inv_rms(sum, a.K, a.eps);
#pragma unroll
  for (int i = 0; i < CPL; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) t[i][e] *= r;
  if (a.normed) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = cl + kStride * i;
      if (c < C) store16_once(a.normed, row * C0 + c, pack8<BF>(t[i]));
    }
  }
  if (!a.x_q) return;
  const float row_s = mx * r / 127.0f;
  const int lpg = a.group_size / 8;              // lanes per scale group, 0: per row
  if (lpg == 0 && cl == 0 && C) a.x_scale[row] = row_s;
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = cl + kStride * i;
    float s = row_s;
    if (lpg) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, __builtin_fabsf(t[i][e]));
#pragma unroll
      for (int off = 4; off >= 1; off >>= 1) m = __builtin_elementwise_maximum(m, __shfl_xor(m, off));
      const float m16 = __builtin_elementwise_maximum(m, __shfl_xor(m, 8));
      s = (lpg == 16 ? m16 : m) / 127.0f;
      if ((lane & (lpg - 1)) == 0 && c < C) a.x_scale[row * (C0 / lpg) + c / lpg] = s;
    }
    if (c < C) {
      const uint2 q = s > 0.0f ? code_bytes_of_values<false>(t[i], s, 1.0f / s, 127.0f) : make_uint2(0, 0);
      *reinterpret_cast<uint2*>(a.x_q + row * a.K + (int64_t)c * 8) = q;
    }
  }
}

// Rows that fit no register path: K > 8192 (VEC = 8, 16-byte chunks), or K %
// 8 != 0 (VEC = 1, one element at a time; per-row scale). One workgroup per
// row, three passes over it: sum of p^2 (with a post-norm), then h, its sum of
// squares and max|h * w|, then the codes from h read back (each thread reads
// only what it wrote itself). The block's rows are read twice with a post-norm,
// and slots and weights again for every chunk. With both norms and a gate, 4096
// rows of 12288 fp16 take 105 us (352 MB, at the copy rate 69) and of 2047 43
// (11); summing 8 expert rows, 2048 rows of 12288 bf16 192 us (528 MB, at the read
// rate 85) and 4096 rows of 2047 169 (28).
template <int VEC, bool BF>
__global__ void __launch_bounds__(kThreads) norm_rows_loop(const NormArgs a) {
  __shared__ float red[2][2 * kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const int64_t K = a.K;
  const int64_t gate_at = a.gate && a.rows_per_gate ? row / a.rows_per_gate * K : 0;

  auto load = [&](const void* base, int64_t at, float (&v)[VEC]) {
    if constexpr (VEC == 8) unpack8<BF>(load16(base, at / 8), v);
    else v[0] = elem_to_float<BF>(static_cast<const uint16_t*>(base)[at]);
  };
  auto store = [&](void* base, int64_t at, const float (&v)[VEC]) {
    if constexpr (VEC == 8) store16(base, at / 8, pack8<BF>(v));
    else static_cast<uint16_t*>(base)[at] = round16<BF>(v[0]);
  };
  auto block_at = [&](int64_t k, float (&p)[VEC]) {
    if (!a.slots) {
      load(a.block, row * K + k, p);
      return;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[e] = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      const int slot = a.slots[row * a.top_k + j];
      if (slot < 0 || slot >= a.block_rows) continue;
      const float w = a.weights[row * a.top_k + j];
      float v[VEC];
      load(a.block, (int64_t)slot * K + k, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) p[e] = __builtin_fmaf(w, v[e], p[e]);
    }
  };

  float r1 = 1.0f;
  if (a.post_weight) {
    float s2 = 0.0f, unused = 0.0f;
    for (int64_t k = (int64_t)threadIdx.x * VEC; k < K; k += kThreads * VEC) {
      float p[VEC];
      block_at(k, p);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s2 = __builtin_fmaf(p[e], p[e], s2);
    }
    row_reduce<kWaves>(s2, unused, red[0], wave, lane);
    r1 = inv_rms(s2, K, a.eps);
  }

  float sum = 0.0f, mx = 0.0f;
  for (int64_t k = (int64_t)threadIdx.x * VEC; k < K; k += kThreads * VEC) {
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = 0.0f;
    if (a.x) load(a.x, row * K + k, h);
    if (a.block) {
      float p[VEC], w[VEC];
      block_at(k, p);
      if (a.post_weight) {
        load(a.post_weight, k, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = p[e] * r1 * w[e];
      }
      if (a.gate) {
        load(a.gate, gate_at + k, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = elem_to_float<BF>(round16<BF>(__builtin_fmaf(a.alpha, p[e], h[e])));
    }
    if (a.h) store(a.h, row * K + k, h);
    if (a.norm_weight) {
      float w[VEC];
      load(a.norm_weight, k, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum = __builtin_fmaf(h[e], h[e], sum);
        mx = __builtin_elementwise_maximum(mx, __builtin_fabsf(h[e] * w[e]));
      }
    }
  }
  if (!a.norm_weight) return;
  row_reduce<kWaves>(sum, mx, red[1], wave, lane);
  const float r = inv_rms(sum, K, a.eps);
  const float row_s = mx * r / 127.0f;
  const int lpg = a.group_size / 8;
  if (lpg == 0 && a.x_q && threadIdx.x == 0) a.x_scale[row] = row_s;
  const void* hsrc = a.h ? a.h : a.x;            // without a block the residual is x itself
  // every lane of a wave runs the same number of steps: the shuffles below
  // need all lanes of a group, and groups never straddle the row's end
  for (int64_t k0 = (int64_t)wave * 64 * VEC; k0 < K; k0 += kThreads * VEC) {
    const int64_t k = k0 + lane * VEC;
    const bool in = k < K;
    float t[VEC], w[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = 0.0f;
    if (in) {
      load(hsrc, row * K + k, t);
      load(a.norm_weight, k, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) t[e] = t[e] * w[e] * r;
      if (a.normed) store(a.normed, row * K + k, t);
    }
    if (!a.x_q) continue;
    float s = row_s;
    if constexpr (VEC == 8) {
      if (lpg) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) m = __builtin_elementwise_maximum(m, __builtin_fabsf(t[e]));
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) m = __builtin_elementwise_maximum(m, __shfl_xor(m, off));
        const float m16 = __builtin_elementwise_maximum(m, __shfl_xor(m, 8));
        s = (lpg == 16 ? m16 : m) / 127.0f;
        if (in && (lane & (lpg - 1)) == 0) a.x_scale[row * (K / a.group_size) + k / a.group_size] = s;
      }
      if (in)
        *reinterpret_cast<uint2*>(a.x_q + row * K + k) =
            s > 0.0f ? code_bytes_of_values<false>(t, s, 1.0f / s, 127.0f) : make_uint2(0, 0);
    } else {
      if (in) {
        float q = s > 0.0f ? __builtin_rintf(t[0] / s) : 0.0f;
        q = __builtin_fminf(__builtin_fmaxf(q, -127.0f), 127.0f);
        a.x_q[row * K + k] = (int8_t)q;
      }
    }
  }
}

template <bool BF>
hipError_t launch_norm_t(const NormArgs& a, hipStream_t st) {
  // Waves and chunks per row. Up to four rows per CU every row is resident at
  // once and its chain of latencies is the time: four waves, each with as few
  // chunks as possible (256 rows of K = 1024 summing 8 expert rows: one wave
  // of 2 chunks 6.4 us, four of 1 4.8; K = 2560 two of 3 8.8, four of 2 6.8;
  // one row 6.1 / 5.2), except up to K = 512, which one wave of 1 holds. With more
  // rows idle lanes cost: one wave up to K = 1024 (2048 rows 4.9 us, four waves
  // 5.3), four from there to K = 2048 (4096 rows of 2048 summing 8: 31.1 us, two
  // waves 33.0, one 36.6; of 1536 24.7, two 26.9, one of 3 chunks 24.5; at K = 1280
  // one of 3 is the faster, 21.3 to 22.0, and without expert rows 10.1 to 12.1),
  // two where four would leave most of their second chunks idle (4096 rows of
  // 2560 with both norms and a gate: 16.6 us, four waves 18.9, one 16.7).
  const dim3 block(kThreads);
  const unsigned rows1 = (unsigned)a.M, rows2 = (rows1 + 1) / 2, rows4 = (rows1 + 3) / 4;
  const int64_t C = a.K / 8;                     // 16-byte chunks per row
  const bool few = a.M <= 4 * 256;
  if (a.K % 8 != 0) norm_rows_loop<1, BF><<<dim3(rows1), block, 0, st>>>(a);
  else if (C <= 64) norm_rows_reg<1, 1, BF><<<dim3(rows4), block, 0, st>>>(a);
  else if (C <= 128 && !few) norm_rows_reg<2, 1, BF><<<dim3(rows4), block, 0, st>>>(a);
  else if (C <= 256) norm_rows_reg<1, kWaves, BF><<<dim3(rows1), block, 0, st>>>(a);
  else if (C <= 384 && !few) norm_rows_reg<3, 2, BF><<<dim3(rows2), block, 0, st>>>(a);
  else if (C <= 512) norm_rows_reg<2, kWaves, BF><<<dim3(rows1), block, 0, st>>>(a);
  else if (C <= 768) norm_rows_reg<3, kWaves, BF><<<dim3(rows1), block, 0, st>>>(a);
  else if (C <= 1024) norm_rows_reg<4, kWaves, BF><<<dim3(rows1), block, 0, st>>>(a);
  else norm_rows_loop<8, BF><<<dim3(rows1), block, 0, st>>>(a);
  return hipGetLastError();
}

// One code's value as a finished fp32 product (the empty asm keeps the backend
// from fusing it with the fp16 conversion into one rounding, which bf16 does
// not have: both types round the same fp32 value).
__device__ __forceinline__ float code_value(int8_t q, float s) {
  float v = (float)q * s;
  asm("" : "+v"(v));
  return v;
}

// y = fp(code * scale), 8 codes per thread when rows are whole 8-byte chunks
// (scale groups are multiples of 8), else one (4096 rows of 2048 4.6 us, of 2047
// 13.5).
template <int VEC, bool BF>
__global__ void __launch_bounds__(kThreads) dequant_rows(const int8_t* __restrict__ q, const float* __restrict__ s,
                                                         int64_t M, int K, int group_size, uint16_t* __restrict__ y) {
  const int per_row = K / VEC;
  const int64_t total = M * per_row;
  const int G = group_size ? K / group_size : 1;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per_row;
    const int c = (int)(i - row * per_row);
    const float sc = s[row * G + (group_size ? c * VEC / group_size : 0)];
    if constexpr (VEC == 8) {
      const uint2 v = reinterpret_cast<const uint2*>(q)[i];
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = code_value((int8_t)((e < 4 ? v.x : v.y) >> (8 * (e & 3))), sc);
      store16_once(y, i, pack8<BF>(t));
    } else {
      y[i] = round16<BF>(code_value(q[i], sc));
    }
  }
}

template <bool BF>
hipError_t launch_dequant_t(const int8_t* q, const float* s, int64_t M, int64_t K, int group_size, void* y,
                            hipStream_t st) {
  const bool vec = K % 8 == 0;
  const int64_t items = M * (vec ? K / 8 : K);
  const unsigned blocks = (unsigned)((items + kThreads - 1) / kThreads < 16384 ? (items + kThreads - 1) / kThreads : 16384);
  if (vec)
    dequant_rows<8, BF><<<dim3(blocks), dim3(kThreads), 0, st>>>(q, s, M, (int)K, group_size, static_cast<uint16_t*>(y));
  else
    dequant_rows<1, BF><<<dim3(blocks), dim3(kThreads), 0, st>>>(q, s, M, (int)K, group_size, static_cast<uint16_t*>(y));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_norm_t<true>(a, stream) : launch_norm_t<false>(a, stream);
}

hipError_t launch_dequant_rows(const int8_t* q, const float* s, int64_t M, int64_t K, int group_size, void* y,
                               bool bf16, hipStream_t stream) {
  return bf16 ? launch_dequant_t<true>(q, s, M, K, group_size, y, stream)
              : launch_dequant_t<false>(q, s, M, K, group_size, y, stream);
}

}  // namespace cider
