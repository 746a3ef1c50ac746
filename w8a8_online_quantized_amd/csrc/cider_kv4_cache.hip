// Writing keys and values into the 4-bit cache, and reading them back:
//
//   kv4_append_rows  per (token, head): x / sqrt(mean(x^2) + eps) * w (q and k,
//                    optional), the rotation (optional), then q to its 16-bit
//                    type, and k and v by the int4 rule of cider_quant_rule.h
//                    (s = max|.| / 7 per group of a head, codes
//                    clamp(rint(. / s))) into the token's slot
//   kv4_read_rows    the slots' codes times their scales -> 16-bit rows
//
// k is rounded to its 16-bit type before it is quantized, so that the codes are
// those of a rotated k that was stored in between. HBM-bound: every row is read
// once, q written once, and the codes are an eighth of what was read.
//
// D / 8 lanes hold one head, eight dimensions each; the sums of a norm and the
// maxima of the groups stay in those lanes. One workgroup takes one token's
// heads (256 * 8 / D of them at a time).
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rope.h"
#include "cider_rows.h"

namespace cider {
namespace {

constexpr int kThreads = 256;

// Byte of a v_codes row at which the codes of dimensions 8c .. 8c + 7 begin,
// and how they lie: pieces of `piece` codes (8, 4 or 2), D / 32 bytes apart.
struct VPlace {
  int byte, piece;
};
template <int LANES>
__device__ __forceinline__ VPlace v_place(int c, int groups) {
  constexpr int kUnit = LANES / 2;              // codes of a sixteenth of the row (D / 16)
  const int per = kUnit / groups;               // of one group
  const int gs = LANES * 8 / groups, g = 8 * c / gs, o = 8 * c - g * gs;
  const int u = o / per;
  return VPlace{(u * kUnit + g * per + o % per) / 2, groups == 1 || per >= 8 ? 8 : per};
}

template <int LANES, bool BF>
__global__ void __launch_bounds__(kThreads) kv4_append_rows(Kv4AppendArgs a) {
  constexpr int D = LANES * 8, kHeads = kThreads / LANES;
  __shared__ float2 turn[D / 2];
  const int64_t t = blockIdx.x;
  const int c = threadIdx.x % LANES;
  const int pairs = a.positions ? a.rotary_dim / 2 : 0;
  const int hkv = a.cache.kv_heads, rows = a.q_heads + 2 * hkv;
  const int row = blockIdx.y * kHeads + threadIdx.x / LANES;
  const bool real = row < rows;
  const bool is_q = row < a.q_heads, is_v = row >= a.q_heads + hkv;
  const int head = is_q ? row : is_v ? row - a.q_heads - hkv : row - a.q_heads;
  const uint16_t* x = static_cast<const uint16_t*>(is_q ? a.q : is_v ? a.v : a.k);
  const int64_t at = is_q   ? t * a.q_row_stride + head * a.q_head_stride
                     : is_v ? t * a.v_row_stride + head * a.v_head_stride
                            : t * a.k_row_stride + head * a.k_head_stride;
  u4 raw = u4{0, 0, 0, 0};
  if (real) raw = load16(x + at, c);
  if (pairs) {
    const int32_t pos = a.positions[t];
    for (int i = threadIdx.x; i < pairs; i += kThreads) turn[i] = rope_turn(pos, a.inv_freq[i], a.rope_scale);
    __syncthreads();
  }
  if (!real) return;                            // whole groups of LANES lanes
  float n[8];
  unpack8<BF>(raw, n);
  const void* norm = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
  if (norm) {
    float sum = 0.0f, w[8];
    unpack8<BF>(load16(norm, c), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(n[e], n[e], sum);
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
    const float r = 1.0f / __builtin_sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = n[e] * r * w[e];
  }
  if (pairs && !is_v) {
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * c + e < pairs) rope_pair(n[2 * e], n[2 * e + 1], turn[4 * c + e]);
    } else {
      const int step = pairs / 8;               // chunks from one end of a pair to the other
      const bool low = c < step, high = !low && c < 2 * step;
      const int lane = threadIdx.x % 64;
      const int other = low ? lane + step : high ? lane - step : lane;
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = __shfl(n[e], other);
      if (low || high) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 cs = turn[8 * (low ? c : c - step) + e];
          float u = low ? n[e] : m[e], w = low ? m[e] : n[e];
          rope_pair(u, w, cs);
          n[e] = low ? u : w;
        }
      }
    }
  }
  const u4 rounded = pack8<BF>(n);
  if (is_q) {
    store16(static_cast<uint16_t*>(a.q_out) + t * a.out_row_stride + head * a.out_head_stride, c, rounded);
    return;
  }
  const int32_t slot = a.slots[t];
  if (slot < 0 || slot >= a.cache.n_pages * a.cache.page_size) return;
  // the group's maximum as a 16-bit pattern: a NaN is above infinity, which is
  // above every finite value, and both leave a scale of NaN
  const int groups = a.cache.groups;
  uint32_t m = abs_max_bits(uint4{rounded.x, rounded.y, rounded.z, rounded.w});
  for (int off = 1; off < LANES / groups; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
  const bool finite = m < (BF ? 0x7F80u : 0x7C00u);
  const float s = finite ? elem_to_float<BF>(m) / 7.0f : __builtin_nanf("");
  uint32_t codes = 0x88888888u;                 // eight codes 0
  if (s > 0.0f) {
    const uint2 b = code_bytes_of_chunk<BF, false>(uint4{rounded.x, rounded.y, rounded.z, rounded.w}, s, 1.0f / s, 7.0f);
    // byte 2j and 2j + 1 -> byte j
    uint32_t lo = (b.x & 0x0F0F0F0Fu) ^ 0x08080808u, hi = (b.y & 0x0F0F0F0Fu) ^ 0x08080808u;
    lo |= lo >> 4;
    hi |= hi >> 4;
    codes = __builtin_amdgcn_perm(hi, lo, 0x06040200u);
  }
  const int64_t page = slot >> a.cache.page_shift;
  const int token = slot & (a.cache.page_size - 1);
  const int64_t ph = page * hkv + head;
  const int64_t base = (ph * a.cache.page_size + token) * (D / 2);
  const int lanes_per_group = LANES / groups;
  if (c % lanes_per_group == 0)
    (is_v ? a.cache.v_scale : a.cache.k_scale)[(ph * groups + c / lanes_per_group) * a.cache.page_size + token] = s;
  if (!is_v) {
    *reinterpret_cast<uint32_t*>(a.cache.k_codes + base + 4 * c) = codes;
    return;
  }
  const VPlace p = v_place<LANES>(c, groups);
  uint8_t* to = a.cache.v_codes + base + p.byte;
  if (p.piece == 8) {
    *reinterpret_cast<uint32_t*>(to) = codes;
  } else if (p.piece == 4) {
    *reinterpret_cast<uint16_t*>(to) = (uint16_t)codes;
    *reinterpret_cast<uint16_t*>(to + D / 32) = (uint16_t)(codes >> 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e * (D / 32)] = (uint8_t)(codes >> (8 * e));
  }
}

// One code's value as a finished fp32 product (both 16-bit types round it).
__device__ __forceinline__ float code_value(uint32_t nibble, float s) {
  float v = (float)((int)nibble - 8) * s;
  asm("" : "+v"(v));
  return v;
}

template <int LANES, bool BF>
__global__ void __launch_bounds__(kThreads) kv4_read_rows(Kv4Cache cache, const int32_t* __restrict__ slots, int64_t n,
                                                          uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int D = LANES * 8, kHeads = kThreads / LANES;
  const int hkv = cache.kv_heads;
  const int64_t rows = n * 2 * hkv;
  const int c = threadIdx.x % LANES;
  for (int64_t row = (int64_t)blockIdx.x * kHeads + threadIdx.x / LANES; row < rows; row += (int64_t)gridDim.x * kHeads) {
    const int64_t i = row / (2 * hkv);
    const int h2 = (int)(row - i * 2 * hkv);
    const bool is_v = h2 >= hkv;
    const int head = is_v ? h2 - hkv : h2;
    const int32_t slot = slots[i];
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = 0.0f;
    if (slot >= 0 && slot < cache.n_pages * cache.page_size) {
      const int64_t ph = (int64_t)(slot >> cache.page_shift) * hkv + head;
      const int token = slot & (cache.page_size - 1);
      const int64_t base = (ph * cache.page_size + token) * (D / 2);
      const float s = (is_v ? cache.v_scale : cache.k_scale)[(ph * cache.groups + c * cache.groups / LANES) *
                                                                 cache.page_size + token];
      uint32_t codes;
      if (!is_v) {
        codes = *reinterpret_cast<const uint32_t*>(cache.k_codes + base + 4 * c);
      } else {
        const VPlace p = v_place<LANES>(c, cache.groups);
        const uint8_t* from = cache.v_codes + base + p.byte;
        if (p.piece == 8) {
          codes = *reinterpret_cast<const uint32_t*>(from);
        } else if (p.piece == 4) {
          codes = *reinterpret_cast<const uint16_t*>(from) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(from + D / 32) << 16;
        } else {
          codes = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) codes |= (uint32_t)from[e * (D / 32)] << (8 * e);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = code_value((codes >> (4 * e)) & 15u, s);
    }
    store16((is_v ? v : k) + (i * hkv + head) * D, c, pack8<BF>(t));
  }
}

template <int LANES, bool BF>
void launch_append_t(const Kv4AppendArgs& a, hipStream_t st) {
  constexpr int kHeads = kThreads / LANES;
  const int rows = a.q_heads + 2 * a.cache.kv_heads;
  kv4_append_rows<LANES, BF><<<dim3((unsigned)a.T, (unsigned)((rows + kHeads - 1) / kHeads)), dim3(kThreads), 0, st>>>(a);
}

template <int LANES, bool BF>
void launch_read_t(const Kv4Cache& cache, const int32_t* slots, int64_t n, void* k, void* v, hipStream_t st) {
  constexpr int kHeads = kThreads / LANES;
  const int64_t blocks = (n * 2 * cache.kv_heads + kHeads - 1) / kHeads;
  kv4_read_rows<LANES, BF><<<dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(kThreads), 0, st>>>(
      cache, slots, n, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
}

}  // namespace

hipError_t launch_kv4_append(const Kv4AppendArgs& a, bool bf16, hipStream_t stream) {
  switch (a.cache.head_dim) {
    case 64: bf16 ? launch_append_t<8, true>(a, stream) : launch_append_t<8, false>(a, stream); break;
    case 128: bf16 ? launch_append_t<16, true>(a, stream) : launch_append_t<16, false>(a, stream); break;
    default: bf16 ? launch_append_t<32, true>(a, stream) : launch_append_t<32, false>(a, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache& cache, const int32_t* slots, int64_t n, void* k, void* v, bool bf16,
                           hipStream_t stream) {
  switch (cache.head_dim) {
    case 64: bf16 ? launch_read_t<8, true>(cache, slots, n, k, v, stream)
                  : launch_read_t<8, false>(cache, slots, n, k, v, stream); break;
    case 128: bf16 ? launch_read_t<16, true>(cache, slots, n, k, v, stream)
                   : launch_read_t<16, false>(cache, slots, n, k, v, stream); break;
    default: bf16 ? launch_read_t<32, true>(cache, slots, n, k, v, stream)
                  : launch_read_t<32, false>(cache, slots, n, k, v, stream); break;
  }
  return hipGetLastError();
}

}  // namespace cider
