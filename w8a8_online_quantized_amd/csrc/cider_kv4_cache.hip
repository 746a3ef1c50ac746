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
// those of a rotated k that was stored in between. Every row is read once, q
// written once, and the codes are a quarter of what was read. (16384 tokens, 16 heads
// of q, 8 of k and v of 128, norms and rotation: 54.7 us for 220 MB = 4.0 TB/s where a
// copy reaches 5.2: the vector units, busy throughout, bound it with HBM close behind;
// read back 22.2 us for 86 MB, bound by its 64-byte pieces of rows.)
//
// D / 8 lanes hold one head, eight dimensions each; the sums of a norm and the
// maxima of the groups stay in those lanes.
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rope.h"
#include "cider_rows.h"

#include <algorithm>

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

// Sums and maxima over aligned groups of 2 .. 32 lanes: within 16 by DPP (pairs,
// pairs of pairs, then mirrored halves, whose lanes hold the same by then).
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
template <class F>
__device__ __forceinline__ int over_lanes(int v, int lanes, F join) {
  v = join(v, dpp<0xB1>(v));                      // quad_perm 1 0 3 2
  if (lanes >= 4) v = join(v, dpp<0x4E>(v));      // quad_perm 2 3 0 1
  if (lanes >= 8) v = join(v, dpp<0x141>(v));     // row_half_mirror
  if (lanes >= 16) v = join(v, dpp<0x140>(v));    // row_mirror
  if (lanes >= 32) v = join(v, __shfl_xor(v, 16));
  return v;
}

// m / 7 correctly rounded, m a 16-bit value's magnitude: with y = fl(1 / 7) and q =
// fl(m y), the residual m - 7 q is exact and fl(q + residual y) is the rounded
// quotient (Markstein 1990), as long as nothing is subnormal; the division else.
__device__ __forceinline__ float seventh(float m) {
  constexpr float kSeventh = 1.0f / 7.0f;
  const float q = m * kSeventh;
  const float s = __builtin_fmaf(__builtin_fmaf(-7.0f, q, m), kSeventh, q);
  return m < 0x1p-100f ? m / 7.0f : s;
}

// Eight nibbles code + 8, the first lowest, by the rule of cider_quant_rule.h for
// qmax 7 (s > 0, min-max: no clamp can act). inv is the GPU's reciprocal, within one
// step of 1 / s, so r is within 7 * 4 * 2^-24 of fl(x / s) and decides the same
// integer unless it lies within 2^-13 of a half; those are divided. Adding 1.5 * 2^23
// + 8 rounds r to an even-tied integer and leaves code + 8 in the low bits; the
// patterns are added up shifted, and what their upper bits add is taken off.
__device__ __forceinline__ uint32_t nibbles_of_values(const float (&x)[8], float s) {
  constexpr float kMagic = 12582920.0f;   // 1.5 * 2^23 + 8
  const float inv = __builtin_amdgcn_rcpf(s);
  float t[8];
  float worst = __builtin_isfinite(inv) ? 0.0f : 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float r = x[e] * inv;
    t[e] = r + kMagic;
    worst = __builtin_fmaxf(worst, __builtin_fabsf((t[e] - kMagic) - r));
  }
  if (worst > kNearHalf) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      t[e] = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(x[e] / s), -7.0f), 7.0f) + kMagic;
  }
  uint32_t sum = __builtin_bit_cast(uint32_t, t[7]), upper = 0;
#pragma unroll
  for (int e = 6; e >= 0; --e) sum = (sum << 4) + __builtin_bit_cast(uint32_t, t[e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) upper += 0x4B400000u << (4 * e);
  return sum - upper;
}

// A wave has one token, or a slice of its heads: its lanes first form the cosines
// and sines, and each keeps those of its eight dimensions. Then 64 / LANES heads of
// q, of k or of v at a time, the next ones on their way while some are worked on.
template <int LANES, bool BF, bool PAST>
__global__ void __launch_bounds__(kThreads) kv4_append_rows(Kv4AppendArgs a) {
  constexpr int D = LANES * 8, kHeads = 64 / LANES;
  __shared__ float2 turns[kThreads / 64][D / 2];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / 64)), lane = threadIdx.x % 64, c = lane % LANES;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (t >= a.T) return;
  const int pairs = a.positions ? a.rotary_dim / 2 : 0;
  const int hkv = a.cache.kv_heads, groups = a.cache.groups;

  // steps of kHeads heads: q's, k's, then v's
  const int nq = (a.q_heads + kHeads - 1) / kHeads, nk = (hkv + kHeads - 1) / kHeads, steps = nq + 2 * nk;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_row_stride;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + t * a.k_row_stride;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + t * a.v_row_stride;
  auto fetch = [&](int i) {              // past the end the last head: no branch around the load
    // (every value by itself first: selected as members, the arguments would go through scratch)
    const uint16_t *pq = q, *pk = k, *pv = v;
    const int64_t sq = a.q_head_stride, sk = a.k_head_stride, sv = a.v_head_stride;
    const int hq = a.q_heads, hk = hkv;
    i = min(i, steps - 1);
    const bool is_q = i < nq, is_v = i >= nq + nk;
    const int head = min((is_q ? i : is_v ? i - nq - nk : i - nq) * kHeads + lane / LANES, (is_q ? hq : hk) - 1);
    return load16((is_q ? pq : is_v ? pv : pk) + head * (is_q ? sq : is_v ? sv : sk), c);
  };
  int i = blockIdx.y;
  u4 raw = fetch(i);
  const int32_t slot = a.slots[t];
  const u4 none = u4{0, 0, 0, 0};
  const u4 q_norm = a.q_norm ? load16(a.q_norm, c) : none, k_norm = a.k_norm ? load16(a.k_norm, c) : none;

  // half layout: dimension 8c + e is one end of pair 8c + e or 8 (c - step) + e;
  // interleaved: dimensions 8c + 2e and 8c + 2e + 1 are pair 4c + e
  const int step = pairs / 8;            // chunks from one end of a pair to the other
  const bool low = c < step, high = !low && c < 2 * step;
  float2 turn[8];
  if (pairs) {
    const int32_t pos = a.positions[t];
    for (int p = lane; p < pairs; p += 64) turns[wave][p] = rope_turn(pos, a.inv_freq[p], a.rope_scale);
    __builtin_amdgcn_wave_barrier();     // a wave's own: LDS keeps its order
    const int first = a.interleaved ? 4 * c : 8 * (low ? c : high ? c - step : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) turn[e] = turns[wave][min(first + e, D / 2 - 1)];
    if (!a.interleaved && low) {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn[e].y = -turn[e].y;
    }
  }
  const bool swap8 = LANES == 16 && 2 * step == LANES;   // the other end is 8 lanes away: a rotation of 16

  // a head of q or k: norm, rotation, and its 16-bit values
  auto turned = [&](u4 x, bool norm, u4 weight) __attribute__((always_inline)) {
    if (!norm && !pairs) return x;
    float n[8];
    unpack8<BF>(x, n);
    if (norm) {
      float sum = 0.0f, w[8];
      unpack8<BF>(weight, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(n[e], n[e], sum);
      sum = __builtin_bit_cast(float, over_lanes(__builtin_bit_cast(int, sum), LANES, [](int x, int y) {
        return __builtin_bit_cast(int, __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y));
      }));
      // 1 / sqrt: the GPU's (one step off at most; eps keeps it out of the subnormals)
      // and one step of Newton's method
      const float z = sum * (1.0f / D) + a.eps;
      float f = __builtin_amdgcn_rsqf(z);
      f = __builtin_isfinite(z) ? __builtin_fmaf(f * __builtin_fmaf(-z * f, f, 1.0f), 0.5f, f) : z - z;
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = n[e] * f * w[e];
    }
    if (pairs && a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * c + e < pairs) rope_pair(n[2 * e], n[2 * e + 1], turn[e]);
    } else if (pairs) {
      float m[8];
      if (swap8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = __builtin_bit_cast(float, dpp<0x128>(__builtin_bit_cast(int, n[e])));
      } else {
        const int other = low ? lane + step : high ? lane - step : lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = __shfl(n[e], other);
      }
      if (low || high) {
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = rope_end(n[e], m[e], turn[e].x, turn[e].y);
      }
    }
    return pack8<BF>(n);
  };

  // a head of k or v: its groups' scales, and eight codes of each lane
  const bool stored = slot >= 0 && slot < a.cache.n_pages * a.cache.page_size;
  const int64_t page = stored ? slot >> a.cache.page_shift : 0;
  const int token = stored ? slot & (a.cache.page_size - 1) : 0;
  const int lanes_per_group = LANES / groups;
  auto quantized = [&](u4 x, int head, float* scales) __attribute__((always_inline)) {
    // the group's maximum as a 16-bit pattern: a NaN is above infinity, which is
    // above every finite value, and both leave a scale of NaN
    const uint32_t m = over_lanes((int)abs_max_bits(uint4{x.x, x.y, x.z, x.w}), lanes_per_group,
                                  [](int x, int y) { return max(x, y); });
    const bool finite = m < (BF ? 0x7F80u : 0x7C00u);
    const float s = finite ? seventh(elem_to_float<BF>(m)) : __builtin_nanf("");
    uint32_t codes = 0x88888888u;        // eight codes 0
    if (s > 0.0f) {
      float n[8];
      unpack8<BF>(x, n);
      codes = nibbles_of_values(n, s);
    }
    if (head < hkv && c % lanes_per_group == 0)
      scales[((page * hkv + head) * groups + c / lanes_per_group) * a.cache.page_size + token] = s;
    return codes;
  };

  const VPlace place = v_place<LANES>(c, groups);
  for (; i < steps; i += gridDim.y) {
    const u4 x = raw;
    raw = fetch(i + gridDim.y);
    if (i < nq) {
      const int head = i * kHeads + lane / LANES;
      const u4 y = turned(x, a.q_norm != nullptr, q_norm);
      if (head < a.q_heads)
        store16_to<PAST>(static_cast<uint16_t*>(a.q_out) + t * a.out_row_stride + head * a.out_head_stride, c, y);
      continue;
    }
    if (!stored) continue;
    const bool is_v = i >= nq + nk;
    const int head = (is_v ? i - nq - nk : i - nq) * kHeads + lane / LANES;
    const int64_t base = ((page * hkv + head) * a.cache.page_size + token) * (D / 2);
    if (!is_v) {
      const uint32_t codes = quantized(turned(x, a.k_norm != nullptr, k_norm), head, a.cache.k_scale);
      if (head < hkv) *reinterpret_cast<uint32_t*>(a.cache.k_codes + base + 4 * c) = codes;
      continue;
    }
    const uint32_t codes = quantized(x, head, a.cache.v_scale);
    if (head >= hkv) continue;
    uint8_t* to = a.cache.v_codes + base + place.byte;
    if (place.piece == 8) {
      *reinterpret_cast<uint32_t*>(to) = codes;
    } else if (place.piece == 4) {
      *reinterpret_cast<uint16_t*>(to) = (uint16_t)codes;
      *reinterpret_cast<uint16_t*>(to + D / 32) = (uint16_t)(codes >> 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) to[e * (D / 32)] = (uint8_t)(codes >> (8 * e));
    }
  }
}

// One code's value as a finished fp32 product (both 16-bit types round it).
__device__ __forceinline__ float code_value(uint32_t nibble, float s) {
  float v = (float)((int)nibble - 8) * s;
  asm("" : "+v"(v));
  return v;
}

// A thread's next row is on its way while one is written.
template <int LANES, bool BF, bool PAST>
__global__ void __launch_bounds__(kThreads) kv4_read_rows(Kv4Cache cache, const int32_t* __restrict__ slots, int64_t n,
                                                          uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int D = LANES * 8, kHeads = kThreads / LANES;
  const int hkv = cache.kv_heads;
  const int64_t rows = n * 2 * hkv, stride = (int64_t)gridDim.x * kHeads;
  const int c = threadIdx.x % LANES;
  const VPlace p = v_place<LANES>(c, cache.groups);
  struct Row {
    int64_t to;                          // row of k or v
    bool is_v, there;
    uint32_t codes;
    float s;
  };
  auto fetch = [&](int64_t row) {
    Row r{0, false, false, 0x88888888u, 0.0f};
    if (row >= rows) return r;
    const int64_t i = row / (2 * hkv);
    const int h2 = (int)(row - i * 2 * hkv);
    r.is_v = h2 >= hkv;
    const int head = r.is_v ? h2 - hkv : h2;
    r.to = i * hkv + head;
    const int32_t slot = slots[i];
    r.there = slot >= 0 && slot < cache.n_pages * cache.page_size;
    if (!r.there) return r;
    const int64_t ph = (int64_t)(slot >> cache.page_shift) * hkv + head;
    const int token = slot & (cache.page_size - 1);
    const int64_t base = (ph * cache.page_size + token) * (D / 2);
    r.s = (r.is_v ? cache.v_scale : cache.k_scale)[(ph * cache.groups + c * cache.groups / LANES) * cache.page_size + token];
    if (!r.is_v) {
      r.codes = *reinterpret_cast<const uint32_t*>(cache.k_codes + base + 4 * c);
    } else {
      const uint8_t* from = cache.v_codes + base + p.byte;
      if (p.piece == 8) {
        r.codes = *reinterpret_cast<const uint32_t*>(from);
      } else if (p.piece == 4) {
        r.codes = *reinterpret_cast<const uint16_t*>(from) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(from + D / 32) << 16;
      } else {
        r.codes = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) r.codes |= (uint32_t)from[e * (D / 32)] << (8 * e);
      }
    }
    return r;
  };
  int64_t row = (int64_t)blockIdx.x * kHeads + threadIdx.x / LANES;
  Row cur = fetch(row);
  for (; row < rows; row += stride) {
    const Row next = fetch(row + stride);
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = cur.there ? code_value((cur.codes >> (4 * e)) & 15u, cur.s) : 0.0f;
    store16_to<PAST>((cur.is_v ? v : k) + cur.to * D, c, pack8<BF>(t));
    cur = next;
  }
}

template <int LANES, bool BF>
void launch_append_t(const Kv4AppendArgs& a, hipStream_t st) {
  constexpr int kHeads = 64 / LANES, kTok = kThreads / 64;
  const int steps = (a.q_heads + kHeads - 1) / kHeads + 2 * ((a.cache.kv_heads + kHeads - 1) / kHeads);
  // slices of a token's heads until there are waves for the whole GPU
  const int64_t slices = std::min<int64_t>(steps, std::max<int64_t>(1, 4096 / a.T));
  const dim3 grid((unsigned)((a.T + kTok - 1) / kTok), (unsigned)slices), block(kThreads);
  if (2 * a.T * a.q_heads * a.cache.head_dim >= kPastCacheBytes) kv4_append_rows<LANES, BF, true><<<grid, block, 0, st>>>(a);
  else kv4_append_rows<LANES, BF, false><<<grid, block, 0, st>>>(a);
}

template <int LANES, bool BF>
void launch_read_t(const Kv4Cache& cache, const int32_t* slots, int64_t n, void* k, void* v, hipStream_t st) {
  constexpr int kHeads = kThreads / LANES;
  const int64_t blocks = (n * 2 * cache.kv_heads + kHeads - 1) / kHeads;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 2048)), block(kThreads);
  uint16_t *to_k = static_cast<uint16_t*>(k), *to_v = static_cast<uint16_t*>(v);
  if (4 * n * cache.kv_heads * cache.head_dim >= kPastCacheBytes)
    kv4_read_rows<LANES, BF, true><<<grid, block, 0, st>>>(cache, slots, n, to_k, to_v);
  else
    kv4_read_rows<LANES, BF, false><<<grid, block, 0, st>>>(cache, slots, n, to_k, to_v);
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
