// Attention over the paged 4-bit cache (cider_kv4.h):
//
//   o = sum_t softmax_t(scale * q . k_t) v_t,  k_t = s_k (c - 8), v_t = s_v (c' - 8)
//
// over the tokens t that the row sees: t < length, with causal t <= p, with a
// window t > p - window, for a query at position p = length - n + i. Rows that
// see nothing are zeros.
//
// A "row" is one (query token, query head); the rows of one key/value head's
// query heads are packed token by token into tiles of 16, so that a group of
// heads shares each read of the cache. One wave holds NQ such tiles and walks
// the tokens 32 at a time with both operands straight from global memory to
// registers: the codes are an eighth of a 16-bit cache's bytes, so nothing is
// gained by staging them. Per 32 tokens:
//   S^T = K Q^T  v_mfma_f32_16x16x32, tokens as rows. A nibble n becomes an operand
//        by a mask and an or: the fp16 pattern 0x5400 | n << 4 is 64 + n, the bf16
//        pattern 0x4300 | n is 128 + n. The sums start at -72 * sum(q) (-136 *
//        sum(q)), so taking n to n - 8 costs nothing, and s_k scales the finished
//        fp32 sums. (fp16 denormals, n * 2^-24, would need no or, but the matrix
//        core aligns products by their exponent fields: sums of them lose ten bits.)
//   p = 2^(S - m): four tokens of one query per lane and sub-tile, which is the
//        layout in which the next product reads them. p * s_v is rounded to fp16
//        (both types: 2^-11 relative, where bf16 would leave 2^-8); s_v is taken
//        relative to a power of two that follows the largest one seen, so that
//        scales of any size fit.
//   O^T += V^T P^T  v_mfma_f32_16x16x32_f16, 16 dimensions as rows: a lane reads its
//        sixteenth of eight tokens' rows, and two v_perm and a few masks turn the
//        words into operands 64 + n. A product with a constant 72 sums what is too much.
// m is raised only when a score passes it by 2^8 (the accumulators are rescaled
// then), so most steps exchange nothing between lanes.
//
// SPLIT: the four waves of a workgroup share one tile of rows and take the
// tokens in turn; otherwise each wave has rows of its own. Either way the
// tokens are also split over workgroups when there are few rows; their partial
// results are joined by a second launch.
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rows.h"

#include <algorithm>

namespace cider {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTokens = 32;            // per step of a wave
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -3.402823466e38f;
constexpr float kRaise = 8.0f;         // log2: p stays below 2^8

typedef float f4 __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ f4 mfma_qk(u4 a, u4 b, f4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma_pv(u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

typedef __attribute__((address_space(1))) const uint8_t gbyte;

template <typename T>
__device__ __forceinline__ T gload(gbyte* p) { return *(__attribute__((address_space(1))) const T*)p; }

// ---- which rows and tokens a workgroup has ------------------------------------

// Token range of one tile of rows, and how many workgroups share it.
struct Share {
  int begin, end;      // tokens [begin, end) that any of its rows sees
  int steps;           // of kTokens, from begin rounded down
  int per, parts;      // steps of one part
};

struct Sequence {
  int64_t q0;          // first query row
  int n, length;       // queries, tokens in the cache
};

__device__ __forceinline__ int clamp_length(const Kv4AttentionArgs& a, int64_t b) {
  const int64_t cap = a.max_pages << a.cache.page_shift;
  const int len = a.lengths[b];
  return len < 0 ? 0 : len > cap ? (int)cap : len;
}

__device__ __forceinline__ Sequence sequence(const Kv4AttentionArgs& a, int64_t b) {
  Sequence s;
  if (a.query_offsets) {
    const int lo = a.query_offsets[b], hi = a.query_offsets[b + 1], most = (int)a.T;
    const int first = lo < 0 ? 0 : lo > most ? most : lo;
    const int last = hi < first ? first : hi > most ? most : hi;
    s.q0 = first;
    s.n = last - first;
  } else {
    s.n = (int)(a.T / a.B);
    s.q0 = b * s.n;
  }
  s.length = clamp_length(a, b);
  return s;
}

// tok_lo, tok_hi: the first and the last query token of the tile.
__device__ __forceinline__ Share share(const Kv4AttentionArgs& a, const Sequence& s, int tok_lo, int tok_hi, int parts,
                                       int least) {
  Share r;
  const int p_lo = s.length - s.n + tok_lo, p_hi = s.length - s.n + tok_hi;
  r.end = a.causal ? min(s.length, p_hi + 1) : s.length;
  r.begin = a.window ? max(0, p_lo - a.window + 1) : 0;
  r.steps = r.end > r.begin ? (r.end - (r.begin & ~(kTokens - 1)) + kTokens - 1) / kTokens : 0;
  r.parts = min(parts, max(1, (r.steps + least - 1) / least));
  r.per = max(1, (r.steps + r.parts - 1) / r.parts);
  r.parts = max(1, (r.steps + r.per - 1) / r.per);
  return r;
}

// The launch: how rows are tiled and tokens split (the same on both sides).
struct Plan {
  int rows;            // of a workgroup's tile
  int parts, least;    // most workgroups per tile, fewest steps of one
  int64_t slots;       // tiles over all sequences, at most
  int64_t tiles_per;   // without query_offsets: tiles of each sequence
};

// ---- the operands ---------------------------------------------------------------

// 8 nibbles of a word as an operand: elements in the order 0 4 1 5 2 6 3 7.
template <bool BF>
__device__ __forceinline__ u4 k_operand(uint32_t w) {
  if constexpr (BF) {
    constexpr uint32_t kMask = 0x000F000Fu, kOne = 0x43004300u;      // 128 + n
    return u4{(w & kMask) | kOne, ((w >> 4) & kMask) | kOne, ((w >> 8) & kMask) | kOne, ((w >> 12) & kMask) | kOne};
  } else {
    constexpr uint32_t kMask = 0x00F000F0u, kOne = 0x54005400u;      // 64 + n
    return u4{((w << 4) & kMask) | kOne, (w & kMask) | kOne, ((w >> 4) & kMask) | kOne, ((w >> 8) & kMask) | kOne};
  }
}
// 16-bit elements 0 .. 7 in that order.
__device__ __forceinline__ u4 k_order(u4 q) {
  return u4{__builtin_amdgcn_perm(q.z, q.x, 0x05040100u), __builtin_amdgcn_perm(q.z, q.x, 0x07060302u),
            __builtin_amdgcn_perm(q.w, q.y, 0x05040100u), __builtin_amdgcn_perm(q.w, q.y, 0x07060302u)};
}

template <int D, int G>
struct Raw {                            // 32 tokens as loaded
  static constexpr int kVW = D / 128 ? D / 128 : 1;   // words of a sixteenth of a V row
  uint32_t k[2][D / 32];
  uint32_t v[8][kVW];
  f4 ks[2][G], vs[2][G];
};

template <int D, int G, bool BF, int NQ, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2) kv4_attention(Kv4AttentionArgs a, Plan plan) {
  constexpr int kTiles = D / 16;        // output tiles of 16 dimensions; also the codes of a sixteenth
  constexpr int kPer = kTiles / G;      // of one group
  constexpr int kSteps = D / 32;        // products of one score
  constexpr int kRowsW = 16 * NQ;       // rows of a wave
  constexpr int kPitch = D + 4;
  __shared__ float shared_o[SPLIT ? kWaves * 16 * NQ * kPitch : 1];
  __shared__ float shared_m[SPLIT ? kWaves * 16 * NQ : 1], shared_l[SPLIT ? kWaves * 16 * NQ : 1];

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int l16 = lane & 15, kb = lane >> 4;
  const int hkv = a.cache.kv_heads, heads = a.q_heads / hkv;

  // ---- the workgroup's tile
  const int h = blockIdx.x % hkv;
  const int64_t rest = blockIdx.x / hkv;
  const int part = (int)(rest % plan.parts);
  const int64_t slot = plan.slots - 1 - rest / plan.parts;      // late tiles see the most tokens: they go first
  int64_t b = 0;
  int tile = 0;
  if (a.query_offsets) {
    // tiles before each sequence, 64 sequences at a time; every wave alike
    int64_t before = 0;
    bool found = false;
    for (int64_t b0 = 0; b0 < a.B && !found; b0 += 64) {
      int count = 0;
      if (b0 + lane < a.B) count = (int)(((int64_t)sequence(a, b0 + lane).n * heads + plan.rows - 1) / plan.rows);
      int sum = count;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(sum, off);
        if (lane >= off) sum += up;
      }
      const uint64_t hit = __ballot(before + sum > slot);
      if (hit) {
        const int first = __builtin_ctzll(hit);
        b = b0 + first;
        tile = (int)(slot - before) - (__shfl(sum, first) - __shfl(count, first));
        found = true;
      }
      before += __shfl(sum, 63);
    }
    if (!found) return;
    b = uniform((int)b);
    tile = uniform(tile);
  } else {
    b = slot / plan.tiles_per;
    tile = (int)(slot - b * plan.tiles_per);
  }
  const Sequence seq = sequence(a, b);
  const int rows = seq.n * heads;       // of this sequence and key/value head
  const int row0 = tile * plan.rows;
  const Share sh = share(a, seq, row0 / heads, (min(rows, row0 + plan.rows) - 1) / heads, plan.parts, plan.least);
  if (part >= sh.parts) return;
  const int step_end = min(sh.steps, (part + 1) * sh.per);
  const int first_token = sh.begin & ~(kTokens - 1);

  // ---- the wave's rows
  const int wrow0 = row0 + (SPLIT ? 0 : wave * kRowsW);
  int64_t q_row[NQ];                    // row of y (and of the partial results), -1 behind the last one
  int see_lo[NQ], see_hi[NQ];
  u4 qf[NQ][kSteps];
  f4 q_off[NQ][G];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int r = wrow0 + 16 * i + l16;
    const bool real = r < rows;
    const int rr = real ? r : rows - 1;
    const int tok = rr / heads, head = h * heads + rr - tok * heads;
    const int pos = seq.length - seq.n + tok;
    q_row[i] = real ? (seq.q0 + tok) * a.q_heads + head : -1;
    see_hi[i] = a.causal ? min(seq.length, pos + 1) : seq.length;
    see_lo[i] = a.window ? max(0, pos - a.window + 1) : 0;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (seq.q0 + tok) * a.q_row_stride + head * a.q_head_stride;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.0f;
#pragma unroll
      for (int st = 0; st < kSteps / G; ++st) {
        const u4 w = load16(q + g * (D / G) + kb * (D / G / 4) + st * 8, 0);
        float t[8];
        unpack8<BF>(w, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += t[e];
        qf[i][g * (kSteps / G) + st] = k_order(w);
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      const float off = sum * (BF ? -136.0f : -72.0f);
      q_off[i][g] = f4{off, off, off, off};
    }
  }
  // tokens that every row of the wave sees, and that some row sees (uniform)
  int all_lo = 0, all_hi = 0, any_hi = 0, any_lo = 0;
  {
    const int last = min(wrow0 + kRowsW, rows) - 1;
    const int p0 = seq.length - seq.n + wrow0 / heads, p1 = seq.length - seq.n + max(last, 0) / heads;
    all_hi = a.causal ? min(seq.length, p0 + 1) : seq.length;
    any_hi = a.causal ? min(seq.length, p1 + 1) : seq.length;
    all_lo = a.window ? max(0, p1 - a.window + 1) : 0;
    any_lo = a.window ? max(0, p0 - a.window + 1) : 0;
    if (last < wrow0) any_hi = 0;       // a wave behind the last row
  }

  f4 o[NQ][kTiles], z[NQ][G];
  float m[NQ], l[NQ];
  float ref = 0x1p-126f, inv_ref = 0x1p126f;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    m[i] = kLeast;
    l[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[i][j] = f4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < G; ++g) z[i][g] = f4{0, 0, 0, 0};
  }

  const float scale = a.softmax_scale * kLog2e;
  const int32_t* table = a.page_table + b * a.max_pages;
  const int page_size = a.cache.page_size, page_shift = a.cache.page_shift;

  // The pages of 64 sub-tiles of 16 tokens from the wave's step `first` on (a
  // lane each, -1 where there is nothing to read), so that the steps' loads wait
  // for no table entry.
  constexpr int kStride = SPLIT ? kWaves : 1;
  auto pages_from = [&](int first) {
    const int t = first_token + (first + (lane >> 1) * kStride) * kTokens + (lane & 1) * 16;
    int p = -1;
    if (t < any_hi) {
      p = table[t >> page_shift];
      if (p < 0 || p >= a.cache.n_pages) p = -1;
    }
    return p;
  };
  using R = Raw<D, G>;
  auto load = [&](int t, const int (&pages)[2], R& r) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool there = pages[s] >= 0;
      const int at = there ? (t + 16 * s) & (page_size - 1) : 0;
      const int64_t ph = (int64_t)(there ? pages[s] : 0) * hkv + h;
      const int64_t base = (ph * page_size + at) * (D / 2);
      gbyte* k = (gbyte*)a.cache.k_codes + base + l16 * (D / 2) + kb * (D / G / 8);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        gbyte* kg = k + g * (D / G / 2);
        constexpr int kW = kSteps / G;
        if constexpr (kW % 4 == 0) {
#pragma unroll
          for (int i = 0; i < kW / 4; ++i) {
            const u4 w = gload<u4>(kg + 16 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.k[s][g * kW + 4 * i + e] = w[e];
          }
        } else if constexpr (kW == 2) {
          typedef uint32_t u2 __attribute__((ext_vector_type(2)));
          const u2 w = gload<u2>(kg);
          r.k[s][g * kW] = w.x;
          r.k[s][g * kW + 1] = w.y;
        } else {
          r.k[s][g] = gload<uint32_t>(kg);
        }
      }
      gbyte* v = (gbyte*)a.cache.v_codes + base + 4 * kb * (D / 2) + l16 * (D / 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gbyte* vi = v + i * (D / 2);
        if constexpr (D == 64) r.v[4 * s + i][0] = gload<uint16_t>(vi);
        else if constexpr (D == 128) r.v[4 * s + i][0] = gload<uint32_t>(vi);
        else {
          typedef uint32_t u2 __attribute__((ext_vector_type(2)));
          const u2 w = gload<u2>(vi);
          r.v[4 * s + i][0] = w.x;
          r.v[4 * s + i][1] = w.y;
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int64_t so = ((ph * G + g) * page_size + at + 4 * kb) * 4;
        r.ks[s][g] = gload<f4>((gbyte*)a.cache.k_scale + so);
        r.vs[s][g] = gload<f4>((gbyte*)a.cache.v_scale + so);
      }
    }
  };

  auto process = [&](int t, const int (&pages)[2], const R& r) {
    // scores, in units of log2
    float x[NQ][8];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        f4 acc[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) acc[i] = q_off[i][g];
#pragma unroll
        for (int st = 0; st < kSteps / G; ++st) {
          const u4 k = k_operand<BF>(r.k[s][g * (kSteps / G) + st]);
#pragma unroll
          for (int i = 0; i < NQ; ++i) acc[i] = mfma_qk<BF>(k, qf[i][g * (kSteps / G) + st], acc[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ks = r.ks[s][g][e] * scale;
#pragma unroll
          for (int i = 0; i < NQ; ++i)
            x[i][4 * s + e] = g == 0 ? acc[i][e] * ks : __builtin_fmaf(acc[i][e], ks, x[i][4 * s + e]);
        }
      }
    }
    float vs[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) vs[g][e] = r.vs[e >> 2][g][e & 3];
    // tokens that not every row sees
    const bool masked = t < all_lo || t + kTokens > all_hi || pages[0] < 0 || pages[1] < 0;
    if (masked) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int tok = t + 16 * (e >> 2) + 4 * kb + (e & 3);
        const bool there = pages[e >> 2] >= 0;
        const bool some = there && tok >= any_lo && tok < any_hi;
#pragma unroll
        for (int g = 0; g < G; ++g) vs[g][e] = some ? vs[g][e] : 0.0f;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          x[i][e] = there && tok >= see_lo[i] && tok < see_hi[i] ? x[i][e] : -__builtin_inff();
      }
    }
    // a larger scale of V than all before: the accumulators are in units of ref
    float top = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = __builtin_fmaxf(top, __builtin_fabsf(vs[g][e]));
    if (__any(top > ref)) {
      for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
      uint32_t bits = (__builtin_bit_cast(uint32_t, top) & 0x7F800000u) + 0x00800000u;   // the next power of two
      bits = min(bits, 0x7E800000u);
      const float to = __builtin_bit_cast(float, bits);
      inv_ref = __builtin_bit_cast(float, 0x7F000000u - bits);
      const float f = ref * inv_ref;
      ref = to;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[i][j] *= f;
#pragma unroll
        for (int g = 0; g < G; ++g) z[i][g] *= f;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) vs[g][e] *= inv_ref;

    u4 pf[NQ][G];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float most = x[i][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) most = __builtin_fmaxf(most, x[i][e]);
      if (__any(most > m[i] + kRaise)) {
        most = __builtin_fmaxf(most, __shfl_xor(most, 16));
        most = __builtin_fmaxf(most, __shfl_xor(most, 32));
        const float to = __builtin_fmaxf(m[i], most);
        const float f = __builtin_amdgcn_exp2f(m[i] - to);
        m[i] = to;
        l[i] *= f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[i][j] *= f;
#pragma unroll
        for (int g = 0; g < G; ++g) z[i][g] *= f;
      }
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[i][e] - m[i]);
        l[i] += p[e];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        f8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = p[e] * vs[g][e];
        if (masked) {                   // a hidden token's scale may be anything
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = x[i][e] == -__builtin_inff() ? 0.0f : w[e];
        }
        pf[i][g] = __builtin_bit_cast(u4, __builtin_convertvector(w, h8));
      }
    }
    // O^T += V^T P^T
    const u4 seventy_two = u4{0x54805480u, 0x54805480u, 0x54805480u, 0x54805480u};
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int g = 0; g < G; ++g) z[i][g] = mfma_pv(seventy_two, pf[i][g], z[i][g]);
    constexpr int kHalves = D == 64 ? 1 : D / 64;   // 16-bit columns of a sixteenth: 4 codes each
#pragma unroll
    for (int c = 0; c < kHalves; ++c) {
      u4 w;
#pragma unroll
      for (int pr = 0; pr < 4; ++pr) {
        const uint32_t lo = r.v[2 * pr][c / 2], hi = r.v[2 * pr + 1][c / 2];
        w[pr] = __builtin_amdgcn_perm(hi, lo, c % 2 ? 0x07060302u : 0x05040100u);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = 4 * c + n;
        const u4 v = ((n == 0 ? w << 4 : w >> (4 * n - 4)) & 0x00F000F0u) | 0x54005400u;
#pragma unroll
        for (int i = 0; i < NQ; ++i) o[i][j] = mfma_pv(v, pf[i][j / kPer], o[i][j]);
      }
    }
  };

  // ---- the tokens, the next step's codes on their way during each step
  {
    int step = part * sh.per + (SPLIT ? wave : 0);
    int stop = step_end;
    if constexpr (!SPLIT) {
      // a wave's own rows may see less than the workgroup's
      stop = min(stop, (any_hi - first_token + kTokens - 1) / kTokens);
      step = max(step, (any_lo - first_token) / kTokens);
    }
    auto token = [&](int s) { return first_token + s * kTokens; };
    if (step < stop) {
      int ids = pages_from(step), at = 0;         // `at`: the sub-tile of ids that comes next
      auto take = [&](int (&p)[2]) {
        p[0] = __builtin_amdgcn_readlane(ids, at);
        p[1] = __builtin_amdgcn_readlane(ids, at + 1);
        at += 2;
      };
      int pages[2], next[2];
      R cur, nxt;
      take(pages);
      load(token(step), pages, cur);
      for (; step < stop; step += kStride) {
        if (step + kStride < stop) {
          if (at == 64) {
            ids = pages_from(step + kStride);
            at = 0;
          }
          take(next);
          load(token(step + kStride), next, nxt);
        }
        process(token(step), pages, cur);
        cur = nxt;
        pages[0] = next[0];
        pages[1] = next[1];
      }
    }
  }

  // ---- finished rows: a lane holds query l16, dimensions of sixteenths 4 kb .. 4 kb + 3
  const bool whole = sh.parts == 1;
  const int64_t all_rows = a.T * a.q_heads;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    l[i] += __shfl_xor(l[i], 16);
    l[i] += __shfl_xor(l[i], 32);
    const float inv = l[i] == 0.0f ? 0.0f : ref / l[i];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[i][j] = (o[i][j] - z[i][j / kPer]) * inv;
  }
  auto dim_of = [&](int unit, int j) { return (j / kPer) * (D / G) + unit * kPer + j % kPer; };
  if constexpr (SPLIT) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int r = wave * kRowsW + 16 * i + l16;
      if (kb == 0) {
        shared_m[r] = m[i];
        shared_l[r] = l[i];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < kTiles; ++j) shared_o[r * kPitch + dim_of(4 * kb + e, j)] = o[i][j][e];
    }
    __syncthreads();
    constexpr int kChunks = D / 8;
    const int n_rows = min(kRowsW, rows - row0);
    for (int item = threadIdx.x; item < n_rows * kChunks; item += kThreads) {
      const int r = item / kChunks, c = item - r * kChunks;
      float top = shared_m[r];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = __builtin_fmaxf(top, shared_m[w * kRowsW + r]);
      float sum = 0.0f, out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(shared_m[w * kRowsW + r] - top) * shared_l[w * kRowsW + r];
        sum += f;
        if (f != 0.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            out[e] = __builtin_fmaf(f, shared_o[(w * kRowsW + r) * kPitch + 8 * c + e], out[e]);
        }
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] *= inv;
      const int tok = (row0 + r) / heads;
      const int64_t to = (seq.q0 + tok) * a.q_heads + h * heads + (row0 + r) - tok * heads;
      if (whole) {
        store16(static_cast<uint16_t*>(a.y) + to * D, c, pack8<BF>(out));
      } else {
        float* po = a.workspace + (part * all_rows + to) * D + 8 * c;
        *reinterpret_cast<f4*>(po) = f4{out[0], out[1], out[2], out[3]};
        *reinterpret_cast<f4*>(po + 4) = f4{out[4], out[5], out[6], out[7]};
        if (c == 0) {
          float* ml = a.workspace + plan.parts * all_rows * D + (part * all_rows + to) * 2;
          ml[0] = top;
          ml[1] = sum;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (q_row[i] < 0) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int unit = 4 * kb + e;
        if (whole) {
          uint16_t* y = static_cast<uint16_t*>(a.y) + q_row[i] * D;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            uint16_t* to = y + dim_of(unit, g * kPer);
            if constexpr (kPer % 8 == 0) {
#pragma unroll
              for (int q = 0; q < kPer / 8; ++q) {
                float t[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) t[n] = o[i][g * kPer + 8 * q + n][e];
                store16(to, q, pack8<BF>(t));
              }
            } else {
#pragma unroll
              for (int n = 0; n < kPer; n += 2) {
                const uint32_t two = round16<BF>(o[i][g * kPer + n][e]) | (uint32_t)round16<BF>(o[i][g * kPer + n + 1][e]) << 16;
                *reinterpret_cast<uint32_t*>(to + n) = two;
              }
            }
          }
        } else {
          float* po = a.workspace + (part * all_rows + q_row[i]) * D;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int n = 0; n < kPer; n += 2) {
              float2 two = make_float2(o[i][g * kPer + n][e], o[i][g * kPer + n + 1][e]);
              *reinterpret_cast<float2*>(po + dim_of(unit, g * kPer + n)) = two;
            }
        }
      }
      if (!whole && kb == 0) {
        float* ml = a.workspace + plan.parts * all_rows * D + (part * all_rows + q_row[i]) * 2;
        ml[0] = m[i];
        ml[1] = l[i];
      }
    }
  }
}

// The parts of each row, joined. One workgroup per row: D / 8 lanes hold its
// dimensions, and the workgroup's slices take the parts in turn.
constexpr int kMaxParts = kThreads;

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads) kv4_join(Kv4AttentionArgs a, Plan plan) {
  constexpr int kLanes = D / 8, kSlices = kThreads / kLanes;
  __shared__ float weight[kMaxParts], wave_top[kWaves], wave_sum[kWaves];
  __shared__ float slice_o[kSlices][D];
  const int64_t row = blockIdx.x, all_rows = a.T * a.q_heads;
  const int64_t token = row / a.q_heads;
  const int head = (int)(row - token * a.q_heads), heads = a.q_heads / a.cache.kv_heads;
  int64_t b;
  if (a.query_offsets) {
    int64_t lo = 0, hi = a.B;           // the last sequence that begins at or before the token
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.query_offsets[mid] <= token) lo = mid; else hi = mid;
    }
    b = lo;
  } else {
    b = token / (a.T / a.B);
  }
  const Sequence seq = sequence(a, b);
  const int64_t tok = token - seq.q0;
  if (tok < 0 || tok >= seq.n) return;
  const int rows = seq.n * heads;
  const int row0 = (int)((tok * heads + head % heads) / plan.rows) * plan.rows;
  const int last = min(rows, row0 + plan.rows) - 1;
  const Share sh = share(a, seq, row0 / heads, last / heads, plan.parts, plan.least);
  if (sh.parts == 1) return;            // written by its workgroup
  const int c = threadIdx.x % kLanes, slice = threadIdx.x / kLanes, wave = threadIdx.x >> 6;

  float m = kLeast, l = 0.0f;
  if ((int)threadIdx.x < sh.parts) {
    const float2 ml = reinterpret_cast<const float2*>(a.workspace + plan.parts * all_rows * D)[threadIdx.x * all_rows + row];
    m = ml.x;
    l = ml.y;
  }
  float top = m;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
  if ((threadIdx.x & 63) == 0) wave_top[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, wave_top[w]);
  const float f = __builtin_amdgcn_exp2f(m - top) * l;
  float sum = f;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) wave_sum[wave] = sum;
  weight[threadIdx.x] = f;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += wave_sum[w];

  float out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = 0.0f;
#pragma unroll 2
  for (int p = slice; p < sh.parts; p += kSlices) {
    const float* po = a.workspace + (p * all_rows + row) * D + 8 * c;
    const f4 u = *reinterpret_cast<const f4*>(po), w = *reinterpret_cast<const f4*>(po + 4);
    const float g = weight[p];
    if (g != 0.0f) {                    // a part without a visible token holds nothing
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[e] = __builtin_fmaf(g, u[e], out[e]);
        out[4 + e] = __builtin_fmaf(g, w[e], out[4 + e]);
      }
    }
  }
  const int used = min(kSlices, sh.parts);
  if (slice > 0 && slice < used) {
#pragma unroll
    for (int e = 0; e < 8; ++e) slice_o[slice][8 * c + e] = out[e];
  }
  __syncthreads();
  if (slice > 0) return;
  for (int s = 1; s < used; ++s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] += slice_o[s][8 * c + e];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] *= inv;
  store16(static_cast<uint16_t*>(a.y) + row * D, c, pack8<BF>(out));
}

// ---- the launch -------------------------------------------------------------------

constexpr int kPrefillTiles = 2;        // NQ of a wave with rows of its own

bool split_tokens(int64_t T, int64_t B, int heads) { return T * heads <= 32 * B; }

Plan plan_of(int64_t T, int64_t B, int q_heads, int kv_heads, int64_t capacity, bool ragged) {
  const int heads = q_heads / kv_heads;
  const bool split = split_tokens(T, B, heads);
  Plan p;
  p.rows = split ? 16 : kWaves * 16 * kPrefillTiles;
  p.tiles_per = (T / std::max<int64_t>(B, 1) * heads + p.rows - 1) / p.rows;
  p.slots = ragged ? T * heads / p.rows + B : B * p.tiles_per;
  p.least = split ? kWaves : 16;
  const int64_t steps = (capacity + kTokens - 1) / kTokens;
  const int64_t groups = std::max<int64_t>(p.slots * kv_heads, 1), want = split ? 2048 : 512;
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>({(want + groups - 1) / groups, (steps + p.least - 1) / p.least, kMaxParts}));
  return p;
}

template <int D, int G, bool BF>
void launch_attention_t(const Kv4AttentionArgs& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.slots * p.parts * a.cache.kv_heads)), block(kThreads);
  if (p.rows == 16) kv4_attention<D, G, BF, 1, true><<<grid, block, 0, st>>>(a, p);
  else kv4_attention<D, G, BF, kPrefillTiles, false><<<grid, block, 0, st>>>(a, p);
  if (p.parts > 1) {
    kv4_join<D, BF><<<dim3((unsigned)(a.T * a.q_heads)), block, 0, st>>>(a, p);
  }
}

template <bool BF>
void launch_attention_d(const Kv4AttentionArgs& a, const Plan& p, hipStream_t st) {
  switch (a.cache.head_dim * 8 + a.cache.groups) {
    case 64 * 8 + 1: launch_attention_t<64, 1, BF>(a, p, st); break;
    case 64 * 8 + 2: launch_attention_t<64, 2, BF>(a, p, st); break;
    case 128 * 8 + 1: launch_attention_t<128, 1, BF>(a, p, st); break;
    case 128 * 8 + 2: launch_attention_t<128, 2, BF>(a, p, st); break;
    case 128 * 8 + 4: launch_attention_t<128, 4, BF>(a, p, st); break;
    case 256 * 8 + 1: launch_attention_t<256, 1, BF>(a, p, st); break;
    case 256 * 8 + 2: launch_attention_t<256, 2, BF>(a, p, st); break;
    default: launch_attention_t<256, 4, BF>(a, p, st); break;
  }
}

}  // namespace

bool kv4_attention_fits(int64_t T, int64_t B, int q_heads, int kv_heads, int64_t capacity) {
  for (const bool ragged : {false, true}) {
    const Plan p = plan_of(T, B, q_heads, kv_heads, capacity, ragged);
    if (p.slots * p.parts * kv_heads * kThreads >= (int64_t(1) << 31)) return false;
    if (p.parts > 1 && T * q_heads * kThreads >= (int64_t(1) << 31)) return false;
  }
  return true;
}

int64_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int64_t capacity) {
  int parts = 1;                        // the call may come with or without query_offsets
  for (const bool ragged : {false, true}) parts = std::max(parts, plan_of(T, B, q_heads, kv_heads, capacity, ragged).parts);
  return parts > 1 ? parts * T * q_heads * (head_dim + 2) * (int64_t)sizeof(float) : 0;
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, bool bf16, hipStream_t stream) {
  const Plan p = plan_of(a.T, a.B, a.q_heads, a.cache.kv_heads, a.max_pages << a.cache.page_shift, a.query_offsets != nullptr);
  bf16 ? launch_attention_d<true>(a, p, stream) : launch_attention_d<false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace cider
