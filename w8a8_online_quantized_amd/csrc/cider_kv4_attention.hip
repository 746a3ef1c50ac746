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
// heads shares each read of the cache. Tokens are taken 32 at a time:
//   S^T = K Q^T  v_mfma_f32_16x16x32, tokens as rows. A nibble n becomes an operand
//        by a mask and an or: the fp16 pattern 0x5400 | n << 4 is 64 + n, the bf16
//        pattern 0x4300 | n is 128 + n. The sums start at -72 * sum(q) (-136 *
//        sum(q)), so taking n to n - 8 costs nothing, and s_k scales the finished
//        fp32 sums. (fp16 denormals, n * 2^-24, would need no or, but the matrix
//        core aligns products by their exponent fields: sums of them lose ten bits.)
//   p = 2^(S - m): four tokens of one query per lane and 16 tokens, which is the
//        layout in which the next product reads them. p * s_v is rounded to fp16
//        (both types: 2^-11 relative, where bf16 would leave 2^-8); s_v is taken
//        in units of a power of two that follow the largest one seen, which is
//        64 to 128 of them: weights end at 2^15, the largest ones that fp16 has,
//        so that small ones lose as little as they can. (A token without weight
//        whose scale is 10^5 times the others', weights spread by 1.5 nats: they
//        lose 0.03% of the result, where the scale as the unit lost them 2.6%,
//        and 0.2% at 10^6.)
//   O^T += V^T P^T  v_mfma_f32_16x16x32_f16, 16 dimensions as rows: operand j is code
//        j of a lane's sixteenth of eight tokens' rows, 64 + n less 72. (Sums of 64 + n
//        with 72 taken off at the end lose what the average of many tokens is smaller
//        than 72: flat weights over 8192, 131072 and 524288 tokens were off by 0.0015,
//        0.02 and 0.1 of the result, with codes as operands by 0.0003 at most.)
// m is raised only when a score passes it by 2^8 (the accumulators are rescaled
// then), so most steps exchange nothing between lanes.
//
// Two kernels. kv4_tokens is for few rows (a decode step): the four waves of a
// workgroup share a tile of 16 rows and take the tokens in turn, codes from
// global memory straight to registers; what bounds it is the stream of the
// codes. kv4_rows is for many: each wave has 16 or 32 rows, and the workgroup
// unpacks a stage of tokens once, into LDS, in the operands' own order. In both
// the tokens are also split over workgroups when there are few tiles; their
// partial results are joined by a second launch.
//
// Measured (heads of 128, bf16): 64 requests of up to 8192 tokens 88 us for 333 MB
// = 3.8 TB/s (the loads alone take 71, the read rate would allow 54); a prompt of
// 8192 tokens, 16 heads, 319 us = 860 TFLOP/s, and 512 queries on 32768 tokens 175
// us = 780 TFLOP/s, where a large matrix product reaches 1190: products, softmax and
// products follow each other in a wave, and the waves of a SIMD start a stage together,
// so the matrix core and the vector unit mostly take turns.
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rows.h"

#include <algorithm>

namespace cider {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTokens = 32;            // of one step of products
// Tiles of 16 rows of a wave of kv4_rows (W waves): what 256 registers hold without
// spills; heads of 64 in two groups one in workgroups of four waves, of which a CU
// then holds three (five prompts of about 1000 tokens 66 us, with two tiles 87; two
// in workgroups of eight: 512 queries on 32768 tokens 172 us, with one tile 226).
constexpr int row_tiles(int D, int G, int W) { return D == 256 || (D / G == 32 && !(D == 64 && W == 8)) ? 1 : 2; }
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -3.402823466e38f;
constexpr float kRaise = 8.0f;         // log2: p stays below 2^8

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

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
__device__ __forceinline__ float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

typedef __attribute__((address_space(1))) const uint8_t gbyte;

template <typename T>
__device__ __forceinline__ T gload(gbyte* p) { return *(__attribute__((address_space(1))) const T*)p; }

// ---- which rows and tokens a workgroup has ------------------------------------

// The launch of kv4_rows: how rows are tiled and tokens split (the same in its join).
struct Plan {
  int waves;           // of a workgroup
  int rows;            // of a workgroup's tile
  int unit;            // tokens of one step of a workgroup's loop
  int parts, least;    // most workgroups per tile, fewest steps of one
  int64_t slots;       // tiles over all sequences, at most
  int64_t tiles_per;   // without query_offsets: tiles of each sequence
};

// Token range of one tile of rows, and how many workgroups share it.
struct Share {
  int begin, end;      // tokens [begin, end) that any of its rows sees
  int steps;           // of plan.unit, from begin rounded down
  int per, parts;      // steps of one part
};

struct Sequence {
  int64_t q0;          // first query row
  int n, length;       // queries, tokens in the cache
};

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
  const int64_t cap = a.max_pages << a.cache.page_shift;
  const int len = a.lengths[b];
  s.length = len < 0 ? 0 : len > cap ? (int)cap : len;
  return s;
}

// tok_lo, tok_hi: the first and the last query token of the tile.
__device__ __forceinline__ Share share(const Kv4AttentionArgs& a, const Plan& plan, const Sequence& s, int tok_lo,
                                       int tok_hi) {
  Share r;
  const int p_lo = s.length - s.n + tok_lo, p_hi = s.length - s.n + tok_hi;
  r.end = a.causal ? min(s.length, p_hi + 1) : s.length;
  r.begin = a.window ? max(0, p_lo - a.window + 1) : 0;
  r.steps = r.end > r.begin ? (r.end - (r.begin & ~(plan.unit - 1)) + plan.unit - 1) / plan.unit : 0;
  r.parts = min(plan.parts, max(1, (r.steps + plan.least - 1) / plan.least));
  r.per = max(1, (r.steps + r.parts - 1) / r.parts);
  r.parts = max(1, (r.steps + r.per - 1) / r.per);
  return r;
}

struct Tile {
  int h, heads;        // key/value head, query heads of each
  int part;
  int64_t b;
  Sequence seq;
  int rows, row0;      // rows of the sequence and head, the tile's first
  Share sh;
};

// The workgroup's tile and part; false where it has none (all threads alike).
__device__ __forceinline__ bool find_tile(const Kv4AttentionArgs& a, const Plan& plan, int lane, Tile& t) {
  const int hkv = a.cache.kv_heads;
  t.heads = a.q_heads / hkv;
  t.h = blockIdx.x % hkv;
  const int64_t rest = blockIdx.x / hkv;
  t.part = (int)(rest % plan.parts);
  const int64_t slot = plan.slots - 1 - rest / plan.parts;      // late tiles see the most tokens: they go first
  int tile = 0;
  if (a.query_offsets) {
    // tiles before each sequence, 64 sequences at a time; every wave alike
    int64_t before = 0;
    bool found = false;
    for (int64_t b0 = 0; b0 < a.B && !found; b0 += 64) {
      int count = 0;
      if (b0 + lane < a.B) count = (int)(((int64_t)sequence(a, b0 + lane).n * t.heads + plan.rows - 1) / plan.rows);
      int sum = count;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(sum, off);
        if (lane >= off) sum += up;
      }
      const uint64_t hit = __ballot(before + sum > slot);
      if (hit) {
        const int first = __builtin_ctzll(hit);
        t.b = uniform((int)b0 + first);
        tile = uniform((int)(slot - before) - (__shfl(sum, first) - __shfl(count, first)));
        found = true;
      }
      before += __shfl(sum, 63);
    }
    if (!found) return false;
  } else {
    t.b = slot / plan.tiles_per;
    tile = (int)(slot - t.b * plan.tiles_per);
  }
  t.seq = sequence(a, t.b);
  t.rows = t.seq.n * t.heads;
  t.row0 = tile * plan.rows;
  t.sh = share(a, plan, t.seq, t.row0 / t.heads, (min(t.rows, t.row0 + plan.rows) - 1) / t.heads);
  return t.part < t.sh.parts;
}

// Tokens that every row of a wave sees, and that some row sees.
struct Sight {
  int all_lo, all_hi, any_lo, any_hi;
};
__device__ __forceinline__ Sight sight(const Kv4AttentionArgs& a, const Tile& t, int first_row, int n_rows) {
  const int last = min(first_row + n_rows, t.rows) - 1;
  const int p0 = t.seq.length - t.seq.n + first_row / t.heads, p1 = t.seq.length - t.seq.n + max(last, 0) / t.heads;
  Sight s;
  s.all_hi = a.causal ? min(t.seq.length, p0 + 1) : t.seq.length;
  s.any_hi = last < first_row ? 0 : a.causal ? min(t.seq.length, p1 + 1) : t.seq.length;
  s.all_lo = a.window ? max(0, p1 - a.window + 1) : 0;
  s.any_lo = a.window ? max(0, p0 - a.window + 1) : 0;
  return s;
}

// The page of the sub-tile of 16 tokens at t, -1 where there is nothing to read.
__device__ __forceinline__ int page_at(const Kv4AttentionArgs& a, int64_t b, int t, int end) {
  int p = -1;
  if (t < end) {
    p = a.page_table[b * a.max_pages + (t >> a.cache.page_shift)];
    if (p < 0 || p >= a.cache.n_pages) p = -1;
  }
  return p;
}

// ---- the operands ---------------------------------------------------------------

// A nibble as an operand: mask, then the exponent of 64 (fp16) or 128 (bf16). The
// constants stay in registers: v_and_or_b32 takes no literals, and v_and and v_or
// with theirs are two instructions.
struct Nibbles {
  uint32_t mask, one;
};
template <bool BF>
__device__ __forceinline__ Nibbles nibbles() {
  Nibbles c{BF ? 0x000F000Fu : 0x00F000F0u, BF ? 0x43004300u : 0x54005400u};
  asm("" : "+s"(c.mask), "+v"(c.one));
  return c;
}
// 8 nibbles of a word as an operand: elements in the order 0 4 1 5 2 6 3 7.
template <bool BF>
__device__ __forceinline__ u4 k_operand(uint32_t w, Nibbles c) {
  const auto pick = [&](uint32_t v) { return (v & c.mask) | c.one; };
  if constexpr (BF) return u4{pick(w), pick(w >> 4), pick(w >> 8), pick(w >> 12)};      // 128 + n
  else return u4{pick(w << 4), pick(w), pick(w >> 4), pick(w >> 8)};                    // 64 + n
}
// 16-bit elements 0 .. 7 in that order.
__device__ __forceinline__ u4 k_order(u4 q) {
  return u4{__builtin_amdgcn_perm(q.z, q.x, 0x05040100u), __builtin_amdgcn_perm(q.z, q.x, 0x07060302u),
            __builtin_amdgcn_perm(q.w, q.y, 0x05040100u), __builtin_amdgcn_perm(q.w, q.y, 0x07060302u)};
}
// Code n of the 16-bit halves of four words (tokens 2i, 2i + 1) as an operand: 64 + its
// nibble, less 72, both exact in fp16.
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u4 v_operand(u4 w, int n, Nibbles c) {
  const auto pick = [&](uint32_t v) {
    const uint32_t b = ((n == 0 ? v << 4 : v >> (4 * n - 4)) & c.mask) | c.one;
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, b) - h2{72, 72});
  };
  return u4{pick(w.x), pick(w.y), pick(w.z), pick(w.w)};
}

// The unit of V's scales for a largest one of v, finite: a power of two (from 2^-126 to
// 2^121) of which v is less than kMostUnits, and the inverse of such a one.
constexpr float kMostUnits = 128.0f;
__device__ __forceinline__ float unit_of(float v) {
  const uint32_t exponent = __builtin_bit_cast(uint32_t, v) & 0x7F800000u;
  return __builtin_bit_cast(float, max(exponent, 7u << 23) - (6u << 23));
}
__device__ __forceinline__ float power_inverse(float v) {
  return __builtin_bit_cast(float, 0x7F000000u - __builtin_bit_cast(uint32_t, v));
}

// What a scale of V asks of the unit: infinities and NaN nothing, as rows that do
// not see them share it.
__device__ __forceinline__ float unit_size(float v) {
  v = __builtin_fabsf(v);
  return v < __builtin_inff() ? v : 0.0f;
}

// ---- the rows of a wave -----------------------------------------------------------

template <int D, int G, int NQ>
struct Rows {
  static constexpr int kTiles = D / 16, kPer = kTiles / G, kSteps = D / 32;
  u4 q[NQ][kSteps];          // operands of the scores
  float q_off[NQ][G];        // what the offset of K's operands adds, negated
  f4 o[NQ][kTiles];          // sums of (p s_v / ref) code: dimension sixteenths 4 kb + e of query l16
  float m[NQ], l[NQ];        // log2 maximum (in steps of kRaise), this lane's part of the sum of p
  float over[NQ];            // how far a score may pass m: kRaise, or kLeast while no token was seen
  float ref[G];              // the unit of s_v, a power of two
  int64_t to[NQ];            // row of y, -1 behind the last one
  int lo[NQ], hi[NQ];        // tokens that the row sees

  template <bool BF>
  __device__ __forceinline__ void begin(const Kv4AttentionArgs& a, const Tile& t, int first_row, int lane) {
    const int l16 = lane & 15, kb = lane >> 4;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int r = first_row + 16 * i + l16;
      const bool real = r < t.rows;
      const int rr = real ? r : t.rows - 1;
      const int tok = rr / t.heads, head = t.h * t.heads + rr - tok * t.heads;
      const int pos = t.seq.length - t.seq.n + tok;
      to[i] = real ? (t.seq.q0 + tok) * a.q_heads + head : -1;
      hi[i] = a.causal ? min(t.seq.length, pos + 1) : t.seq.length;
      lo[i] = a.window ? max(0, pos - a.window + 1) : 0;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (t.seq.q0 + tok) * a.q_row_stride + head * a.q_head_stride;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int st = 0; st < kSteps / G; ++st) {
          const u4 w = load16(src + g * (D / G) + kb * (D / G / 4) + st * 8, 0);
          float v[8];
          unpack8<BF>(w, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += v[e];
          q[i][g * (kSteps / G) + st] = k_order(w);
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        q_off[i][g] = sum * (BF ? -136.0f : -72.0f);
      }
      m[i] = l[i] = 0.0f;
      over[i] = kLeast;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) o[i][j] = f4{0, 0, 0, 0};
    }
#pragma unroll
    for (int g = 0; g < G; ++g) ref[g] = 0x1p-126f;
  }

  // V's scales of group g are in units of `to_ref` (a power of two) from here on.
  __device__ __forceinline__ void units(int g, float to_ref) {
    const float f = ref[g] * power_inverse(to_ref);
    ref[g] = to_ref;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[i][g * kPer + j] *= f;
  }

  // 32 tokens from `token` on. k(s, step), v(j): operands of sub-tile s and of
  // output tile j; ks(s, g): log2 scales of the scores of tokens 16 s + 4 kb ..,
  // vs(s, g): scales of V in units of ref. masked: not every row sees every token;
  // there(s): sub-tile s may be read at all. AHEAD: operands come from LDS, whose
  // latency is hidden by reading several before the first is needed.
  template <bool BF, bool AHEAD, class K, class V, class KS, class VS, class There>
  __device__ __forceinline__ void step(int token, int kb, bool masked, K k, V v, KS ks, VS vs, There there) {
    float x[NQ][8];                      // scores less m
    u4 k_ahead[2][AHEAD ? kSteps : 1];
    if constexpr (AHEAD && kSteps <= 4) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int st = 0; st < kSteps; ++st) k_ahead[s][st] = k(s, st);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        f4 acc[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) acc[i] = f4{q_off[i][g], q_off[i][g], q_off[i][g], q_off[i][g]};
#pragma unroll
        for (int st = 0; st < kSteps / G; ++st) {
          const u4 op = AHEAD && kSteps <= 4 ? k_ahead[s][g * (kSteps / G) + st] : k(s, g * (kSteps / G) + st);
#pragma unroll
          for (int i = 0; i < NQ; ++i) acc[i] = mfma_qk<BF>(op, q[i][g * (kSteps / G) + st], acc[i]);
        }
        const f4 scale = ks(s, g);
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[i][4 * s + e] = __builtin_fmaf(acc[i][e], scale[e], g == 0 ? -m[i] : x[i][4 * s + e]);
      }
    }
    if (masked) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int tok = token + 16 * (e >> 2) + 4 * kb + (e & 3);
        const bool some = there(e >> 2);
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          x[i][e] = some && tok >= lo[i] && tok < hi[i] ? x[i][e] : -__builtin_inff();
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    float most[NQ];
    bool raise = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      most[i] = x[i][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) most[i] = __builtin_fmaxf(most[i], x[i][e]);
      raise |= most[i] > over[i];
    }
    if (__any(raise)) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        most[i] = __builtin_fmaxf(most[i], __shfl_xor(most[i], 16));
        most[i] = __builtin_fmaxf(most[i], __shfl_xor(most[i], 32));
        const bool fresh = over[i] != kRaise, seen = most[i] > kLeast;
        // up, or down too when these are the row's first tokens
        const float by = !seen ? 0.0f : fresh ? most[i] : __builtin_fmaxf(most[i], 0.0f);
        const float f = fresh ? 1.0f : __builtin_amdgcn_exp2f(-by);
        m[i] += by;
        if (seen) over[i] = kRaise;
        l[i] *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] -= by;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[i][j] *= f;
      }
    }
    constexpr int kAhead = AHEAD ? 4 : 1;
    u4 v_ahead[kAhead];
    if constexpr (AHEAD) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) v_ahead[j] = v(j);
      __builtin_amdgcn_sched_barrier(0);
    }
    u4 p16[NQ][G];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[i][e]);
        l[i] += p[e];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const f4 v0 = vs(0, g), v1 = vs(1, g);
        f8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = p[e] * (e < 4 ? v0[e & 3] : v1[e & 3]);
        if (masked) {                    // a hidden token's scale may be anything
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = x[i][e] == -__builtin_inff() ? 0.0f : w[e];
        }
        p16[i][g] = __builtin_bit_cast(u4, __builtin_convertvector(w, h8));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const u4 op = AHEAD ? v_ahead[j % kAhead] : v(j);
      if constexpr (AHEAD) {
        if (j + kAhead < kTiles) v_ahead[j % kAhead] = v(j + kAhead);
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) o[i][j] = mfma_pv(op, p16[i][j / kPer], o[i][j]);
      if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // o becomes the rows' averages; m and l those of the whole row.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      l[i] += __shfl_xor(l[i], 16);
      l[i] += __shfl_xor(l[i], 32);
      if (over[i] != kRaise) m[i] = kLeast;
      const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // (ref * inv may be subnormal; uniform, or the compiler keeps an array in LDS,
        // whose addresses take the dispatch packet: 3 to 10 us of a launch)
        const float unit = uniform(ref[g]);
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[i][g * kPer + j] = o[i][g * kPer + j] * inv * unit;
      }
    }
  }

  // Dimension of sixteenth u (of 16) and code j of it.
  static __device__ __forceinline__ int dim(int u, int j) { return (j / kPer) * (D / G) + u * kPer + j % kPer; }
};

// Partial results: fp32 averages [parts][T * q_heads][D], then (m, l) of each.
__device__ __forceinline__ float* part_row(const Kv4AttentionArgs& a, int part, int64_t row, int D) {
  return a.workspace + (part * a.T * a.q_heads + row) * D;
}
__device__ __forceinline__ float2* part_ml(const Kv4AttentionArgs& a, const Plan& plan, int part, int64_t row, int D) {
  return reinterpret_cast<float2*>(a.workspace + plan.parts * a.T * a.q_heads * D) + part * a.T * a.q_heads + row;
}

// ---- few rows -------------------------------------------------------------------
//
// The launch has a fixed number of workgroups, and each takes an equal share of
// all the work: rounds of 128 tokens (one step per wave) of one tile of rows and
// one key/value head ("segment"), in the order of sequences, heads, tiles. A
// workgroup may so end one segment, have some of its own, and begin another; what
// it has not alone goes to the workspace, and the workgroup in which a segment
// began notes there where its other parts are.

constexpr int kRoundTokens = kTokens * kWaves;

// A segment that began in workgroup i (entry i): its parts are that workgroup's
// second partial result and the first ones of the next parts - 1.
struct Note {
  int parts, q0, h, row0, rows;        // parts 0: none; rows: of the tile, rows there are
  int pad[3];
};

// Workspace: notes [blocks], then partial results [blocks][2][16] rows of fp32
// averages [D], then their (m, l).
__device__ __forceinline__ float* piece_row(const Kv4AttentionArgs& a, int blocks, int64_t piece, int row, int D) {
  return a.workspace + blocks * 8 + (piece * 16 + row) * D;
}
__device__ __forceinline__ float2* piece_ml(const Kv4AttentionArgs& a, int blocks, int64_t piece, int row, int D) {
  return reinterpret_cast<float2*>(a.workspace + blocks * 8 + (int64_t)blocks * 32 * D) + piece * 16 + row;
}

// Rounds of each of a sequence's segments, and how many segments it has.
__device__ __forceinline__ int rounds_of(const Kv4AttentionArgs& a, const Sequence& s) {
  const int begin = (a.window ? max(0, s.length - s.n - a.window + 1) : 0) & ~(kTokens - 1);
  return s.length > begin ? (s.length - begin + kRoundTokens - 1) / kRoundTokens : 1;   // rows of zeros take one, too
}
__device__ __forceinline__ int tiles_of(const Sequence& s, int heads) { return (int)(((int64_t)s.n * heads + 15) / 16); }

// One step's 32 tokens as loaded: a lane has the codes of its K row (l16) and of
// its sixteenth of eight V rows, and one token's scale of K (lanes 0 .. 31) or V.
template <int D, int G>
struct Raw {
  static constexpr int kVW = D / 128 ? D / 128 : 1;   // words of a sixteenth of a V row
  uint32_t k[2][D / 32];
  uint32_t v[8][kVW];
  float s[G];
};

// Workgroups of kv4_tokens that a CU holds at once: two waves per SIMD, without
// spills (three: the decode batch below 107 us instead of 89), one for D = 256, which
// needs more than 256 registers (24 requests of 5 queries in a window of 3000: two 56
// us with spills, one 35).
constexpr int tokens_per_cu(int D) { return D == 256 ? 1 : 2; }

template <int D, int G, bool BF>
__global__ void __launch_bounds__(kThreads, tokens_per_cu(D)) kv4_tokens(Kv4AttentionArgs a, int blocks) {
  using R = Rows<D, G, 1>;
  constexpr int kSteps = R::kSteps, kPitch = D + 4;
  union Shared {
    struct {
      float o[kWaves][16][kPitch], m[kWaves][16], l[kWaves][16];
    } out;
    float s[kWaves][G][64];              // a step's scales, each wave its own
    struct {
      int64_t sum[kWaves], before, b;
    } plan;
  };
  __shared__ Shared shared;
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, kb = lane >> 4;
  const int hkv = a.cache.kv_heads, heads = a.q_heads / hkv;
  // one XCD's workgroups are neighbours in the work, so that a head's tiles share its L2
  const int block = blocks % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8) * (blocks / 8) + (int)blockIdx.x / 8;
  Note* const note = reinterpret_cast<Note*>(a.workspace) + block;

  // ---- the share: rounds [pos, pos_end) of all
  auto work_of = [&](int64_t b) {
    const Sequence q = sequence(a, b);
    return (int64_t)tiles_of(q, heads) * hkv * rounds_of(a, q);
  };
  auto scan = [&](int64_t v, int64_t& total) {          // inclusive sums over the workgroup
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t up = __shfl_up(v, off);
      if (lane >= off) v += up;
    }
    __syncthreads();
    if (lane == 63) shared.plan.sum[wave] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) v += shared.plan.sum[w];
      total += shared.plan.sum[w];
    }
    return v;
  };
  int64_t all = 0;
  int64_t mine = 0, upto = 0;            // of sequence threadIdx.x, kept when there are no more
  for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
    mine = b0 + threadIdx.x < a.B ? work_of(b0 + threadIdx.x) : 0;
    int64_t total;
    upto = scan(mine, total);
    all += uniform(total);
  }
  const int64_t share = (all + blocks - 1) / blocks;
  int64_t pos = block * share;
  const int64_t pos_end = min(all, pos + share);
  if (pos >= pos_end) {
    if (a.workspace && threadIdx.x == 0) note->parts = 0;
    return;
  }
  {
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
      int64_t total = all;
      if (a.B > kThreads) {
        mine = b0 + threadIdx.x < a.B ? work_of(b0 + threadIdx.x) : 0;
        upto = scan(mine, total);
      }
      if (before + upto > pos && before + upto - mine <= pos) {
        shared.plan.before = before + upto - mine;
        shared.plan.b = b0 + threadIdx.x;
      }
      if (before + total > pos) break;
      before += uniform(total);
    }
  }
  __syncthreads();
  int64_t b = uniform((int)shared.plan.b);
  int in_b = uniform((int)(pos - shared.plan.before));  // rounds of this sequence before pos: below 2^31
  __syncthreads();

  const float scale = a.softmax_scale * kLog2e;
  const int page_size = a.cache.page_size;
  const Nibbles k_nib = nibbles<BF>(), v_nib = nibbles<false>();

  // ---- a segment, or the part of it that is in the share
  struct Segment {
    Tile t;
    Sight see;
    int rounds, first_round, n_rounds;   // of the segment; those in the share
    int64_t began;                       // the first of those, of all
    int first_token, step, step_end;     // this wave's steps, kWaves apart
  } seg;
  Sequence seq = sequence(a, b);
  auto next = [&]() {
    if (pos >= pos_end) return false;
    int tiles;
    while (true) {
      tiles = tiles_of(seq, heads);
      seg.rounds = rounds_of(a, seq);
      if (in_b < tiles * hkv * seg.rounds) break;
      in_b -= tiles * hkv * seg.rounds;  // the next sequence (this one may have no queries)
      seq = sequence(a, ++b);
    }
    const int which = in_b / seg.rounds;
    seg.first_round = in_b - which * seg.rounds;
    seg.n_rounds = (int)min((int64_t)(seg.rounds - seg.first_round), pos_end - pos);
    seg.began = pos;
    in_b += seg.n_rounds;
    pos += seg.n_rounds;
    Tile& t = seg.t;
    t.heads = heads;
    t.b = b;
    t.seq = seq;
    t.rows = seq.n * heads;
    t.h = which / tiles;
    t.row0 = (which - t.h * tiles) * 16;
    seg.see = sight(a, t, t.row0, 16);
    // (a sequence's segments all begin where its first query's window does)
    seg.first_token = ((a.window ? max(0, seq.length - seq.n - a.window + 1) : 0) & ~(kTokens - 1)) +
                      seg.first_round * kRoundTokens;
    seg.step_end = min(seg.n_rounds * kWaves, (seg.see.any_hi - seg.first_token + kTokens - 1) / kTokens);
    seg.step = wave;
    if (seg.see.any_lo > seg.first_token) seg.step += (seg.see.any_lo - seg.first_token) / kRoundTokens * kWaves;
    return true;
  };

  const uint32_t k_lane = l16 * (D / 2) + kb * (D / G / 8), v_lane = 4 * kb * (D / 2) + l16 * (D / 32);
  auto load = [&](int token, const int (&pages)[2], Raw<D, G>& r) {
    int64_t ph[2];
    int at[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool there = pages[s] >= 0;
      at[s] = there ? (token + 16 * s) & (page_size - 1) : 0;
      ph[s] = (int64_t)(there ? pages[s] : 0) * hkv + seg.t.h;
      const int64_t base = (ph[s] * page_size + at[s]) * (D / 2);
      gbyte* k = (gbyte*)a.cache.k_codes + base;      // uniform; the lane's part is a 32-bit offset
#pragma unroll
      for (int g = 0; g < G; ++g) {
        gbyte* kg = k + k_lane + g * (D / G / 2);
        constexpr int kW = kSteps / G;
        if constexpr (kW % 4 == 0) {
#pragma unroll
          for (int i = 0; i < kW / 4; ++i) {
            const u4 w = gload<u4>(kg + 16 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.k[s][g * kW + 4 * i + e] = w[e];
          }
        } else if constexpr (kW == 2) {
          const u2 w = gload<u2>(kg);
          r.k[s][g * kW] = w.x;
          r.k[s][g * kW + 1] = w.y;
        } else {
          r.k[s][g] = gload<uint32_t>(kg);
        }
      }
      gbyte* v = (gbyte*)a.cache.v_codes + base;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gbyte* vi = v + v_lane + i * (D / 2);
        if constexpr (D == 64) r.v[4 * s + i][0] = gload<uint16_t>(vi);
        else if constexpr (D == 128) r.v[4 * s + i][0] = gload<uint32_t>(vi);
        else {
          const u2 w = gload<u2>(vi);
          r.v[4 * s + i][0] = w.x;
          r.v[4 * s + i][1] = w.y;
        }
      }
    }
    const bool second = lane & 16;
    const int64_t so = (second ? ph[1] : ph[0]) * G * page_size + (second ? at[1] : at[0]) + l16;
    gbyte* from = lane < 32 ? (gbyte*)a.cache.k_scale : (gbyte*)a.cache.v_scale;
#pragma unroll
    for (int g = 0; g < G; ++g) r.s[g] = gload<float>(from + (so + g * page_size) * 4);
  };

  R rows;
  auto process = [&](int token, const int (&pages)[2], Raw<D, G>& r) {
    const Sight& see = seg.see;
    const bool masked = token < see.all_lo || token + kTokens > see.all_hi || pages[0] < 0 || pages[1] < 0;
    if (masked) {
      // scales that no row may see are nothing
      const int tok = token + (lane & 31);
      const bool there0 = pages[0] >= 0, there1 = pages[1] >= 0;
      const bool some = ((lane & 16) ? there1 : there0) && tok >= see.any_lo && tok < see.any_hi;
#pragma unroll
      for (int g = 0; g < G; ++g) r.s[g] = some ? r.s[g] : 0.0f;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float v = lane < 32 ? 0.0f : unit_size(r.s[g]);
      if (__any(v > rows.ref[g] * kMostUnits)) {
        float top = v;
        for (int off = 16; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
        rows.units(g, unit_of(__shfl(top, 32)));
      }
      shared.s[wave][g][lane] = r.s[g] * (lane < 32 ? scale : power_inverse(rows.ref[g]));
    }
    auto k = [&](int s, int st) { return k_operand<BF>(r.k[s][st], k_nib); };
    u4 w[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int pr = 0; pr < 4; ++pr)
        w[c][pr] = __builtin_amdgcn_perm(r.v[2 * pr + 1][c / 2], r.v[2 * pr][c / 2], c % 2 ? 0x07060302u : 0x05040100u);
    auto v = [&](int j) { return v_operand(w[j / 4], j % 4, v_nib); };
    auto ks = [&](int s, int g) { return *reinterpret_cast<const f4*>(&shared.s[wave][g][16 * s + 4 * kb]); };
    auto vs = [&](int s, int g) { return *reinterpret_cast<const f4*>(&shared.s[wave][g][32 + 16 * s + 4 * kb]); };
    auto there = [&](int s) { return s ? pages[1] >= 0 : pages[0] >= 0; };
    rows.template step<BF, false>(token, kb, masked, k, v, ks, vs, there);
  };

  // The pages of 32 steps, a lane each, so that no step waits for a table entry.
  auto pages_from = [&](int first) {
    return page_at(a, seg.t.b, seg.first_token + (first + (lane >> 1) * kWaves) * kTokens + (lane & 1) * 16, seg.see.any_hi);
  };
  int ids = 0, at = 0;                   // `at`: the sub-tile of ids that comes next
  int ahead = 0;                         // the step whose codes are loaded next
  struct Step {
    int token, pages[2];
    Raw<D, G> raw;
  };
  // Two steps in registers, one on its way while the other is worked on (64 requests
  // of up to 8192 tokens 89 us; three steps 93, four 94). The loads are unconditional
  // (past the end, of the last codes again): behind a branch the wait for one step's
  // would be one for all in flight.
  constexpr int kRing = 2;
  Step ring[kRing];
  auto fetch = [&](Step& to) {
    if (at == 64) {
      ids = pages_from(ahead);
      at = 0;
    }
    to.pages[0] = __builtin_amdgcn_readlane(ids, at);
    to.pages[1] = __builtin_amdgcn_readlane(ids, at + 1);
    to.token = seg.first_token + ahead * kTokens;
    load(to.token, to.pages, to.raw);
    if (ahead + kWaves < seg.step_end) {
      ahead += kWaves;
      at += 2;
    }
  };
  auto fetch_first = [&]() {
    ids = pages_from(seg.step);
    at = 0;
    ahead = seg.step;
#pragma unroll
    for (int i = 0; i + 1 < kRing; ++i) fetch(ring[i]);
  };

  bool noted = false;
  next();
  fetch_first();
  while (true) {
    rows.template begin<BF>(a, seg.t, seg.t.row0, lane);       // its loads behind the first codes'
    bool more = seg.step < seg.step_end;
    while (more) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        fetch(ring[(i + kRing - 1) % kRing]);
        process(ring[i].token, ring[i].pages, ring[i].raw);
        seg.step += kWaves;
        more = seg.step < seg.step_end;
        if (!more) break;
      }
    }
    // the next segment's first codes are on their way while this one is finished
    const Segment done = seg;
    const bool again = next();
    if (again) fetch_first();

    // the waves' parts of each row, joined
    const Tile& t = done.t;
    const bool whole = done.n_rounds == done.rounds;
    rows.finish();
    __syncthreads();                       // every wave is done with its scales
    if (kb == 0) {
      shared.out.m[wave][l16] = rows.m[0];
      shared.out.l[wave][l16] = rows.l[0];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < R::kTiles; ++j) shared.out.o[wave][l16][R::dim(4 * kb + e, j)] = rows.o[0][j][e];
    __syncthreads();
    constexpr int kChunks = D / 8;
    const int n_rows = min(16, t.rows - t.row0);
    for (int item = threadIdx.x; item < n_rows * kChunks; item += kThreads) {
      const int r = item / kChunks, c = item - r * kChunks;
      float top = kLeast;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, shared.out.m[w][r]);
      float sum = 0.0f, f[kWaves], out[8];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(shared.out.m[w][r] - top) * shared.out.l[w][r];
        sum += f[w];
      }
      // (parts of the sum first: averages times sums may pass fp32's largest where the result does not)
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        if (f[w] != 0.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) out[e] = __builtin_fmaf(f[w] * inv, shared.out.o[w][r][8 * c + e], out[e]);
        }
      const int tok = (t.row0 + r) / t.heads;
      const int64_t to = (t.seq.q0 + tok) * a.q_heads + t.h * t.heads + (t.row0 + r) - tok * t.heads;
      if (whole) {
        store16(static_cast<uint16_t*>(a.y) + to * D, c, pack8<BF>(out));
      } else {
        const int64_t piece = 2 * (int64_t)block + (done.first_round == 0);
        float* po = piece_row(a, blocks, piece, r, D) + 8 * c;
        *reinterpret_cast<f4*>(po) = f4{out[0], out[1], out[2], out[3]};
        *reinterpret_cast<f4*>(po + 4) = f4{out[4], out[5], out[6], out[7]};
        if (c == 0) *piece_ml(a, blocks, piece, r, D) = make_float2(top, sum);
      }
    }
    if (!whole && done.first_round == 0) {
      noted = true;
      if (threadIdx.x == 0) {
        const int64_t last = (done.began + done.rounds - 1) / share;      // the workgroup of its last round
        note->parts = (int)(last - block) + 1;
        note->q0 = (int)t.seq.q0;
        note->h = t.h;
        note->row0 = t.row0;
        note->rows = n_rows;
      }
    }
    if (!again) break;
    __syncthreads();                     // the next segment's scales take the place of these sums
  }
  if (a.workspace && !noted && threadIdx.x == 0) note->parts = 0;
}

// The pieces of one row of the segment that began in workgroup blockIdx.x, joined:
// D / 8 lanes hold its dimensions, and the workgroup's slices take the pieces in turn.
template <int D, bool BF>
__global__ void __launch_bounds__(kThreads) kv4_join_pieces(Kv4AttentionArgs a, int blocks) {
  constexpr int kLanes = D / 8, kSlices = kThreads / kLanes;
  __shared__ float slice_o[kSlices][D], wave_top[kWaves], wave_sum[kWaves];
  const int block = blockIdx.x, r = blockIdx.y;
  const Note note = reinterpret_cast<const Note*>(a.workspace)[block];
  if (note.parts == 0 || r >= note.rows) return;
  const int c = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
  auto piece = [&](int p) { return p == 0 ? 2 * (int64_t)block + 1 : 2 * (int64_t)(block + p); };
  // the maximum and the sum of all pieces, so that the averages enter with their parts of it
  float top = kLeast, sum = 0.0f;
  for (int p = threadIdx.x; p < note.parts; p += kThreads) {
    const float2 ml = *piece_ml(a, blocks, piece(p), r, D);
    const float to = __builtin_fmaxf(top, ml.x);
    sum = sum * __builtin_amdgcn_exp2f(top - to) + ml.y * __builtin_amdgcn_exp2f(ml.x - to);
    top = to;
  }
  float most = top;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, off));
  sum *= __builtin_amdgcn_exp2f(top - most);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) {
    wave_top[threadIdx.x >> 6] = most;
    wave_sum[threadIdx.x >> 6] = sum;
  }
  __syncthreads();
  top = kLeast;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, wave_top[w]);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += wave_sum[w] * __builtin_amdgcn_exp2f(wave_top[w] - top);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = 0.0f;
#pragma unroll 4
  for (int p = slice; p < note.parts; p += kSlices) {
    const float2 ml = *piece_ml(a, blocks, piece(p), r, D);
    const float* po = piece_row(a, blocks, piece(p), r, D) + 8 * c;
    const f4 u = *reinterpret_cast<const f4*>(po), w = *reinterpret_cast<const f4*>(po + 4);
    const float g = __builtin_amdgcn_exp2f(ml.x - top) * ml.y * inv;
    if (g != 0.0f) {                    // a piece without a visible token holds nothing
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[e] = __builtin_fmaf(g, u[e], out[e]);
        out[4 + e] = __builtin_fmaf(g, w[e], out[4 + e]);
      }
    }
  }
  const int used = min(kSlices, note.parts);
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
  const int hkv = a.cache.kv_heads, heads = a.q_heads / hkv, tok = (note.row0 + r) / heads;
  const int64_t to = ((int64_t)note.q0 + tok) * a.q_heads + note.h * heads + (note.row0 + r) - tok * heads;
  store16(static_cast<uint16_t*>(a.y) + to * D, c, pack8<BF>(out));
}

// ---- many rows ------------------------------------------------------------------

// Workgroups of W waves, 4 (two per CU, of heads of 64 three) or 8 (one, with twice the
// rows and tokens per stage: a wave then unpacks half as much per token).
// Tokens of a stage: two stages of operands are 64 KB (128 KB), of D = 64 half that.
constexpr int stage_tokens(int D, int W) { return (D == 256 ? 32 : 64) * W / 4; }

// Waves per SIMD: two, of heads of 64 in workgroups of four waves three (one group,
// five prompts of about 1000 tokens: 57 us with three, 62 with two; two groups are no
// faster with four than with three, 67 us).
constexpr int rows_per_simd(int D, int W) { return D == 64 && W == 4 ? 3 : 2; }

template <int D, int G, bool BF, int W>
__global__ void __launch_bounds__(64 * W, rows_per_simd(D, W)) kv4_rows(Kv4AttentionArgs a, Plan plan) {
  constexpr int NQ = row_tiles(D, G, W);
  using R = Rows<D, G, NQ>;
  constexpr int S = stage_tokens(D, W), kSubs = S / 16, kHalves = S / 32;
  constexpr int kSteps = R::kSteps, kTiles = R::kTiles;
  // what a wave unpacks: steps of one sub-tile of K, tiles of one half of V
  constexpr int kKPer = kSteps * kSubs / W, kVPer = kTiles * kHalves / W;
  constexpr int kArrays = 2 * G;         // of scales: K's groups, then V's
  constexpr int kOwn = (kArrays + W - 1) / W, kSpan = (S + 63) / 64;   // a wave's arrays, a lane's tokens
  __shared__ u4 lds_k[2][kSubs][kSteps][64];
  __shared__ u4 lds_v[2][kHalves][kTiles][64];
  __shared__ float lds_s[2][kArrays][S];
  __shared__ float lds_ref[2][G];
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, kb = lane >> 4;
  Tile t;
  if (!find_tile(a, plan, lane, t)) return;
  const int wave_row = t.row0 + wave * 16 * NQ;
  R rows;
  rows.template begin<BF>(a, t, wave_row, lane);
  const Sight see = sight(a, t, wave_row, 16 * NQ);
  const int stage0 = t.part * t.sh.per, stages = min(t.sh.steps, stage0 + t.sh.per) - stage0;
  const int first_token = (t.sh.begin & ~(S - 1)) + stage0 * S;
  const float scale = a.softmax_scale * kLog2e;
  const int page_size = a.cache.page_size, hkv = a.cache.kv_heads;
  const Nibbles k_nib = nibbles<BF>(), v_nib = nibbles<false>();

  // ---- staging: codes and scales of the next stage in registers
  const int k_sub = wave % kSubs, k_step = wave / kSubs * kKPer;
  const int v_half = wave % kHalves, v_tile = wave / kHalves * kVPer;
  uint32_t raw_k[kKPer], raw_v[8];
  float raw_s[kOwn][kSpan];
  float top_ref[kOwn];                   // of the V scales that this wave stages
#pragma unroll
  for (float& r : top_ref) r = 0x1p-126f;
  bool some_s[kSpan];                    // whether any row may see this lane's tokens
  int ids = 0;                           // pages of 64 sub-tiles, a lane each
  int have = 0, have_next = 0;           // which sub-tiles of a stage may be read (bits)
  auto sub_base = [&](int page, int token) {
    const int at = page >= 0 ? token & (page_size - 1) : 0;
    return (((int64_t)(page >= 0 ? page : 0) * hkv + t.h) * page_size + at) * (D / 2);
  };
  auto load = [&](int stage) {
    const int token = first_token + stage * S;
    const int at = stage % (64 / kSubs) * kSubs;
    if (at == 0) ids = page_at(a, t.b, token + lane * 16, t.sh.end);
    int pages[kSubs], bits = 0;
#pragma unroll
    for (int s = 0; s < kSubs; ++s) {
      pages[s] = __builtin_amdgcn_readlane(ids, at + s);
      bits |= (pages[s] >= 0) << s;
    }
    have_next = bits;
    {
      const int page = __builtin_amdgcn_readlane(ids, at + k_sub);
      gbyte* k = (gbyte*)a.cache.k_codes + sub_base(page, token + 16 * k_sub) + l16 * (D / 2) + kb * (D / G / 8);
      constexpr int kW = kSteps / G;     // words of one group in a row's lane
      if constexpr (kW % 4 == 0 && kKPer % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kKPer / 4; ++i) {
          const int st = k_step + 4 * i;
          const u4 w = gload<u4>(k + st / kW * (D / G / 2) + st % kW * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) raw_k[4 * i + e] = w[e];
        }
      } else if constexpr (kW % 2 == 0 && kKPer % 2 == 0) {
#pragma unroll
        for (int i = 0; i < kKPer / 2; ++i) {
          const int st = k_step + 2 * i;
          const u2 w = gload<u2>(k + st / kW * (D / G / 2) + st % kW * 4);
          raw_k[2 * i] = w.x;
          raw_k[2 * i + 1] = w.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kKPer; ++i) {
          const int st = k_step + i;
          raw_k[i] = gload<uint32_t>(k + st / kW * (D / G / 2) + st % kW * 4);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {        // 16 bits of a sixteenth, of four tokens' rows
      const int sub = 2 * v_half + s;
      const int page = __builtin_amdgcn_readlane(ids, at + sub);
      gbyte* v = (gbyte*)a.cache.v_codes + sub_base(page, token + 16 * sub) + 4 * kb * (D / 2) + l16 * (D / 32) +
                 v_tile / 4 * 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) raw_v[4 * s + i] = gload<uint16_t>(v + i * (D / 2));
    }
    // scales: a token (or two, 64 apart) per lane
#pragma unroll
    for (int p = 0; p < kSpan; ++p) {
      int page = pages[4 * p];
#pragma unroll
      for (int s = 1; s < (kSubs < 4 ? kSubs : 4); ++s) page = (lane & (S - 1) & 63) >> 4 == s ? pages[4 * p + s] : page;
      const int tok = token + 64 * p + (lane & (S - 1) & 63);
      some_s[p] = page >= 0 && tok >= t.sh.begin && tok < t.sh.end;
      const int64_t ph = (int64_t)(page >= 0 ? page : 0) * hkv + t.h;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int arr = wave + W * i;
        if (arr >= kArrays) break;
        const int g = arr < G ? arr : arr - G;
        gbyte* from = (arr < G ? (gbyte*)a.cache.k_scale : (gbyte*)a.cache.v_scale) +
                      ((ph * G + g) * page_size + (page >= 0 ? tok & (page_size - 1) : 0)) * 4;
        raw_s[i][p] = gload<float>(from);  // (looked at in store(): not waited for here)
      }
    }
  };
  auto store = [&](int stage) {
    const int buf = stage & 1;
#pragma unroll
    for (int i = 0; i < kKPer; ++i) lds_k[buf][k_sub][k_step + i][lane] = k_operand<BF>(raw_k[i], k_nib);
    u4 w;
#pragma unroll
    for (int pr = 0; pr < 4; ++pr) w[pr] = raw_v[2 * pr] | raw_v[2 * pr + 1] << 16;
    if constexpr (kVPer == 4) {
#pragma unroll
      for (int n = 0; n < 4; ++n) lds_v[buf][v_half][v_tile + n][lane] = v_operand(w, n, v_nib);
    } else {                             // half of the four tiles of these 16 bits
      if (v_tile % 4) w >>= 8;
#pragma unroll
      for (int n = 0; n < 2; ++n) lds_v[buf][v_half][v_tile + n][lane] = v_operand(w, n, v_nib);
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int arr = wave + W * i;
      if (arr >= kArrays) break;
      float value[kSpan], f = scale, top = 0.0f;
#pragma unroll
      for (int p = 0; p < kSpan; ++p) {
        value[p] = some_s[p] ? raw_s[i][p] : 0.0f;
        top = __builtin_fmaxf(top, unit_size(value[p]));
      }
      if (arr >= G) {
        if (__any(top > top_ref[i] * kMostUnits)) {
          for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
          top_ref[i] = unit_of(top);
        }
        f = power_inverse(top_ref[i]);
        if (lane == 0) lds_ref[buf][arr - G] = top_ref[i];
      }
#pragma unroll
      for (int p = 0; p < kSpan; ++p)
        if (S >= 64 || lane < S) lds_s[buf][arr][64 * p + lane] = value[p] * f;
    }
  };

  if (stages > 0) {
    load(0);
    store(0);
  }
  __syncthreads();
  for (int stage = 0; stage < stages; ++stage) {
    have = have_next;
    if (stage + 1 < stages) load(stage + 1);
    const int buf = stage & 1, token = first_token + stage * S;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float to = uniform(lds_ref[buf][g]);
      if (to != uniform(rows.ref[g])) rows.units(g, to);
    }
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      const int first = token + 32 * half;
      if (first >= see.any_hi || first + 32 <= see.any_lo) continue;
      const int bits = have >> (2 * half) & 3;
      auto k = [&](int s, int st) { return lds_k[buf][2 * half + s][st][lane]; };
      auto v = [&](int j) { return lds_v[buf][half][j][lane]; };
      auto ks = [&](int s, int g) { return *reinterpret_cast<const f4*>(&lds_s[buf][g][32 * half + 16 * s + 4 * kb]); };
      auto vs = [&](int s, int g) { return *reinterpret_cast<const f4*>(&lds_s[buf][G + g][32 * half + 16 * s + 4 * kb]); };
      auto there = [&](int s) { return (bits >> s & 1) != 0; };
      const bool masked = first < see.all_lo || first + 32 > see.all_hi || bits != 3;
      rows.template step<BF, true>(first, kb, masked, k, v, ks, vs, there);
    }
    if (stage + 1 < stages) store(stage + 1);
    __syncthreads();
  }

  rows.finish();
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    if (rows.to[i] < 0) continue;
    const bool whole = t.sh.parts == 1;
    constexpr int kPer = R::kPer;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int d = R::dim(4 * kb + e, g * kPer);    // kPer dimensions from here
        if (!whole) {
          float* to = part_row(a, t.part, rows.to[i], D) + d;
#pragma unroll
          for (int n = 0; n < kPer; n += 2)
            *reinterpret_cast<float2*>(to + n) = make_float2(rows.o[i][g * kPer + n][e], rows.o[i][g * kPer + n + 1][e]);
        } else if constexpr (kPer % 8 == 0) {
#pragma unroll
          for (int c = 0; c < kPer / 8; ++c) {
            float v[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] = rows.o[i][g * kPer + 8 * c + n][e];
            store16(static_cast<uint16_t*>(a.y) + rows.to[i] * D + d, c, pack8<BF>(v));
          }
        } else {
          uint16_t* to = static_cast<uint16_t*>(a.y) + rows.to[i] * D + d;
#pragma unroll
          for (int n = 0; n < kPer; n += 2)
            *reinterpret_cast<uint32_t*>(to + n) = round16<BF>(rows.o[i][g * kPer + n][e]) |
                                                   (uint32_t)round16<BF>(rows.o[i][g * kPer + n + 1][e]) << 16;
        }
      }
    }
    if (!whole && kb == 0) *part_ml(a, plan, t.part, rows.to[i], D) = make_float2(rows.m[i], rows.l[i]);
  }
}

// ---- the join -------------------------------------------------------------------

// An average in pieces: (m, l, o) each, joined in their order. It stays an average (of what
// was joined): a sum of l * o may pass fp32's largest where the result does not.
struct Average {
  float top = kLeast, sum = 0.0f, out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  __device__ __forceinline__ void add(float m, float l, const f4& u, const f4& w) {
    if (l == 0.0f) return;               // a piece without a visible token holds nothing
    const float to = __builtin_fmaxf(top, m);
    const float f = __builtin_amdgcn_exp2f(top - to) * sum, g = __builtin_amdgcn_exp2f(m - to) * l;
    top = to;
    sum = f + g;
    // (the GPU's reciprocal, one step off at most: 2^-18 over the 32 pieces of a chain)
    const float inv = __builtin_amdgcn_rcpf(sum), old = f * inv, part = g * inv;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = __builtin_fmaf(part, u[e], out[e] * old);
      out[4 + e] = __builtin_fmaf(part, w[e], out[4 + e] * old);
    }
  }
};

// The parts of each row, joined: SLICES * D / 8 threads hold a row, the slices take
// its parts in turn (1 where there are few parts: sixteen rows of 128 per workgroup;
// a workgroup per row instead took 270 us for 131072 rows of two parts).
constexpr int kMaxParts = 256;

template <int D, bool BF, int SLICES>
__global__ void __launch_bounds__(kThreads) kv4_join(Kv4AttentionArgs a, Plan plan) {
  constexpr int kLanes = D / 8, kRows = kThreads / (kLanes * SLICES);
  __shared__ float slice_o[SLICES > 1 ? SLICES : 1][SLICES > 1 ? D : 1], slice_ml[SLICES > 1 ? SLICES : 1][2];
  static_assert(SLICES == 1 || kRows == 1);
  const int row = blockIdx.x * kRows + threadIdx.x / (kLanes * SLICES);
  const int c = threadIdx.x % kLanes, slice = threadIdx.x / kLanes % SLICES;
  if (row >= (int)a.T * a.q_heads) return;
  const int token = row / a.q_heads;
  const int head = row - token * a.q_heads, heads = a.q_heads / a.cache.kv_heads;
  int64_t b;
  if (a.query_offsets) {
    int64_t lo = 0, hi = a.B;           // the last sequence that begins at or before the token
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.query_offsets[mid] <= token) lo = mid; else hi = mid;
    }
    b = lo;
  } else {
    b = token / (int)(a.T / a.B);
  }
  const Sequence seq = sequence(a, b);
  const int64_t tok = token - seq.q0;
  if (tok < 0 || tok >= seq.n) return;
  const int rows = seq.n * heads;
  const int row0 = ((int)tok * heads + head % heads) / plan.rows * plan.rows;
  const int last = min(rows, row0 + plan.rows) - 1;
  const Share sh = share(a, plan, seq, row0 / heads, last / heads);
  if (sh.parts == 1) return;            // written by its workgroup
  Average avg;
#pragma unroll 2
  for (int p = slice; p < sh.parts; p += SLICES) {
    const float2 ml = *part_ml(a, plan, p, row, D);
    const float* po = part_row(a, p, row, D) + 8 * c;
    avg.add(ml.x, ml.y, *reinterpret_cast<const f4*>(po), *reinterpret_cast<const f4*>(po + 4));
  }
  if constexpr (SLICES > 1) {
    if (slice > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) slice_o[slice][8 * c + e] = avg.out[e];
      if (c == 0) {
        slice_ml[slice][0] = avg.top;
        slice_ml[slice][1] = avg.sum;
      }
    }
    __syncthreads();
    if (slice > 0) return;
    const int used = min(SLICES, sh.parts);
    float top = avg.top;
    for (int s = 1; s < used; ++s) top = __builtin_fmaxf(top, slice_ml[s][0]);
    const float own = __builtin_amdgcn_exp2f(avg.top - top) * avg.sum;
    float sum = own;
    for (int s = 1; s < used; ++s) sum += __builtin_amdgcn_exp2f(slice_ml[s][0] - top) * slice_ml[s][1];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) avg.out[e] *= own * inv;
    for (int s = 1; s < used; ++s) {
      const float part = __builtin_amdgcn_exp2f(slice_ml[s][0] - top) * slice_ml[s][1] * inv;
#pragma unroll
      for (int e = 0; e < 8; ++e) avg.out[e] = __builtin_fmaf(part, slice_o[s][8 * c + e], avg.out[e]);
    }
  }
  store16(static_cast<uint16_t*>(a.y) + (int64_t)row * D, c, pack8<BF>(avg.out));
}

// ---- the launch -------------------------------------------------------------------

// Up to two tiles of 16 rows per sequence and key/value head. With a threshold of 16,
// 32 and 64 (us, 8192 tokens, heads of 128, 8 per key/value head, 2 of those): sixteen
// sequences of 24 rows 35, 32, 32; two of 64 rows 23, 23, 31; sixteen of 64 rows 44,
// 44, 42. Past 32 it depends on how many sequences there are, and few would lose more.
// The rule takes the average, since the host does not know the offsets: 63 single tokens
// on 8192 and 512 queries on 8192 in one call 203 us (two calls 132 + 73), on 32768 432
// (132 + 181), 2048 queries on 8192 537 (132 + 168), as a long sequence's tiles of 16 rows
// each unpack its tokens again.
bool few_rows(int64_t T, int64_t B, int heads) { return T * heads <= 32 * B; }

// kv4_rows. Whole prompts (no more than twice as many tokens as queries) have tiles of
// all lengths, which are done as workgroups come free; other queries see about as many
// tokens each. Eight waves per workgroup pay from 8192 rows per sequence and key/value
// head in the first case (heads of 128, two query heads each; us with 8, 4 waves: 8192
// tokens 319, 356; 4096 tokens 119, 126; 2048 tokens 67, 66; five of about 1000 tokens,
// three heads of 64: 82, 66), from 1024 in the second (512 queries on 8192 tokens 67, 71;
// on 32768 175, 191). Tokens are split until there are as many parts as workgroups are
// resident, for whole prompts twice as many (4096 tokens: 1 part 152, 2 parts 119; 2048
// tokens: 2 parts 59, 4 parts 66; 512 queries on 32768 tokens: 8 parts 175, 16 parts 200).
Plan plan_of(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int groups, int64_t capacity, bool ragged) {
  const int heads = q_heads / kv_heads;
  const int64_t rows = T * heads;
  const bool prompts = capacity < 2 * (T / B);
  Plan p;
  p.waves = rows >= (prompts ? 8192 : 1024) * B ? 8 : 4;
  p.rows = p.waves * 16 * row_tiles(head_dim, groups, p.waves);
  p.unit = stage_tokens(head_dim, p.waves);
  p.least = std::max(1, 256 / p.unit);
  p.tiles_per = (T / B * heads + p.rows - 1) / p.rows;
  p.slots = ragged ? rows / p.rows + B : B * p.tiles_per;
  const int64_t steps = (capacity + p.unit - 1) / p.unit, resident = p.waves == 8 ? 256 : 512;
  const int64_t want = prompts ? 2 * resident : resident;
  const int64_t tiles = B * ((rows + B * p.rows - 1) / (B * p.rows)) * kv_heads;   // of sequences of one length
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>({(want + tiles / 2) / tiles, (steps + p.least - 1) / p.least, kMaxParts}));
  return p;
}

// Workgroups of kv4_tokens: those that are resident at once, or one per round if
// no sequence can have so many. With one round per segment at most, nothing is
// split and nothing joined.
int tokens_blocks(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int64_t capacity) {
  const int64_t segments = (T * (q_heads / kv_heads) / 16 + B) * kv_heads;
  const int64_t rounds = std::max<int64_t>(1, (capacity + kTokens + kRoundTokens - 1) / kRoundTokens);
  const int64_t most = 256 * tokens_per_cu(head_dim);
  return (int)(segments < most ? std::min(most, segments * rounds) : most);
}

template <int D, int G, bool BF>
void launch_attention_t(const Kv4AttentionArgs& a, hipStream_t st) {
  const int hkv = a.cache.kv_heads, heads = a.q_heads / hkv;
  const int64_t capacity = a.max_pages << a.cache.page_shift;
  const dim3 block(kThreads);
  if (few_rows(a.T, a.B, heads)) {
    const int blocks = tokens_blocks(a.T, a.B, a.q_heads, hkv, D, capacity);
    kv4_tokens<D, G, BF><<<dim3(blocks), block, 0, st>>>(a, blocks);
    if (a.workspace) {
      const unsigned rows = a.query_offsets ? 16 : (unsigned)std::min<int64_t>(16, a.T / a.B * heads);
      kv4_join_pieces<D, BF><<<dim3(blocks, rows), block, 0, st>>>(a, blocks);
    }
    return;
  }
  const Plan p = plan_of(a.T, a.B, a.q_heads, hkv, D, G, capacity, a.query_offsets != nullptr);
  const dim3 grid((unsigned)(p.slots * p.parts * hkv));
  if (p.waves == 8) kv4_rows<D, G, BF, 8><<<grid, dim3(512), 0, st>>>(a, p);
  else kv4_rows<D, G, BF, 4><<<grid, block, 0, st>>>(a, p);
  if (p.parts > 8) {
    kv4_join<D, BF, kThreads / (D / 8)><<<dim3((unsigned)(a.T * a.q_heads)), block, 0, st>>>(a, p);
  } else if (p.parts > 1) {
    constexpr int kRows = kThreads / (D / 8);
    kv4_join<D, BF, 1><<<dim3((unsigned)((a.T * a.q_heads + kRows - 1) / kRows)), block, 0, st>>>(a, p);
  }
}

template <bool BF>
void launch_attention_d(const Kv4AttentionArgs& a, hipStream_t st) {
  switch (a.cache.head_dim * 8 + a.cache.groups) {
    case 64 * 8 + 1: launch_attention_t<64, 1, BF>(a, st); break;
    case 64 * 8 + 2: launch_attention_t<64, 2, BF>(a, st); break;
    case 128 * 8 + 1: launch_attention_t<128, 1, BF>(a, st); break;
    case 128 * 8 + 2: launch_attention_t<128, 2, BF>(a, st); break;
    case 128 * 8 + 4: launch_attention_t<128, 4, BF>(a, st); break;
    case 256 * 8 + 1: launch_attention_t<256, 1, BF>(a, st); break;
    case 256 * 8 + 2: launch_attention_t<256, 2, BF>(a, st); break;
    default: launch_attention_t<256, 4, BF>(a, st); break;
  }
}

}  // namespace

bool kv4_attention_fits(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int64_t capacity) {
  constexpr int64_t kLimit = int64_t(1) << 31;
  const int heads = q_heads / kv_heads;
  if (few_rows(T, B, heads)) {           // a sequence's rounds are counted in 32 bits
    return (T * heads / 16 + 1) * kv_heads * ((capacity + kTokens) / kRoundTokens + 1) < kLimit;
  }
  for (int i = 0; i < 6; ++i) {
    const Plan p = plan_of(T, B, q_heads, kv_heads, head_dim, 1 << i / 2, capacity, i % 2);
    if (p.slots * p.parts * kv_heads * 64 * p.waves >= kLimit) return false;
    if (p.parts > 1 && T * q_heads * kThreads >= kLimit) return false;
  }
  return true;
}

int64_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int64_t capacity) {
  if (few_rows(T, B, q_heads / kv_heads)) {
    if (capacity <= kRoundTokens) return 0;            // no segment has a second round
    const int64_t blocks = tokens_blocks(T, B, q_heads, kv_heads, head_dim, capacity);
    return blocks * (8 + 2 * 16 * (head_dim + 2)) * (int64_t)sizeof(float);
  }
  int parts = 1;                        // with or without query_offsets, for any groups
  for (int i = 0; i < 6; ++i)
    parts = std::max(parts, plan_of(T, B, q_heads, kv_heads, head_dim, 1 << i / 2, capacity, i % 2).parts);
  return parts > 1 ? parts * T * q_heads * (head_dim + 2) * (int64_t)sizeof(float) : 0;
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, bool bf16, hipStream_t stream) {
  bf16 ? launch_attention_d<true>(a, stream) : launch_attention_d<false>(a, stream);
  return hipGetLastError();
}

}  // namespace cider
