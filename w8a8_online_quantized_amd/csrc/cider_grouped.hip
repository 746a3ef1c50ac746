// Int8 products grouped by expert, with ragged group sizes that only the GPU
// knows: rows offsets[e] .. offsets[e+1] of the output are the products of
// their activation rows (gathered by an index, or in place) with expert e's
// weights. Per-channel W8A8 or W4A8, the dequant fused as in the dense GEMMs,
// or the gated activation fused on top of it.
//
//   acc[p,n] = sum_k x_q[src(p), k] * w_q[e(p), n, k]          (exact int32)
//   v[p,n]   = ((float)acc * x_scale[src(p)]) * w_scale[e(p), n]       (fp32)
//   plain:   y[p,n] = fp(v[p,n])                    - the dense GEMM's bits
//   swiglu:  y[p,n] = fp(v[p,n] / (1 + exp(-v[p,n])) * v[p, N/2 + n])
//
// The product runs on v_mfma_i32_16x16x64_i8 with the operands streamed
// global -> LDS by buffer-load DMA, NS stages of 128 codes deep, in the
// layouts of the dense kernels (cider_gemm.hip): the weight tile is the
// MFMA's first operand, so lane l holds y[m = l % 16][n = 4 * (l / 16) + r].
// For the gated product a tile holds 16 gate rows, the 16 matching up rows,
// 16 gate rows, ...: a lane then owns the gate and the up value of the same
// output and the activation needs no exchange.
//
// Which tiles exist is decided on the device: each wave scans the group sizes
// (64 experts a step, a DPP prefix sum) and block b takes work unit b of the
// resulting list; blocks past its end leave. The grid covers the longest
// possible list, sum_e ceil(c_e / BM) <= P / BM + min(E, P).
#include <algorithm>
#include <type_traits>

#include "../../include/cider.h"
#include "cider_gemm_common.h"
#include "cider_internal.h"

namespace cider {
namespace {

// Inclusive prefix sum over the 64 lanes of a wave: within rows of 16 by
// shifts, then the row totals across rows.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);   // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);   // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);   // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31
  return x;
}

// Rows [lo, hi) of expert e. Offsets that do not ascend within 0 .. P are
// clamped, so bad values cannot reach past the buffers.
__device__ __forceinline__ void group_bounds(const int32_t* __restrict__ offsets, int E, int P, int e, int& lo, int& hi) {
  lo = hi = 0;
  if (e < E) {
    lo = min(max(offsets[e], 0), P);
    hi = min(max(offsets[e + 1], lo), P);
  }
}

// Activation row of row index i (row_index[p] / row_div), -1 out of range. The
// division is a multiplication: div_mul = ceil(2^(31 + l) / row_div) with
// 2^(l - 1) < row_div <= 2^l is exact for every i < 2^31.
__device__ __forceinline__ int source_of(const GroupedArgs& g, int i) {
  const int src = g.div_mul ? (int)(__umulhi((uint32_t)i, g.div_mul) >> g.div_shift) : i;
  return i >= 0 && src < (int)g.x_rows ? src : -1;
}

struct Unit {
  int e, m0, rows, tn;   // expert, first output row, rows (<= BM), column tile; rows 0: no work
};

// Work unit of block b: units are (row tile, column tile), column tiles
// fastest, and each of the 8 XCDs (block b runs on XCD b % 8) takes a
// contiguous range of them, so that the tiles of one expert share an L2.
constexpr int kGroupM = 4;
template <int BM>
__device__ __forceinline__ Unit find_unit(const int32_t* __restrict__ offsets, int E, int P, int nbn, int b, int lane) {
  Unit u{0, 0, 0, 0};
  int lo, hi;
  group_bounds(offsets, E, P, lane, lo, hi);
  const int t0 = (hi - lo + BM - 1) / BM;
  const int incl0 = wave_scan(t0);
  int tiles = __builtin_amdgcn_readlane(incl0, 63);
  for (int g = 64; g < E; g += 64) {
    int l, h;
    group_bounds(offsets, E, P, g + lane, l, h);
    tiles += __builtin_amdgcn_readlane(wave_scan((h - l + BM - 1) / BM), 63);
  }
  const int units = tiles * nbn;
  const int xcd = b & 7, idx = b >> 3;
  const int per = units >> 3, rem = units & 7;
  if (idx >= per + (xcd < rem ? 1 : 0)) return u;
  const int unit = xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
  int mt = unit / nbn;
  u.tn = unit - mt * nbn;
  int base = 0, t = t0, incl = incl0;
  for (int g = 0; g < E; g += 64) {
    if (g) {
      group_bounds(offsets, E, P, g + lane, lo, hi);
      t = (hi - lo + BM - 1) / BM;
      incl = wave_scan(t);
    }
    const int before = base + incl - t;
    const uint64_t hit = __ballot(mt >= before && mt < before + t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      u.e = g + l;
      const int first = __builtin_amdgcn_readlane(lo, l), last = __builtin_amdgcn_readlane(hi, l);
      const int start = __builtin_amdgcn_readlane(before, l), n = (last - first + BM - 1) / BM;
      if (n > kGroupM) {
        // groups of row tiles, rows fastest within one: the blocks of an XCD
        // then share both operands' panels
        const int local = unit - start * nbn, group = local / (kGroupM * nbn), in = local - group * kGroupM * nbn;
        const int size = min(kGroupM, n - group * kGroupM);
        u.tn = in / size;
        mt = start + group * kGroupM + in - u.tn * size;
      }
      u.m0 = first + (mt - start) * BM;
      u.rows = min(BM, last - u.m0);
      return u;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return u;
}

// 16 packed int4 codes (8 bytes, nibble = code + 8) as bytes 16 * code, in the
// order 0,2,4,6 | 1,3,5,7 | 8,10,12,14 | 9,11,13,15: a nibble in a byte's upper
// half with its top bit flipped is 16 * (nibble - 8) in two's complement, two
// or three operations for four codes where sign-extending them takes five. The
// sums stay exact for every code and nibble, 16 * 128 * 8 * K < 2^31 up to
// CIDER_MOE_MAX_K_PACKED, and are shifted back once at the end.
__device__ __forceinline__ v4i unpack16(int lo, int hi) {
  v4i o;
  o.x = (int)((((uint32_t)lo << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
  o.y = (int)(((uint32_t)lo & 0xF0F0F0F0u) ^ 0x80808080u);
  o.z = (int)((((uint32_t)hi << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
  o.w = (int)(((uint32_t)hi & 0xF0F0F0F0u) ^ 0x80808080u);
  return o;
}

// silu(g) * u. exp is the hardware's 2^x on g * log2(e), whose rounding makes
// its relative error grow as |g| * 2^-24 (5e-6 where exp reaches the end of
// fp32); it and the reciprocal stay far below the 16-bit rounding that follows.
// For g below -87.3 the reciprocal's value leaves the normal range and the
// result may be -0 (the formula's is below 1.2e-36 * |u|).
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

typedef float f4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 scaled4(v4i acc, float sa, float4 sw) {
  return f4{((float)acc.x * sa) * sw.x, ((float)acc.y * sa) * sw.y, ((float)acc.z * sa) * sw.z,
            ((float)acc.w * sa) * sw.w};
}

template <int BM, int BN, int WGM, int WGN, int NS, int WK, bool BF, bool GATED>
__global__ void __launch_bounds__(WGM * WGN * 64)
grouped_kernel(const GroupedArgs g) {
  constexpr int BK = 128, NW = WGM * WGN;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int TM = WTM / 16, TN = WTN / 16;
  constexpr bool kI4 = WK == kWeightI4;
  constexpr int RBA = BK, RBW = kI4 ? BK / 2 : BK;       // bytes per tile row and stage
  constexpr int kBA = BM * RBA / 1024, kBW = BN * RBW / 1024;   // 1 KiB DMA blocks per stage
  constexpr int kIA = (kBA + NW - 1) / NW, kIW = (kBW + NW - 1) / NW;   // per wave (spares go to the pad)
  constexpr int LPS = kIA + kIW;
  constexpr int kStageBytes = BM * RBA + BN * RBW;
  constexpr bool kPad = kBA % NW != 0 || kBW % NW != 0;
  constexpr int kPadBytes = kPad ? 1024 : 0;
  constexpr int BNO = GATED ? BN / 2 : BN;               // output columns per tile
  constexpr int TNO = GATED ? TN / 2 : TN;               // 16-column output fragments per wave
  static_assert(int64_t(16) * 128 * 8 * CIDER_MOE_MAX_K_PACKED < (int64_t(1) << 31), "int4 sums");
  static_assert(TM * 16 == WTM && TN * 16 == WTN && (!GATED || TN % 2 == 0), "wave tile");
  static_assert(BM * RBA % 1024 == 0 && BN * RBW % 1024 == 0, "whole DMA blocks");
  static_assert((NW * (1024 / RBA)) % 16 == 0 && (NW * (1024 / RBW)) % 16 == 0, "a wave's blocks share a swizzle slot");

  // the store stage's slab of output rows reuses the operand stages
  constexpr int kRowB = BNO * 2 + 16;
  constexpr int kAvail = NS * kStageBytes;
  constexpr int R = BM * kRowB <= kAvail ? BM : (BM / 2) * kRowB <= kAvail ? BM / 2 : BM / 4;
  constexpr int NP = BM / R, RB = 16 * TM / NP;
  static_assert(R % 16 == 0 && R * kRowB <= kAvail && TM % NP == 0 && WGM * RB == R, "store slab");

  __shared__ __attribute__((aligned(1024))) int8_t smem[NS * kStageBytes + kPadBytes + (BM + BN) * 4];
  int8_t* const pad = smem + NS * kStageBytes;
  float* const lsc = reinterpret_cast<float*>(smem + NS * kStageBytes + kPadBytes);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // waves 0 .. 3 sit on the four SIMDs and share their rows, so a tile with
  // rows for the first of them only still keeps every SIMD busy
  const int wm = (wave / WGN) * WTM, wn = (wave % WGN) * WTN;
  const int l16 = lane & 15, l4 = lane >> 4;
  const int N = (int)g.N, K = (int)g.K, NO = GATED ? N / 2 : N;
  const int nbn = (NO + BNO - 1) / BNO;

  const Unit u = find_unit<BM>(g.offsets, g.E, (int)g.P, nbn, blockIdx.x, lane);
  if (u.rows <= 0) return;                               // uniform: every wave finds the same unit
  const int n0 = u.tn * BNO;
  const uint32_t lda = (uint32_t)K, ldw = kI4 ? (uint32_t)K / 2 : (uint32_t)K;

  // weight row of tile row r, -1 past the matrix
  auto weight_row = [&](int r) {
    if constexpr (!GATED) return n0 + r < N ? n0 + r : -1;
    const int n = n0 + (r >> 5) * 16 + (r & 15);
    return n < NO ? (r & 16 ? NO + n : n) : -1;
  };

  // Descriptors: the expert's whole weight matrix; all activation rows when
  // they are gathered, else the tile's own. A row that does not exist gets an
  // offset past every descriptor and arrives as zeros.
  constexpr uint32_t kNone = 0x80000000u;
  const __amdgpu_buffer_rsrc_t ra =
      g.row_index ? make_rsrc(g.a, (uint32_t)(g.x_rows * K)) : make_rsrc(g.a + (int64_t)u.m0 * K, (uint32_t)u.rows * lda);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(static_cast<const int8_t*>(g.w) + (int64_t)u.e * N * ldw, (uint32_t)N * ldw);
  const int ca = slot_of<RBA>(wave * (1024 / RBA) + lane / (RBA / 16), lane % (RBA / 16)) * 16;
  const int cw = slot_of<RBW>(wave * (1024 / RBW) + lane / (RBW / 16), lane % (RBW / 16)) * 16;
  uint32_t offa[kIA], offw[kIW];
  auto issue_a = [&](int kt, int buf) {
    int8_t* st = smem + buf * kStageBytes;
    const int kb = kt * BK;
    const bool none = kb + BK > K && kb + ca >= K;       // chunks past K arrive as zeros
#pragma unroll
    for (int i = 0; i < kIA; ++i) {
      const int j = wave + i * NW;
      uint32_t off = offa[i] + (uint32_t)kb;             // (an expression in the call leaves the host side without the kernel)
      if (none) off = kNone;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(kBA % NW != 0 && j >= kBA ? pad : st + j * 1024), 16, off,
                                               0, 0, 0);
    }
  };
  auto issue_w = [&](int kt, int buf) {
    int8_t* st = smem + buf * kStageBytes + BM * RBA;
    const int kb = kt * RBW;
    const bool none = kb + RBW > (int)ldw && kb + cw >= (int)ldw;
#pragma unroll
    for (int i = 0; i < kIW; ++i) {
      const int j = wave + i * NW;
      uint32_t off = offw[i] + (uint32_t)kb;
      if (none) off = kNone;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(kBW % NW != 0 && j >= kBW ? pad : st + j * 1024), 16, off,
                                               0, 0, 0);
    }
  };

  // The row indexes are asked for first and the first weights (which need no
  // index) go out before they are used: loads complete in order.
  int ri[kIA];
#pragma unroll
  for (int i = 0; i < kIA; ++i) {
    const int j = wave + i * NW, r = j * (1024 / RBA) + lane / (RBA / 16);
    ri[i] = j < kBA && r < u.rows ? (g.row_index ? g.row_index[u.m0 + r] : r) : -1;
  }
  constexpr int kScalesPerThread = (BM + BN + NW * 64 - 1) / (NW * 64);
  int rs[kScalesPerThread];                              // scale t of the tile: row t, then column t - BM
#pragma unroll
  for (int i = 0; i < kScalesPerThread; ++i) {
    const int t = threadIdx.x + i * NW * 64;
    rs[i] = t < BM ? (t < u.rows ? (g.row_index ? g.row_index[u.m0 + t] : u.m0 + t) : -1) : weight_row(t - BM);
  }
#pragma unroll
  for (int i = 0; i < kIW; ++i) {
    const int j = wave + i * NW;
    const int r = weight_row(j * (1024 / RBW) + lane / (RBW / 16));
    offw[i] = j < kBW && r >= 0 ? (uint32_t)r * ldw + (uint32_t)cw : kNone;
  }
  issue_w(0, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kIA; ++i) {
    const int src = g.row_index ? source_of(g, ri[i]) : ri[i];
    offa[i] = src >= 0 ? (uint32_t)src * lda + (uint32_t)ca : kNone;
  }
  // the tile's scales, zero where there is no row or column: loaded before the
  // other DMA, written to LDS behind it
  float scl[kScalesPerThread];
#pragma unroll
  for (int i = 0; i < kScalesPerThread; ++i) {
    const int t = threadIdx.x + i * NW * 64;
    const int src = t < BM && g.row_index ? source_of(g, rs[i]) : rs[i];
    scl[i] = src >= 0 && t < BM + BN ? (t < BM ? g.sa[src] : g.sw[(int64_t)u.e * N + src]) : 0.0f;
  }
  issue_a(0, 0);

  const int KT = (K + BK - 1) / BK;
#pragma unroll
  for (int s = 1; s < NS - 1; ++s) {
    issue_a(s, s);
    issue_w(s, s);
  }

#pragma unroll
  for (int i = 0; i < kScalesPerThread; ++i) {
    const int t = threadIdx.x + i * NW * 64;
    if (t < BM + BN) lsc[t] = scl[i];
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);                    // lgkmcnt(0): published by the first stage barrier

  v4i acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = zero4();

  // 16-row fragments of this wave that hold rows of the group: the others are
  // neither read nor multiplied, so a short last tile costs what its rows cost
  const int nb = min(max((u.rows - wm + 15) >> 4, 0), TM);

  if constexpr (NS == 2) {
    // Two stages: the next stage's wait, barrier, DMA issue (two stages ahead)
    // and first fragment reads sit in the middle of the current stage's second
    // 64-code step, which runs from registers (as in gemm_dma_kernel). Packed
    // weights are read once per stage, in lane group l4 chunk l4 of their row
    // (codes 32 l4 .. 32 l4 + 31): step h takes its half h, with activation
    // chunk 2 l4 + h.
    auto read_w = [&](const int8_t* st, int ks, int a) {
      return *reinterpret_cast<const v4i*>(st + BM * RBA + tile_off<RBW>(wn + 16 * a + l16, kI4 ? l4 : 4 * ks + l4));
    };
    auto read_a = [&](const int8_t* st, int ks, int b) {
      return *reinterpret_cast<const v4i*>(st + tile_off<RBA>(wm + 16 * b + l16, kI4 ? 2 * l4 + ks : 4 * ks + l4));
    };
    constexpr int kFreeW = TM > TN ? TN : TM - 1;  // the fragment after which all weights have been read
    wait_vmcnt<0>();
    stage_barrier();
    // `full` (every fragment has rows) is a type, so that its loop has no branch
    // between the reads and MFMAs: at a branch the compiler waits for whatever
    // either side may have in flight.
    auto stages = [&](auto full) __attribute__((always_inline)) {
      v4i wf[TN], af[TM], nwf[TN], naf[TM];
#pragma unroll
      for (int a = 0; a < TN; ++a) wf[a] = read_w(smem, 0, a);
#pragma unroll
      for (int b = 0; b < 2 && b < TM; ++b) af[b] = read_a(smem, 0, b);
      __builtin_amdgcn_sched_barrier(0);
      issue_w(1, 1);
      issue_a(1, 1);
      __builtin_amdgcn_sched_barrier(0);
      for (int kt = 0; kt < KT; ++kt) {
        const int8_t* st = smem + (kt & 1) * kStageBytes;
        if constexpr (kI4) {
#pragma unroll
          for (int a = 0; a < TN; ++a) {
            nwf[a] = wf[a];
            wf[a] = unpack16(nwf[a].x, nwf[a].y);
          }
        }
#pragma unroll
        for (int b = 0; b < TM; ++b) {
          if (full.value || b < nb) {
            const v4i x = kI4 ? even_odd_bytes(af[b]) : af[b];
#pragma unroll
            for (int a = 0; a < TN; ++a) acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[a], x, acc[a][b], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (b + 2 < TM) af[b + 2] = read_a(st, 0, b + 2);
            naf[b] = read_a(st, 1, b);
          }
          // step 1's weights: one per fragment, the rest with the last one
#pragma unroll
          for (int a = b; a < TN && (a == b || b == TM - 1); ++a) {
            if constexpr (kI4) nwf[a] = unpack16(nwf[a].z, nwf[a].w);
            else nwf[a] = read_w(st, 1, a);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (b == kFreeW) {
            __builtin_amdgcn_s_waitcnt(0xC07F);
            stage_barrier();                      // everyone has read stage kt's weights
            issue_w(kt + 2, kt & 1);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        constexpr int kHalf = TM / 2;
#pragma unroll
        for (int b = 0; b < kHalf; ++b)
          if (full.value || b < nb) {
            const v4i x = kI4 ? even_odd_bytes(naf[b]) : naf[b];
#pragma unroll
            for (int a = 0; a < TN; ++a) acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(nwf[a], x, acc[a][b], 0, 0, 0);
          }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);       // own reads of stage kt returned
        if (kt + 1 < KT) {
          wait_vmcnt<kIW>();                      // stage kt+1 landed (own DMA)
          stage_barrier();                        // everyone's: stage kt+1 ready, stage kt free
          issue_a(kt + 2, kt & 1);                // past the end: zeros that nobody reads
          const int8_t* sn = smem + ((kt + 1) & 1) * kStageBytes;
#pragma unroll
          for (int a = 0; a < TN; ++a) wf[a] = read_w(sn, 0, a);
#pragma unroll
          for (int b = 0; b < 2 && b < TM; ++b) af[b] = read_a(sn, 0, b);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = kHalf; b < TM; ++b)
          if (full.value || b < nb) {
            const v4i x = kI4 ? even_odd_bytes(naf[b]) : naf[b];
#pragma unroll
            for (int a = 0; a < TN; ++a) acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(nwf[a], x, acc[a][b], 0, 0, 0);
          }
      }
    };
    if (nb == TM) stages(std::true_type{});
    else stages(std::false_type{});
  } else {
  int cur = 0, nxt = NS - 1;                             // buffers of stage kt and of stage kt + NS - 1
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<(NS - 2) * LPS>();
    stage_barrier();
    issue_a(kt + NS - 1, nxt);                           // past the end: zeros that nobody reads
    issue_w(kt + NS - 1, nxt);
    const int8_t* sa_ = smem + cur * kStageBytes;
    const int8_t* sw_ = sa_ + BM * RBA;
    nxt = cur;
    cur = cur + 1 == NS ? 0 : cur + 1;
    if constexpr (!kI4) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        v4i wf[TN], af[TM];
#pragma unroll
        for (int a = 0; a < TN; ++a)
          wf[a] = *reinterpret_cast<const v4i*>(sw_ + tile_off<RBW>(wn + 16 * a + l16, 4 * ks + l4));
#pragma unroll
        for (int b = 0; b < TM; ++b)
          af[b] = *reinterpret_cast<const v4i*>(sa_ + tile_off<RBA>(wm + 16 * b + l16, 4 * ks + l4));
#pragma unroll
        for (int b = 0; b < TM; ++b)
          if (TM == 1 || b < nb) {
#pragma unroll
            for (int a = 0; a < TN; ++a)
              acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[a], af[b], acc[a][b], 0, 0, 0);
          }
      }
    } else {
      // lane group l4 holds packed chunk l4 of its weight row (codes 32 l4 ..
      // 32 l4 + 31); half h of it pairs with activation chunk 2 l4 + h. The
      // codes come out times 16 (unpack16).
      v4i wraw[TN];
#pragma unroll
      for (int a = 0; a < TN; ++a)
        wraw[a] = *reinterpret_cast<const v4i*>(sw_ + tile_off<RBW>(wn + 16 * a + l16, l4));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4i wf[TN], af[TM];
#pragma unroll
        for (int a = 0; a < TN; ++a) wf[a] = h ? unpack16(wraw[a].z, wraw[a].w) : unpack16(wraw[a].x, wraw[a].y);
#pragma unroll
        for (int b = 0; b < TM; ++b)
          af[b] = even_odd_bytes(*reinterpret_cast<const v4i*>(sa_ + tile_off<RBA>(wm + 16 * b + l16, 2 * l4 + h)));
#pragma unroll
        for (int b = 0; b < TM; ++b)
          if (TM == 1 || b < nb) {
#pragma unroll
            for (int a = 0; a < TN; ++a)
              acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[a], af[b], acc[a][b], 0, 0, 0);
          }
      }
    }
  }
  }
  if constexpr (kI4) {
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] >>= 4;
  }
  wait_vmcnt<0>();

  // Four consecutive outputs of fragment (a, b) as 8 bytes: a is the output
  // fragment, which for the gated product holds weight fragments 2a and 2a + 1.
  const float* const lsa = lsc;
  const float* const lsw = lsc + BM;
  auto out4 = [&](int a, int b, float sam) -> uint2 {
    if constexpr (GATED) {
      const f4 gt = scaled4(acc[2 * a][b], sam, *reinterpret_cast<const float4*>(lsw + wn + 32 * a + 4 * l4));
      const f4 up = scaled4(acc[2 * a + 1][b], sam, *reinterpret_cast<const float4*>(lsw + wn + 32 * a + 16 + 4 * l4));
      f4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = silu_mul(gt[r], up[r]);
      if constexpr (BF) return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf4));
      else return __builtin_bit_cast(uint2, __builtin_convertvector(v, h4));
    } else {
      const float4 sw4 = *reinterpret_cast<const float4*>(lsw + wn + 16 * a + 4 * l4);
      if constexpr (BF) return __builtin_bit_cast(uint2, dequant4_bf(acc[a][b], sam, sw4));
      else return __builtin_bit_cast(uint2, dequant4(acc[a][b], sam, sw4));
    }
  };
  const int wno = GATED ? wn / 2 : wn;                   // the wave's first output column in the tile
  uint16_t* const Y = static_cast<uint16_t*>(g.y);

  if ((NO & 7) == 0) {
    // through LDS as whole 16-byte row chunks with nontemporal stores, pass p
    // taking the same fragment rows of every wave (as in gemm_dma_kernel)
    constexpr int CPR = BNO / 8;
    constexpr int kIt = (R * CPR + NW * 64 - 1) / (NW * 64);
    stage_barrier();                                     // every wave is done with the operand stages
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int bl = 0; bl < TM / NP; ++bl) {
        const int b = p * (TM / NP) + bl;
        const int r0 = (wave / WGN) * RB + 16 * bl;
        const float sam = lsa[wm + 16 * b + l16];
#pragma unroll
        for (int a = 0; a < TNO; ++a)
          *reinterpret_cast<uint2*>(smem + (r0 + l16) * kRowB + (wno + 16 * a + 4 * l4) * 2) = out4(a, b, sam);
      }
      lds_write_barrier();
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int f = (i * NW + wave) * 64 + lane;
        const int row = f / CPR, ch = f - row * CPR;
        const int m = (row / RB) * WTM + p * RB + row % RB, n = n0 + ch * 8;
        if (f < R * CPR && m < u.rows && n < NO)
          __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(smem + row * kRowB + ch * 16),
                                      reinterpret_cast<v4i*>(Y + (int64_t)(u.m0 + m) * NO + n));
      }
      if (p + 1 < NP) stage_barrier();
    }
    return;
  }
  // Rows that are not whole 16-byte chunks: single elements straight from the
  // fragments. Few rows do not feel it (308 int4 rows of 1003 or 1008 columns 9.0
  // us); 32768 rows of 2047 columns with K = 1024 take 180 us, of 2048 95.
#pragma unroll
  for (int b = 0; b < TM; ++b) {
    const int m = wm + 16 * b + l16;
    if (m >= u.rows) continue;
    const float sam = lsa[m];
#pragma unroll
    for (int a = 0; a < TNO; ++a) {
      const int n = n0 + wno + 16 * a + 4 * l4;
      const uint2 o = out4(a, b, sam);
      uint16_t* dst = Y + (int64_t)(u.m0 + m) * NO + n;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < NO) dst[r] = (uint16_t)((r < 2 ? o.x : o.y) >> (16 * (r & 1)));
    }
  }
}

// Tile choice. Only P and the number of experts are known here, not the group
// sizes: an expert is taken to end in half a tile. Up to 8 rows per expert the
// weights are read for so few rows that bytes in flight count (three blocks
// of four stages per CU); above, a launch of T tiles with bpc blocks to a CU runs
// about ceil(T / (256 bpc)) rounds of bpc * BM * BN * cost, and the cheapest is
// taken. `cost` (time per tile element and round, relative) was measured on
// 4096 rows times [12288, 2048] with one expert: 256 x 256 93 us, 256 x 192
// 101, 128 x 256 117, 64 x 128 154. Measured against forcing each tile: 192
// rows over 64 experts of 2048 x 2048 43.5 us (32 x 64; 64 x 128 45.2, 16 x 64
// 47.0, 256 x 256 54), 4096 rows 55.1 (64 x 128; 128 x 256 66, 32 x 64 78,
// 256 x 256 69), 8192 rows 65.9 (128 x 256; 256 x 192 75, 256 x 256 82), 32768
// rows 159 (256 x 256; 256 x 192 177, 128 x 256 182), 3000 rows over 8 experts
// of 2560 x 2560 27.7 (256 x 192; 256 x 256 33, 128 x 256 41).
struct Tile {
  int bm, bn, threads, cost, bpc;
};
constexpr Tile kTiles[] = {{32, 64, 256, 0, 3}, {64, 128, 512, 100, 3}, {128, 256, 512, 78, 1}, {256, 192, 512, 67, 1},
                           {256, 256, 512, 62, 1}};

inline int pick_tile(const GroupedArgs& g, bool gated) {
  const int64_t experts = std::min<int64_t>(g.E, g.P);
  if (g.P <= 8 * experts) return 0;
  int best = 1;
  int64_t best_est = 0;
  for (int i = 1; i < 5; ++i) {
    const Tile& t = kTiles[i];
    const int64_t no = gated ? g.N / 2 : g.N, bno = gated ? t.bn / 2 : t.bn;
    const int64_t tiles = (2 * g.P + experts * t.bm) * ((no + bno - 1) / bno) / (2 * t.bm);
    const int64_t est = std::max<int64_t>(1, (tiles + 256 * t.bpc - 1) / (256 * t.bpc)) * t.bpc * t.bm * t.bn * t.cost;
    if (i == 1 || est < best_est) {
      best = i;
      best_est = est;
    }
  }
  return best;
}

// Blocks of the launch: the longest possible list of work units, whole rounds over the XCDs.
inline int64_t grid_blocks(const GroupedArgs& g, int bm, int bno, int64_t no) {
  const int64_t units = (g.P / bm + std::min<int64_t>(g.E, g.P)) * ((no + bno - 1) / bno);
  return (units + 7) / 8 * 8;
}

template <int T, int WGM, int WGN, int NS, int WK, bool BF, bool GATED>
hipError_t launch_tile(const GroupedArgs& g, hipStream_t st) {
  constexpr int BM = kTiles[T].bm, BN = kTiles[T].bn;
  static_assert(WGM * WGN * 64 == kTiles[T].threads, "tile table");
  const int64_t blocks = grid_blocks(g, BM, GATED ? BN / 2 : BN, GATED ? g.N / 2 : g.N);
  grouped_kernel<BM, BN, WGM, WGN, NS, WK, BF, GATED><<<dim3((unsigned)blocks), dim3(WGM * WGN * 64), 0, st>>>(g);
  return hipGetLastError();
}

template <int WK, bool BF, bool GATED>
hipError_t launch_t(const GroupedArgs& g, hipStream_t st) {
  switch (pick_tile(g, GATED)) {
    case 0: return launch_tile<0, 2, 2, 4, WK, BF, GATED>(g, st);
    case 1: return launch_tile<1, 2, 4, 2, WK, BF, GATED>(g, st);
    case 2: return launch_tile<2, 2, 4, 2, WK, BF, GATED>(g, st);
    case 3: return launch_tile<3, 4, 2, 2, WK, BF, GATED>(g, st);
    default: return launch_tile<4, 2, 4, 2, WK, BF, GATED>(g, st);
  }
}

template <int WK>
hipError_t launch_wk(const GroupedArgs& g, bool bf16, bool gated, hipStream_t st) {
  if (bf16) return gated ? launch_t<WK, true, true>(g, st) : launch_t<WK, true, false>(g, st);
  return gated ? launch_t<WK, false, true>(g, st) : launch_t<WK, false, false>(g, st);
}

}  // namespace

bool grouped_launch_fits(const GroupedArgs& g, bool gated) {
  const Tile& t = kTiles[pick_tile(g, gated)];
  return grid_blocks(g, t.bm, gated ? t.bn / 2 : t.bn, gated ? g.N / 2 : g.N) < (int64_t(1) << 31) / t.threads;
}

hipError_t launch_grouped(const GroupedArgs& args, WeightKind wk, bool bf16, bool gated, hipStream_t stream) {
  GroupedArgs g = args;
  if (g.row_index && g.row_div > 1) {
    int l = 1;
    while ((int64_t(1) << l) < g.row_div) ++l;
    g.div_mul = (uint32_t)(((uint64_t(1) << (31 + l)) + g.row_div - 1) / g.row_div);
    g.div_shift = l - 1;
  }
  return wk == kWeightI4 ? launch_wk<kWeightI4>(g, bf16, gated, stream) : launch_wk<kWeightI8>(g, bf16, gated, stream);
}

}  // namespace cider
