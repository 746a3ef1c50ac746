// Rotary positions of q or k rows: y = x with the first rotary_dim dimensions
// of each head turned by its token's position (cider_rope.h).
//
// HBM-bound: 2 bytes in and 2 out per element (16384 tokens of 24 heads of 128: 201
// MB in 39.4 us = 5.1 TB/s, a copy's rate). One workgroup per token (and
// slice of its heads): its threads first form the token's rotary_dim / 2
// cosines and sines into LDS, shared by all heads; other workgroups' rows are on
// their way meanwhile. A thread then owns both ends of the pairs it turns, so y may be x.
#include "cider_internal.h"
#include "cider_quant_rule.h"
#include "cider_rope.h"
#include "cider_rows.h"

namespace cider {
namespace {

constexpr int kThreads = 256;

// One item = what one thread turns or copies of one head:
//   half layout, 16-byte chunks: pair of chunks (c, c + rd / 16), c < rd / 16;
//       then the chunks behind rd, one each
//   interleaved: one chunk of 8 (4 pairs, or fewer at rd's end, or none)
template <bool BF, bool INTERLEAVED, bool PAST>
__global__ void __launch_bounds__(kThreads) rope_rows(RopeArgs a) {
  __shared__ float2 turn[kMaxRotaryPairs];
  const int64_t t = blockIdx.x;
  const int pairs = a.rotary_dim / 2, chunks = a.head_dim / 8;
  const int per_head = INTERLEAVED ? chunks : chunks - pairs / 8;
  const int items = a.heads * per_head;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.x_row_stride;
  uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.y_row_stride;
  const int32_t pos = a.positions[t];
  for (int i = threadIdx.x; i < pairs; i += kThreads) turn[i] = rope_turn(pos, a.inv_freq[i], a.scale);
  __syncthreads();
  for (int item = blockIdx.y * kThreads + threadIdx.x; item < items; item += gridDim.y * kThreads) {
    const int head = item / per_head, c = item - head * per_head;
    const uint16_t* xh = x + head * a.x_head_stride;
    uint16_t* yh = y + head * a.y_head_stride;
    if constexpr (INTERLEAVED) {
      float v[8];
      unpack8<BF>(load16(xh, c), v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * c + e;
        if (i < pairs) rope_pair(v[2 * e], v[2 * e + 1], turn[i]);
      }
      store16_to<PAST>(yh, c, pack8<BF>(v));
    } else {
      const int step = pairs / 8;
      if (c < step) {
        float u[8], w[8];
        unpack8<BF>(load16(xh, c), u);
        unpack8<BF>(load16(xh, c + step), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) rope_pair(u[e], w[e], turn[8 * c + e]);
        store16_to<PAST>(yh, c, pack8<BF>(u));
        store16_to<PAST>(yh, c + step, pack8<BF>(w));
      } else {
        store16_to<PAST>(yh, c + step, load16(xh, c + step));
      }
    }
  }
}

// Any even rotary_dim, head size and strides: one pair, or one dimension
// behind rd, per thread.
template <bool BF>
__global__ void __launch_bounds__(kThreads) rope_elements(RopeArgs a) {
  __shared__ float2 turn[kMaxRotaryPairs];
  const int64_t t = blockIdx.x;
  const int pairs = a.rotary_dim / 2, per_head = a.head_dim - pairs;
  const int items = a.heads * per_head;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.x_row_stride;
  uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.y_row_stride;
  const int32_t pos = a.positions[t];
  for (int i = threadIdx.x; i < pairs; i += kThreads) turn[i] = rope_turn(pos, a.inv_freq[i], a.scale);
  __syncthreads();
  for (int item = blockIdx.y * kThreads + threadIdx.x; item < items; item += gridDim.y * kThreads) {
    const int head = item / per_head, i = item - head * per_head;
    const uint16_t* xh = x + head * a.x_head_stride;
    uint16_t* yh = y + head * a.y_head_stride;
    if (i < pairs) {
      const int iu = a.interleaved ? 2 * i : i, iw = a.interleaved ? 2 * i + 1 : i + pairs;
      float u = elem_to_float<BF>(xh[iu]), w = elem_to_float<BF>(xh[iw]);
      rope_pair(u, w, turn[i]);
      yh[iu] = round16<BF>(u);
      yh[iw] = round16<BF>(w);
    } else {
      yh[i + pairs] = xh[i + pairs];
    }
  }
}

bool whole_chunks(const RopeArgs& a) {
  const auto whole = [](int64_t v) { return v % 8 == 0; };
  return whole(a.head_dim) && whole(a.x_row_stride) && whole(a.x_head_stride) && whole(a.y_row_stride) &&
         whole(a.y_head_stride) && (a.interleaved || a.rotary_dim % 16 == 0);
}

// Workgroups per token: a slice of its items each.
int64_t slices(const RopeArgs& a) {
  const int pairs = a.rotary_dim / 2;
  const int per_head = !whole_chunks(a) ? a.head_dim - pairs : a.interleaved ? a.head_dim / 8 : a.head_dim / 8 - pairs / 8;
  return ((int64_t)a.heads * per_head + kThreads - 1) / kThreads;
}

template <bool BF, bool PAST>
void launch_rope_rows(const RopeArgs& a, dim3 grid, hipStream_t st) {
  if (a.interleaved) rope_rows<BF, true, PAST><<<grid, dim3(kThreads), 0, st>>>(a);
  else rope_rows<BF, false, PAST><<<grid, dim3(kThreads), 0, st>>>(a);
}

template <bool BF>
hipError_t launch_rope_t(const RopeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.T, (unsigned)slices(a));
  if (!whole_chunks(a)) rope_elements<BF><<<grid, dim3(kThreads), 0, st>>>(a);
  else if (2 * a.T * a.heads * a.head_dim >= kPastCacheBytes) launch_rope_rows<BF, true>(a, grid, st);
  else launch_rope_rows<BF, false>(a, grid, st);
  return hipGetLastError();
}

}  // namespace

bool rope_fits(const RopeArgs& a) { return a.T * slices(a) * kThreads < (int64_t(1) << 31) && slices(a) < 65536; }

hipError_t launch_rope(const RopeArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_rope_t<true>(a, stream) : launch_rope_t<false>(a, stream);
}

}  // namespace cider
