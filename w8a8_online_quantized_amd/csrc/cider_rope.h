// Rotary positions, shared by the rotation alone and by the cache's writer.
//
// A pair (u, w) of a token at position p turns by the angle a = p * f_i:
//   u' = scale * (u cos a - w sin a),   w' = scale * (w cos a + u sin a).
// The angle is formed and reduced to one turn in 64 bits: at p = 10^6 an fp32
// product is off by up to 0.03 rad, the fp64 one by 10^-10. The remainder,
// within half a turn, goes to the fp32 sine and cosine of half turns (one
// rounding of 2^-25 turns, 1.9e-7 rad, before the functions' own).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cider {

// Pairs of a head that one workgroup holds in its LDS table (rotary_dim / 2).
constexpr int kMaxRotaryPairs = 256;

// (scale * cos, scale * sin) of position * inv_freq.
__device__ __forceinline__ float2 rope_turn(int32_t position, double inv_freq, float scale) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double turns = (double)position * inv_freq * kInvTwoPi;
  const float part = (float)(turns - rint(turns));   // [-1/2, 1/2] turns
  float s, c;
  sincospif(2.0f * part, &s, &c);
  return make_float2(c * scale, s * scale);
}

// The pair turned, as finished fp32 values: the empty asm keeps the backend
// from fusing them with a conversion to fp16 into one rounding, which bf16 does
// not have and another kernel's code might not get.
__device__ __forceinline__ void rope_pair(float& u, float& w, float2 cs) {
  float p = __builtin_fmaf(u, cs.x, -(w * cs.y)), q = __builtin_fmaf(w, cs.x, u * cs.y);
  asm("" : "+v"(p), "+v"(q));
  u = p;
  w = q;
}

// One end of a pair turned, `other` being the other end and `sine` negated at the
// first one: the same products and sum as rope_pair, so the same bits.
__device__ __forceinline__ float rope_end(float own, float other, float cosine, float sine) {
  float p = __builtin_fmaf(own, cosine, other * sine);
  asm("" : "+v"(p));
  return p;
}

}  // namespace cider
