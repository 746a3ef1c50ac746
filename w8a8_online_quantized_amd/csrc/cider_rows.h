// 16-bit rows in registers, shared by the kernels that read and write them:
// 16-byte loads and stores of global memory, and eight values to and from fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cider {
namespace {

template <bool BF>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// 16 bytes at chunk c of a global buffer. (Pointers that arrive in a struct
// would give flat loads, one dword each where they are conditional.)
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) u4 global_u4;

__device__ __forceinline__ u4 load16(const void* base, int64_t c) { return ((const global_u4*)base)[c]; }
__device__ __forceinline__ void store16(void* base, int64_t c, u4 v) { ((global_u4*)base)[c] = v; }

// Stores of results that the last-level cache (256 MB) would not keep for their
// reader anyway go past it: rotating 16384 tokens of 24 heads of 128 (100 MB in, 100
// out) 47.7 -> 39.4 us. Smaller ones stay for the next launch. (A kernel has one or
// the other: of two stores behind a branch the compiler makes one ordinary store.)
constexpr int64_t kPastCacheBytes = int64_t(64) << 20;
template <bool PAST>
__device__ __forceinline__ void store16_to(void* base, int64_t c, u4 v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, (global_u4*)base + c);
  else store16(base, c, v);
}

// Eight values at once, as vectors: the conversions then come in pairs.
typedef float f8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

template <bool BF>
__device__ __forceinline__ u4 pack8(const float (&v)[8]) {
  const f8 t{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  if constexpr (BF) return __builtin_bit_cast(u4, __builtin_convertvector(t, b8));
  else return __builtin_bit_cast(u4, __builtin_convertvector(t, h8));
}

template <bool BF>
__device__ __forceinline__ void unpack8(u4 q, float (&v)[8]) {
  if constexpr (BF) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  } else {
    const f8 t = __builtin_convertvector(__builtin_bit_cast(h8, q), f8);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t[i];
  }
}

}  // namespace
}  // namespace cider
