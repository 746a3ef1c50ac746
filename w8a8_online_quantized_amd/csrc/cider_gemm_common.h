// Device helpers shared by the GEMM translation units (the dense kernels and
// the products grouped by expert): vector types, the dequant arithmetic, the
// int4 unpacking, and the global -> LDS staging primitives.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cider {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4i zero4() { return v4i{0, 0, 0, 0}; }

// The lane index recomputed where it is used (mbcnt), so that no register
// holds it across a long loop.
__device__ __forceinline__ int lane_id() { return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)); }

// Per-channel dequant of one element: fp16(fp32(fp32(acc) * s_a) * s_w), each
// product rounded to fp32 before the round-to-nearest-even fp16 conversion.
// The empty asm pins the second product as an fp32 register value: without it
// the backend fuses that multiply with the conversion into v_fma_mixlo_f16
// (even with contraction off), whose result differs from the two-step
// rounding in rare cases.
__device__ __forceinline__ _Float16 dequant1(int32_t acc, float sa, float sw) {
  float t = (float)acc * sa;
  t = t * sw;
  asm("" : "+v"(t));
  return (_Float16)t;
}

// fp16(fp32(t * s)): a finished fp32 sum times one scale (two roundings, as above).
__device__ __forceinline__ _Float16 scale1(float t, float s) {
  t = t * s;
  asm("" : "+v"(t));
  return (_Float16)t;
}

// Four consecutive outputs of one row (the same rounding as dequant1).
__device__ __forceinline__ h4 dequant4(v4i acc, float sa, float4 sw) {
  float4 t;
  t.x = ((float)acc.x * sa) * sw.x;
  t.y = ((float)acc.y * sa) * sw.y;
  t.z = ((float)acc.z * sa) * sw.z;
  t.w = ((float)acc.w * sa) * sw.w;
  asm("" : "+v"(t.x), "+v"(t.y), "+v"(t.z), "+v"(t.w));
  typedef float f4 __attribute__((ext_vector_type(4)));
  return __builtin_convertvector(f4{t.x, t.y, t.z, t.w}, h4);
}

// The same two fp32 roundings with a bfloat16 output (round to nearest even).
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __bf16 dequant1_bf(int32_t acc, float sa, float sw) {
  float t = (float)acc * sa;
  t = t * sw;
  asm("" : "+v"(t));
  return (__bf16)t;
}

__device__ __forceinline__ bf4 dequant4_bf(v4i acc, float sa, float4 sw) {
  float4 t;
  t.x = ((float)acc.x * sa) * sw.x;
  t.y = ((float)acc.y * sa) * sw.y;
  t.z = ((float)acc.z * sa) * sw.z;
  t.w = ((float)acc.w * sa) * sw.w;
  asm("" : "+v"(t.x), "+v"(t.y), "+v"(t.z), "+v"(t.w));
  typedef float f4 __attribute__((ext_vector_type(4)));
  return __builtin_convertvector(f4{t.x, t.y, t.z, t.w}, bf4);
}

// A finished fp32 value to bfloat16.
__device__ __forceinline__ __bf16 to_bf16(float t) {
  asm("" : "+v"(t));
  return (__bf16)t;
}

// bf16(fp32(t * s)): a finished fp32 sum times one scale, two roundings.
__device__ __forceinline__ __bf16 scale1_bf(float t, float s) {
  t = t * s;
  asm("" : "+v"(t));
  return (__bf16)t;
}

// Reorder 16 activation codes (4 dwords, K order 0..15) into the order the
// unpacked int4 weights come in: 0,2,4,6 | 1,3,5,7 | 8,10,12,14 | 9,11,13,15.
__device__ __forceinline__ v4i even_odd_bytes(v4i v) {
  v4i o;
  o.x = (int)__builtin_amdgcn_perm((uint32_t)v.y, (uint32_t)v.x, 0x06040200u);
  o.y = (int)__builtin_amdgcn_perm((uint32_t)v.y, (uint32_t)v.x, 0x07050301u);
  o.z = (int)__builtin_amdgcn_perm((uint32_t)v.w, (uint32_t)v.z, 0x06040200u);
  o.w = (int)__builtin_amdgcn_perm((uint32_t)v.w, (uint32_t)v.z, 0x07050301u);
  return o;
}

// Nibbles u in [0, 15] of four bytes -> signed codes u - 8 in each byte,
// without carries between bytes: ((u | 0x80) - 8) ^ 0x80.
__device__ __forceinline__ uint32_t nib_to_code(uint32_t u) {
  return ((u | 0x80808080u) - 0x08080808u) ^ 0x80808080u;
}

__device__ __forceinline__ v4i unpack_int4(uint2 p) {
  v4i o;
  o.x = (int)nib_to_code(p.x & 0x0F0F0F0Fu);
  o.y = (int)nib_to_code((p.x >> 4) & 0x0F0F0F0Fu);
  o.z = (int)nib_to_code(p.y & 0x0F0F0F0Fu);
  o.w = (int)nib_to_code((p.y >> 4) & 0x0F0F0F0Fu);
  return o;
}

// ---------------------------------------------------------------------------
// Direct-to-LDS pipeline (per-channel and W4A8).
//
// Each stage moves BK codes of every tile row from global memory straight
// into LDS with buffer_load_dwordx4 ... lds (one wave instruction fills one
// contiguous KiB of LDS), NS stages deep, so the loads of stage k+NS-1 are in
// flight while the MFMAs of stage k run. The buffer descriptor covers exactly
// the valid rows of the tile; chunks past K get an out-of-range offset, so
// every out-of-bounds element arrives as 0 without a branch. Stage order is
// kept with s_waitcnt vmcnt (own loads) followed by s_barrier (everyone's).
// ---------------------------------------------------------------------------

// Physical 16-byte slot of logical chunk c in tile row r, for rows of RB bytes.
// Both XOR patterns were chosen by measurement on gfx950 (64 LDS banks): with
// them the MFMA fragment reads (16 consecutive rows per 16-lane group for the
// 16x16x64 shape, 32 rows per 32-lane group for 32x32x32) complete in 4
// cycles per ds_read_b128 with no bank-conflict cycles, while e.g. c ^ (r & 3)
// on 64-byte rows or c ^ (r & 7) on 128-byte rows take 8 for some of them.
template <int RB>
__device__ __forceinline__ int slot_of(int r, int c) {
  if constexpr (RB == 64) return c ^ ((r >> 1) & 3);
  else return c ^ ((r >> 1) & 7);
}

template <int RB>
__device__ __forceinline__ int tile_off(int r, int c) { return r * RB + (slot_of<RB>(r, c) << 4); }

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  // dword 3 = 0x00020000: raw buffer, 32-bit data format (gfx9 family)
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// DMA instructions each wave issues per stage for a ROWS x RB-byte tile.
template <int ROWS, int RB, int NW>
constexpr int dma_per_wave() {
  static_assert(ROWS * RB % 1024 == 0, "a stage tile is a whole number of 1 KiB blocks");
  return (ROWS * RB / 1024 + NW - 1) / NW;
}

// Issue the DMA loads of one stage of a ROWS x RB-byte operand tile. Block j
// of 1 KiB holds rows j*(1024/RB) ...; lane L writes LDS bytes L*16..L*16+15
// of its block, i.e. physical slot L % (RB/16) of block row L / (RB/16). When
// the blocks do not split evenly over the NW waves, a wave with no block left
// issues a zero-fill load (out-of-range offset) into the 1 KiB `pad`, so that
// every wave issues the same number of DMA instructions per stage and one
// s_waitcnt vmcnt count fits all waves. `wave` must be wave-uniform.
template <int ROWS, int RB, int NW>
__device__ __forceinline__ void dma_stage(__amdgpu_buffer_rsrc_t rsrc, int8_t* lds, int8_t* pad, int wave,
                                          int lane, uint32_t ld, int kb0, int kb_total) {
  constexpr int kBlocks = ROWS * RB / 1024;
  constexpr int kSlots = RB / 16;
  constexpr int kRowsPerBlock = 1024 / RB;
#pragma unroll
  for (int i = 0; i < dma_per_wave<ROWS, RB, NW>(); ++i) {
    const int j = wave + i * NW;
    const int r = j * kRowsPerBlock + lane / kSlots;
    const int p = lane % kSlots;
    const int c = slot_of<RB>(r, p);          // the XOR swizzle is an involution
    const int kb = kb0 + c * 16;
    uint32_t off = kb < kb_total ? (uint32_t)r * ld + (uint32_t)kb : 0x80000000u;
    int8_t* dst = lds + j * 1024;
    if constexpr (kBlocks % NW != 0) {
      if (j >= kBlocks) {
        off = 0x80000000u;
        dst = pad;
      }
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)dst, 16, off, 0, 0, 0);
  }
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  // gfx9 s_waitcnt: vmcnt[3:0] | expcnt[6:4]=7 | lgkmcnt[11:8]=15 | vmcnt[5:4] at [15:14]
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// stage_barrier after this wave's LDS writes have landed (lgkmcnt(0)): the
// barrier alone does not wait for them
__device__ __forceinline__ void lds_write_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  stage_barrier();
}

}  // namespace
}  // namespace cider
