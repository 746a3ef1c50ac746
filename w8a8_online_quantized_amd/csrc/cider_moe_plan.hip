// The routing plan of an expert block: a stable counting sort of the tokens'
// expert ids. P = T * top_k ids give offsets[e] (how many kept ids are below
// e), rows (the flat indexes t * top_k + j sorted by expert, equal experts in
// index order) and slots (each flat index's place in that order; -1 when its
// id lies outside [0, E) and it belongs to no expert).
//
// A wave owns a contiguous range of ids and walks it 64 at a time. Within
// the 64, the lanes with the same id are found by ballots over the id's bits
// (one per bit, so ~log2 E): a lane's rank among them is the number of set
// bits below it, and the lowest of them adds the group's size to the wave's
// counter in LDS. Nothing depends on the order of atomics: a counter belongs
// to one wave, and counters are combined in wave (and block) order.
//
// Latency-bound at decode sizes, so one workgroup does everything in one
// launch up to kOneBlockIds ids; beyond, a first launch counts each block's
// ids and a second one places them, every block summing the counts of the
// blocks before it by itself.
#include "cider_internal.h"

namespace cider {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kOneBlockIds = 8192;
constexpr int kMaxBlocks = 256;

struct PlanShape {
  int blocks;
  int64_t chunk;   // ids per block, a multiple of kThreads
};

inline PlanShape plan_shape(int64_t P) {
  if (P <= kOneBlockIds) return {1, (P + kThreads - 1) / kThreads * kThreads};
  int64_t chunk = 2 * kThreads;
  if (P > chunk * kMaxBlocks) chunk = ((P + kMaxBlocks - 1) / kMaxBlocks + kThreads - 1) / kThreads * kThreads;
  return {(int)((P + chunk - 1) / chunk), chunk};
}

// The lanes of this wave whose id equals this lane's, among those with `ok`.
__device__ __forceinline__ uint64_t same_id(int id, bool ok, int bits) {
  uint64_t m = __ballot(ok);
  for (int b = 0; b < bits; ++b) {
    const uint64_t v = __ballot((id >> b) & 1);
    m &= (id >> b) & 1 ? v : ~v;
  }
  return m;
}

// Each wave's ids counted into cnt[wave][e]; `first` and `last` bound the block's range.
__device__ __forceinline__ void count_ids(const int32_t* __restrict__ ids, int64_t first, int64_t last, int E, int bits,
                                          int* cnt, int wave, int lane) {
  const int64_t per = (last - first + kWaves * 64 - 1) / (kWaves * 64) * 64;
  const int64_t lo = first + wave * per, hi = min(last, lo + per);
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const int id = i < hi ? ids[i] : -1;
    const bool ok = id >= 0 && id < E;
    const uint64_t m = same_id(id, ok, bits);
    if (ok && (m & ((1ull << lane) - 1)) == 0) atomicAdd(&cnt[wave * E + id], __popcll(m));
  }
}

__global__ void __launch_bounds__(kThreads) plan_count(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
                                                       int bits, int32_t* __restrict__ ws) {
  extern __shared__ int cnt[];   // [kWaves][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kWaves * E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = min(P, first + chunk);
  count_ids(ids, first, last, E, bits, cnt, wave, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int n = 0;
    for (int w = 0; w < kWaves; ++w) n += cnt[w * E + e];
    ws[(int64_t)blockIdx.x * E + e] = n;
  }
}

// ws: every block's counts [blocks][E], or null when this is the only block.
__global__ void __launch_bounds__(kThreads) plan_place(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
                                                       int bits, const int32_t* __restrict__ ws,
                                                       int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                       int32_t* __restrict__ slots) {
  extern __shared__ int cnt[];   // [kWaves][E], then one sum per wave
  int* const wsum = cnt + kWaves * E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kWaves * E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = min(P, first + chunk);
  count_ids(ids, first, last, E, bits, cnt, wave, lane);
  __syncthreads();

  // thread e: the ids of expert e in this block, before it and in all
  const int e = threadIdx.x;
  int own = 0, before = 0, total = 0;
  if (e < E) {
    for (int w = 0; w < kWaves; ++w) own += cnt[w * E + e];
    total = own;
    if (ws) {
      total = 0;
#pragma unroll 8
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int n = ws[(int64_t)b * E + e];
        if (b < (int)blockIdx.x) before += n;
        total += n;
      }
    }
  }
  // exclusive scan of `total` over the experts
  int incl = total;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int start = incl - total, kept = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) start += wsum[w];
    kept += wsum[w];
  }
  if (e < E) {
    if (blockIdx.x == 0) offsets[e] = start;
    int at = start + before;
    for (int w = 0; w < kWaves; ++w) {   // counts become each wave's first place
      const int n = cnt[w * E + e];
      cnt[w * E + e] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = kept;
  __syncthreads();

  const int64_t per = (last - first + kWaves * 64 - 1) / (kWaves * 64) * 64;
  const int64_t lo = first + wave * per, hi = min(last, lo + per);
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const int id = i < hi ? ids[i] : -1;
    const bool ok = id >= 0 && id < E;
    const uint64_t m = same_id(id, ok, bits);
    const uint64_t below = m & ((1ull << lane) - 1);
    int base = 0;
    if (ok && below == 0) base = atomicAdd(&cnt[wave * E + id], __popcll(m));
    base = __shfl(base, ok ? __builtin_ctzll(m) : lane);
    const int place = base + __popcll(below);
    if (i < hi) {
      slots[i] = ok ? place : -1;
      if (ok) rows[place] = (int32_t)i;
      if (i >= kept) rows[i] = -1;       // places no id takes
    }
  }
}

}  // namespace

int64_t moe_plan_workspace_bytes(int64_t P, int E) {
  const PlanShape s = plan_shape(P);
  return s.blocks > 1 ? (int64_t)s.blocks * E * 4 : 0;
}

hipError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* rows, int32_t* slots,
                           void* ws, hipStream_t stream) {
  const PlanShape s = plan_shape(P);
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  const size_t lds = (size_t)(kWaves * E + kWaves) * 4;
  int32_t* counts = s.blocks > 1 ? static_cast<int32_t*>(ws) : nullptr;
  if (counts) {
    plan_count<<<dim3((unsigned)s.blocks), dim3(kThreads), lds, stream>>>(ids, P, s.chunk, E, bits, counts);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  plan_place<<<dim3((unsigned)s.blocks), dim3(kThreads), lds, stream>>>(ids, P, s.chunk, E, bits, counts, offsets, rows,
                                                                       slots);
  return hipGetLastError();
}

}  // namespace cider
