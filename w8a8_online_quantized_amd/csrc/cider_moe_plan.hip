// The routing plan of an expert block: a stable counting sort of the tokens'
// expert ids. P = T * top_k ids give offsets[e] (how many kept ids are below
// e), rows (the flat indexes t * top_k + j sorted by expert, equal experts in
// index order) and slots (each flat index's place in that order; -1 when its
// id lies outside [0, E) and it belongs to no expert).
//
// A wave owns a contiguous range of ids and walks it twice, 64 at a time: once
// to count them in LDS, once to place them. Within the 64, the lanes with the
// same id are found by ballots over the id's bits (~log2 E of them): a lane's
// rank among them is the number of set bits below it, and the lowest of them
// advances the wave's counter by the group's size. Nothing depends on the order
// of atomics: sums of integers, and counters that belong to one wave, combined
// in wave (and block) order.
//
// Latency-bound at decode sizes, so one workgroup does everything in one
// launch up to kOneBlockIds ids; beyond, a first launch counts each block's
// ids and a second one places them, every block summing the counts of the
// blocks before it by itself. Kernel times (HIP events): 128 ids 3.4-3.9 us (an
// empty launch 3.5), 4096 ids 5.9, 8192 ids 8.5, 262144 ids 11.5 (3.1 MB; two
// launches, the second of which counts its ids again, and scattered 4-byte
// stores bound it).
#include "cider_internal.h"

namespace cider {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
// One launch or two. The kernels alone cross near 6500 ids (64 experts, one /
// two: 4096 ids 5.9 / 7.7 us, 6144 7.2 / 7.7, 8192 8.5 / 7.8; 512 experts, 8192
// ids: 10.1 / 10.5), but two launches also need a workspace: 8192 ids from
// Python take 8.9 / 13.2 us among others and 24.4 / 25.9 alone.
constexpr int kOneBlockIds = 8192;
constexpr int kMaxBlocks = 256;

struct PlanShape {
  int blocks;
  int64_t chunk;   // ids per block, a multiple of kThreads
};

// Ids per block: 2048, or 4096 with many experts, whose counts every block adds
// up (262144 ids: 128 experts 11.7 us with 2048, 12.3 with 4096; 512 experts
// 20.3 and 16.4).
inline PlanShape plan_shape(int64_t P, int E) {
  if (P <= kOneBlockIds) return {1, (P + kThreads - 1) / kThreads * kThreads};
  int64_t chunk = (E <= 256 ? 2 : 4) * kThreads;
  if (P > chunk * kMaxBlocks) chunk = ((P + kMaxBlocks - 1) / kMaxBlocks + kThreads - 1) / kThreads * kThreads;
  return {(int)((P + chunk - 1) / chunk), chunk};
}

// The lanes of this wave whose id equals this lane's, among those with `ok`:
// per bit of the id, a ballot and m & ~(ballot ^ (bit ? ~0 : 0)) on each half.
__device__ __forceinline__ uint64_t same_id(int id, bool ok, int bits) {
  const uint64_t all = __ballot(ok);
  uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
  for (int b = 0; b < bits; ++b) {
    const int mine = -((id >> b) & 1);
    const uint64_t v = __ballot(mine != 0);
    lo &= ~((uint32_t)v ^ (uint32_t)mine);
    hi &= ~((uint32_t)(v >> 32) ^ (uint32_t)mine);
  }
  return (uint64_t)hi << 32 | lo;
}

// Calls step(i, id, ok) for the wave's share of ids [first, last), 64 at a
// time in order; ok: the id names an expert. kAhead loads are in flight before
// the first is used.
constexpr int kAhead = 8;
template <class Step>
__device__ __forceinline__ void for_ids(const int32_t* __restrict__ ids, int64_t first, int64_t last, int E, int wave,
                                        int lane, Step step) {
  const int64_t per = (last - first + kWaves * 64 - 1) / (kWaves * 64) * 64;
  const int64_t lo = first + wave * per, hi = min(last, lo + per);
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = i0 + 64 * j + lane;
      id[j] = i < hi ? ids[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + 64 * j >= hi) break;                                       // uniform
      step(i0 + 64 * j + lane, id[j], id[j] >= 0 && id[j] < E);
    }
  }
}

// Each wave's ids counted into cnt[wave][e]; `first` and `last` bound the block's range.
__device__ __forceinline__ void count_ids(const int32_t* __restrict__ ids, int64_t first, int64_t last, int E,
                                          int* cnt, int wave, int lane) {
  for_ids(ids, first, last, E, wave, lane, [&](int64_t, int id, bool ok) {
    if (ok) atomicAdd(&cnt[wave * E + id], 1);   // integers: the order of the adds does not show
  });
}

__global__ void __launch_bounds__(kThreads) plan_count(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
                                                       int32_t* __restrict__ ws) {
  extern __shared__ int cnt[];   // [kWaves][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kWaves * E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = min(P, first + chunk);
  count_ids(ids, first, last, E, cnt, wave, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) n += cnt[w * E + e];
    ws[(int64_t)blockIdx.x * E + e] = n;
  }
}

// ws: every block's counts [blocks][E], or null when this is the only block.
__global__ void __launch_bounds__(kThreads) plan_place(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
                                                       int bits, const int32_t* __restrict__ ws,
                                                       int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                       int32_t* __restrict__ slots) {
  extern __shared__ int cnt[];   // [kWaves][E], one sum per wave, then two partial sums per thread
  int* const wsum = cnt + kWaves * E;
  int* const part_before = wsum + kWaves;
  int* const part_total = part_before + kThreads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kWaves * E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = min(P, first + chunk);
  count_ids(ids, first, last, E, cnt, wave, lane);
  // the other blocks' counts, each thread a part of the blocks for one expert
  // (one memory latency instead of one for every 8 blocks: 262144 ids over 128
  // experts 15.3 -> 13.3 us)
  const int parts = kThreads / E;
  if (ws) {
    const int part = threadIdx.x / E, pe = threadIdx.x % E;
    const int per = ((int)gridDim.x + parts - 1) / parts;
    const int b0 = part * per, b1 = min((int)gridDim.x, b0 + per);
    int before = 0, total = 0;
    if (part < parts) {
#pragma unroll 16
      for (int b = b0; b < b1; ++b) {
        const int n = ws[(int64_t)b * E + pe];
        if (b < (int)blockIdx.x) before += n;
        total += n;
      }
    }
    part_before[threadIdx.x] = before;
    part_total[threadIdx.x] = total;
  }
  __syncthreads();

  // thread e: the ids of expert e in the blocks before this one and in all
  const int e = threadIdx.x;
  int before = 0, total = 0;
  if (e < E) {
    if (ws) {
      for (int p = 0; p < parts; ++p) {
        before += part_before[p * E + e];
        total += part_total[p * E + e];
      }
    } else {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += cnt[w * E + e];
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
    int at = start + before, n[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) n[w] = cnt[w * E + e];   // all in flight before the first is overwritten
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {                        // counts become each wave's first place
      cnt[w * E + e] = at;
      at += n[w];
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = kept;
  __syncthreads();

  for_ids(ids, first, last, E, wave, lane, [&](int64_t i, int id, bool ok) {
    const uint64_t m = same_id(id, ok, bits);
    const uint64_t below = m & ((1ull << lane) - 1);
    int base = 0;
    if (ok && below == 0) base = atomicAdd(&cnt[wave * E + id], __popcll(m));
    base = __shfl(base, ok ? __builtin_ctzll(m) : lane);
    const int place = base + __popcll(below);
    if (i < last) {
      slots[i] = ok ? place : -1;
      if (ok) rows[place] = (int32_t)i;
      if (i >= kept) rows[i] = -1;       // places no id takes
    }
  });
}

}  // namespace

int64_t moe_plan_workspace_bytes(int64_t P, int E) {
  const PlanShape s = plan_shape(P, E);
  return s.blocks > 1 ? (int64_t)s.blocks * E * 4 : 0;
}

hipError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* rows, int32_t* slots,
                           void* ws, hipStream_t stream) {
  const PlanShape s = plan_shape(P, E);
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  const size_t lds = (size_t)(kWaves * E + kWaves + 2 * kThreads) * 4;   // at most 41 KB
  int32_t* counts = s.blocks > 1 ? static_cast<int32_t*>(ws) : nullptr;
  if (counts) {
    plan_count<<<dim3((unsigned)s.blocks), dim3(kThreads), lds, stream>>>(ids, P, s.chunk, E, counts);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  plan_place<<<dim3((unsigned)s.blocks), dim3(kThreads), lds, stream>>>(ids, P, s.chunk, E, bits, counts, offsets, rows,
                                                                       slots);
  return hipGetLastError();
}

}  // namespace cider
