// lora.h -- low-rank adapters of many requests: host interface of lora.hip
// and the term that the GEMVs add to a projection's output (device).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.h"
#include "token_rows.h"

namespace moe {

constexpr int kLoraTile = 32;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = kSortMaxGroups - 1;  // and a group of the rows without one

// Adapter i: A [max_rank, k] and B [n, max_rank] (bf16), its first rank[i]
// ranks (all of max_rank without rank) used, times scale[i].
struct LoraArgs {
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* rank;
  const float* scale;
  const int32_t* ids;  // [rows] adapter of each row; outside [0, adapters): none
  int adapters, max_rank, n, k, rows;
  // scale A x of each row [rows][max_rank] (0 past the adapter's rank); with
  // rows grouped, A x by sorted row, [k_parts][rows][max_rank] partial sums
  float* v;
  int k_parts;
  // many rows: grouped by adapter, in tiles of kLoraTile rows (v by sorted row)
  int32_t *order, *pos, *offsets, *counts, *n_tiles;
  RowTile* tiles;
  int max_tiles;
};

__device__ __forceinline__ int lora_rank(const LoraArgs& l, int adapter) {
  if (!l.rank) return l.max_rank;
  const int r = l.rank[adapter];
  return r < 0 ? 0 : (r < l.max_rank ? r : l.max_rank);
}

// What a block's epilogue needs of its rows' adapters, in LDS: id (-1: none),
// ranks used, and v = scale A x (lora_shrink_kernel's).  load() is called by
// every thread of the block, which then synchronises.
struct LoraRows {
  float v[kMaxRows * kLoraMaxRank];
  int id[kMaxRows], rank[kMaxRows];
  __device__ __forceinline__ void load(const LoraArgs& l, int rows, int tid, int threads) {
    for (int i = tid; i < rows * l.max_rank; i += threads) v[i] = l.v[i];
    if (tid < rows) {
      const int i = l.ids[tid];
      const bool on = (uint32_t)i < (uint32_t)l.adapters;
      id[tid] = on ? i : -1;
      rank[tid] = on ? lora_rank(l, i) : 0;
    }
  }
  // What the adapter of row r, which has one, adds at output n: sum_j B[n, j]
  // v[j] over its ranks, 8 at a time; B past them is not used, whatever it holds.
  __device__ __forceinline__ float term(const LoraArgs& l, int r, int n) const {
    const int i = id[r], rk = rank[r];
    const uint16_t* b = l.b + ((size_t)i * l.n + n) * l.max_rank;
    const float* vr = v + r * l.max_rank;
    float s = 0.f;
    for (int j = 0; j < rk; j += 8) {
      const u32x4 u = ld16(b + j);
#pragma unroll
      for (int q = 0; q < 8; q++) {
        const float f = __uint_as_float(q & 1 ? u[q >> 1] & 0xFFFF0000u : u[q >> 1] << 16);
        s = j + q < rk ? fmaf(f, vr[j + q], s) : s;
      }
    }
    return s;
  }
};

// The GEMVs' epilogue beside adapters (LORA) or without: Rows is its part of
// the block's LDS, filled by load() before a barrier.  The term reads B's row
// after the sum it joins, one latency: at rank 16 [9728, 2560] of 1 bit takes
// 5.8 us with it and 4.5 without at 1 row, 9.3 and 7.9 at 8; [6144, 6144] of
// FP8 12.1 and 9.4, of bf16 17.6 and 14.6.  A pass of its own over y would
// cost a launch and round twice.
struct NoLoraRows {};
template <bool LORA>
struct GemvTail {
  using Rows = NoLoraRows;
  __device__ __forceinline__ void load(Rows&, int, int, int) const {}
  __device__ __forceinline__ float add(float v, int, int, const Rows&) const { return v; }
};
template <>
struct GemvTail<true> {
  using Rows = LoraRows;
  LoraArgs l;
  __device__ __forceinline__ void load(Rows& rows, int n_rows, int tid, int threads) const {
    rows.load(l, n_rows, tid, threads);
  }
  __device__ __forceinline__ float add(float v, int r, int n, const Rows& rows) const {
    return rows.id[r] < 0 ? v : v + rows.term(l, r, n);  // (-0 + 0 would be 0)
  }
};

// The workspace of a call: its size, and its parts in *l at base (rows,
// adapters, max_rank, n and k of *l set).
size_t lora_plan(LoraArgs* l, void* base);
hipError_t launch_lora_shrink(const LoraArgs& l, const uint16_t* x, hipStream_t stream);
hipError_t launch_lora(LoraArgs l, const uint16_t* x, const uint16_t* base, uint16_t* y,
                       hipStream_t stream);

}  // namespace moe
