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
  float* v;            // [k_parts][rows][max_rank] partial sums of A x
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

// Rows and adapters of a block's epilogue: sv[row][j] = scale * (A x)_j, the
// K parts added in part order, 0 past the adapter's rank and for rows without
// an adapter.  Called by every thread of the block, which then synchronises.
__device__ __forceinline__ void lora_load_v(const LoraArgs& l, int rows, float* sv, int tid,
                                            int threads) {
  for (int i = tid; i < rows * l.max_rank; i += threads) {
    const int r = i / l.max_rank, j = i - r * l.max_rank;
    const int id = l.ids[r];
    float s = 0.f;
    if ((uint32_t)id < (uint32_t)l.adapters && j < lora_rank(l, id)) {
      for (int p = 0; p < l.k_parts; p++) s += l.v[((size_t)p * l.rows + r) * l.max_rank + j];
      s *= l.scale[id];
    }
    sv[i] = s;
  }
}

// sum_j B[n, j] v[j] over the adapter's ranks (8 at a time: the ranks past
// the adapter's are masked, whatever they hold).
__device__ __forceinline__ float lora_dot(const LoraArgs& l, int adapter, int rank, int n,
                                          const float* v) {
  const uint16_t* b = l.b + ((size_t)adapter * l.n + n) * l.max_rank;
  float s = 0.f;
  for (int j = 0; j < rank; j += 8) {
    const u32x4 u = ld16(b + j);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float f = __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
      s = j + i < rank ? fmaf(f, v[j + i], s) : s;
    }
  }
  return s;
}

// What row r's adapter adds at output n, from the block's sv.
__device__ __forceinline__ float lora_term(const LoraArgs& l, int r, int n, const float* sv) {
  const int id = l.ids[r];
  if ((uint32_t)id >= (uint32_t)l.adapters) return 0.f;
  return lora_dot(l, id, lora_rank(l, id), n, sv + r * l.max_rank);
}

// The GEMVs' epilogue beside adapters (LORA) or without: sv is kSv floats
// of the block's LDS, filled by load() before a barrier.
template <bool LORA>
struct GemvTail {
  static constexpr int kSv = 1;
  __device__ __forceinline__ void load(int, float*, int, int) const {}
  __device__ __forceinline__ float add(float v, int, int, const float*) const { return v; }
};
template <>
struct GemvTail<true> {
  static constexpr int kSv = kMaxRows * kLoraMaxRank;
  LoraArgs l;
  __device__ __forceinline__ void load(int rows, float* sv, int tid, int threads) const {
    lora_load_v(l, rows, sv, tid, threads);
  }
  __device__ __forceinline__ float add(float v, int r, int n, const float* sv) const {
    return v + lora_term(l, r, n, sv);
  }
};

// The workspace of a call: its size, and its parts in *l at base (rows,
// adapters, max_rank, n and k of *l set).
size_t lora_plan(LoraArgs* l, void* base);
hipError_t launch_lora_shrink(const LoraArgs& l, const uint16_t* x, hipStream_t stream);
hipError_t launch_lora(LoraArgs l, const uint16_t* x, const uint16_t* base, uint16_t* y,
                       hipStream_t stream);

}  // namespace moe
