// sort_rows.h -- device parts of the stable sort by group (token_rows.hip) and of
// reading and writing rows of bf16 or fp32.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "token_rows.h"

namespace moe {

// ---------------------------------------------------------------------- sort
// A block takes a chunk of 1024 x steps picks, its 16 waves 64 x steps
// consecutive ones each.  A wave ranks 64 picks at a time: ballots over the
// id's bits give each lane the lanes with its id, so the lanes below it are
// its rank among them, and the lowest of them adds their number to the wave's
// count of that id in LDS (one wave's own row: its LDS operations complete in
// order).  The exclusive sums over the waves' counts, group by group, then
// turn the ranks into places.  Bound by the latency of that chain, not by its
// bytes (4 read and 8 written a pick): 128 picks of 256 groups 3.8 us, 6001 of
// 25 groups 7.6 us in one block, 65536 of 256 in two launches 4.7 + 8 us.  Every
// block of the second reads all chunks' counts: little up to some 2^20 picks (31
// us of 256 groups), most of the time at the 2^24 that it takes (0.8 ms of 256
// groups, 1.7 of 1024).
constexpr int kSortWaves = kSortThreads / kWave;

struct SortShared {
  int2 scan[kSortWaves];
};

// Exclusive sums of v's parts over the block's threads, and the block's
// totals.
__device__ __forceinline__ int2 block_scan(int2 v, SortShared& sh, int tid, int2* total) {
  const int lane = tid & 63, wv = tid >> 6;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int x = __shfl_up(s.x, o, kWave), y = __shfl_up(s.y, o, kWave);
    if (lane >= o) {
      s.x += x;
      s.y += y;
    }
  }
  if (lane == 63) sh.scan[wv] = s;
  __syncthreads();
  int2 before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < kSortWaves; w++) {
    const int2 t = sh.scan[w];
    before.x += w < wv ? t.x : 0;
    before.y += w < wv ? t.y : 0;
    all.x += t.x;
    all.y += t.y;
  }
  *total = all;
  return int2{before.x + s.x - v.x, before.y + s.y - v.y};
}

// The group of pick i, which is `id`'s, -1 for none; in a sort by a digit of the
// id the digit of one that is kept.
template <bool DIGIT>
__device__ __forceinline__ int group_of(const SortArgs& a, int id, bool there) {
  if constexpr (DIGIT) return there && (uint32_t)id < (uint32_t)a.ids_below ? (id >> a.shift) & ((1 << a.bits) - 1) : -1;
  const int other = a.spill ? a.groups - 1 : -1;
  const int e = (uint32_t)id < (uint32_t)(a.groups - a.spill) ? id : other;
  return there ? e : -1;
}

// The block's picks: id (or -1) and rank among the wave's picks of that id;
// cnt [waves][groups] ends as the waves' counts.
template <bool DIGIT>
__device__ __forceinline__ void rank_chunk(const SortArgs& a, int chunk, uint16_t* cnt, int tid,
                                           int (&id)[kSortSteps], int (&rk)[kSortSteps]) {
  const int lane = tid & 63, wv = tid >> 6;
  const int64_t i0 = (int64_t)chunk * (kSortThreads * a.steps) + (int64_t)wv * (kWave * a.steps) + lane;
  const int64_t there = DIGIT && a.by ? (a.kept ? *a.kept : a.kept_here) : a.picks;
  // the loads carry no condition of the lane's (past the last pick they repeat
  // it), so that all of them are under way at once
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    id[s] = -1;
    if (s >= a.steps) continue;
    const int64_t i = i0 + 64 * s;
    int64_t at = i < a.picks ? i : a.picks - 1;
    if (DIGIT && a.by) at = i < there ? a.by[i] : 0;
    id[s] = a.ids[at];
  }
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    id[s] = group_of<DIGIT>(a, id[s], s < a.steps && i0 + 64 * s < there);
  }
  for (int i = tid; i < kSortWaves * a.groups; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  uint16_t* mine = cnt + wv * a.groups;
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    if (s >= a.steps) continue;
    const int e = id[s];
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < a.bits; b++) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    if (e >= 0) {
      const int below = lanes_below(same);
      rk[s] = mine[e] + below;
      // every lane of the id has read the count before the lowest adds to it
      asm volatile("" ::: "memory");
      if (below == 0) mine[e] = (uint16_t)(rk[s] + __popcll(same));
      asm volatile("" ::: "memory");
    }
  }
  __syncthreads();
}

// Pick i goes to place p (-1: to none).
template <bool DIGIT>
__device__ __forceinline__ void put_place(const SortArgs& a, int64_t i, int p) {
  if constexpr (DIGIT) {
    if (p >= 0) a.order[p] = a.by ? a.by[i] : (int)i;
  } else {
    a.pos[i] = p;
    if (p >= 0) a.order[p] = (int)i;
  }
}

// Tiles of a group with `count` rows.
__device__ __forceinline__ int tiles_of(const SortArgs& a, int count) {
  return a.tiles ? (count + a.tile_rows - 1) / a.tile_rows : 0;
}

// The tiles covering every group's rows, in group order, and behind them those
// of the extra rows [picks, picks + extra).  Threads below `groups` hold their
// group's first row, rows and first tile; `routed` is the groups' tiles.
__device__ __forceinline__ void write_tiles(const SortArgs& a, int first, int count, int at,
                                            int routed, int tid) {
  if (!a.tiles) return;
  for (int i = 0; i * a.tile_rows < count; i++)
    a.tiles[at + i] = RowTile{tid, first + i * a.tile_rows, first + count};
  const int more = a.extra > 0 ? (a.extra + a.extra_rows - 1) / a.extra_rows : 0;
  for (int i = tid; i < more; i += kSortThreads)
    a.tiles[routed + i] = RowTile{a.groups, (int)a.picks + i * a.extra_rows, (int)a.picks + a.extra};
  if (tid == 0) *a.n_tiles = routed + more;
}

// One chunk: the whole sort in one block (E <= 1024 = a group a thread).
// Returns the picks in a group.
template <bool DIGIT>
__device__ __forceinline__ int sort_one(const SortArgs& a, uint16_t* cnt, SortShared& sh, int32_t* base) {
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk<DIGIT>(a, 0, cnt, tid, id, rk);
  int total = 0;
  if (tid < a.groups) {
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) {
      const int c = cnt[w * a.groups + tid];
      cnt[w * a.groups + tid] = (uint16_t)total;
      total += c;
    }
  }
  int2 all;
  const int2 at = block_scan(int2{total, tiles_of(a, total)}, sh, tid, &all);
  const int first = at.x;
  if (tid < a.groups) {
    base[tid] = first;
    a.offsets[tid] = first;
    if (tid == a.groups - 1) a.offsets[a.groups] = first + total;
  }
  __syncthreads();
  const int lane = tid & 63, wv = tid >> 6;
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    const int64_t i = (int64_t)wv * (kWave * a.steps) + lane + 64 * s;
    if (s < a.steps && i < a.picks) {
      const int p = id[s] >= 0 ? base[id[s]] + cnt[wv * a.groups + id[s]] + rk[s] : -1;
      put_place<DIGIT>(a, i, p);
    }
  }
  write_tiles(a, first, total, at.y, all.y, tid);
  return all.x;
}

// More chunks: each chunk's counts [chunk][group], ...
template <bool DIGIT>
__device__ __forceinline__ void sort_count(const SortArgs& a, uint16_t* cnt) {
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk<DIGIT>(a, blockIdx.x, cnt, tid, id, rk);
  for (int g = tid; g < a.groups; g += kSortThreads) {
    int total = 0;
    for (int w = 0; w < kSortWaves; w++) total += cnt[w * a.groups + g];
    a.counts[(size_t)blockIdx.x * a.groups + g] = total;
  }
}

// ... and the places, every block summing the counts it needs: of its group
// over the chunks before its own, and of the groups before over all chunks.
template <bool DIGIT>
__device__ __forceinline__ void sort_place(const SortArgs& a, uint16_t* cnt, SortShared& sh, int32_t* base) {
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk<DIGIT>(a, blockIdx.x, cnt, tid, id, rk);
  int before = 0, total = 0;
  if (tid < a.groups) {
    for (int c0 = 0; c0 < a.chunks; c0 += 16) {  // 16 loads under way at once
      int n[16];
#pragma unroll
      for (int c = 0; c < 16; c++)
        n[c] = a.counts[(size_t)(c0 + c < a.chunks ? c0 + c : a.chunks - 1) * a.groups + tid];
#pragma unroll
      for (int c = 0; c < 16; c++) {
        before += c0 + c < (int)blockIdx.x ? n[c] : 0;
        total += c0 + c < a.chunks ? n[c] : 0;
      }
    }
    int w0 = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) {
      const int c = cnt[w * a.groups + tid];
      cnt[w * a.groups + tid] = (uint16_t)w0;
      w0 += c;
    }
  }
  int2 all;
  const int2 at = block_scan(int2{total, tiles_of(a, total)}, sh, tid, &all);
  const int first = at.x;
  if (tid < a.groups) {
    base[tid] = first + before;
    if (blockIdx.x == 0) {
      a.offsets[tid] = first;
      if (tid == a.groups - 1) a.offsets[a.groups] = first + total;
    }
  }
  __syncthreads();
  const int lane = tid & 63, wv = tid >> 6;
  const int64_t i0 = (int64_t)blockIdx.x * (kSortThreads * a.steps) + (int64_t)wv * (kWave * a.steps) + lane;
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    const int64_t i = i0 + 64 * s;
    if (s < a.steps && i < a.picks) {
      const int p = id[s] >= 0 ? base[id[s]] + cnt[wv * a.groups + id[s]] + rk[s] : -1;
      put_place<DIGIT>(a, i, p);
    }
  }
  if (blockIdx.x == 0) write_tiles(a, first, total, at.y, all.y, tid);
}

// -------------------------------------------------------------- rows
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, uint16_t& o) { o = f32_to_bf16(v); }

// Elements c .. c + V (those below n) of a row, as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int c, int n, float (&f)[V]) {
  if constexpr (V > 1) {
    if (c + V <= n) {
      const u32x4_a4 u = *reinterpret_cast<const u32x4_a4*>(row + c);
#pragma unroll
      for (int i = 0; i < V; i++) {
        if constexpr (sizeof(T) == 4)
          f[i] = __uint_as_float(u[i]);
        else
          f[i] = __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i++) f[i] = c + i < n ? to_f32(row[c + i]) : 0.f;
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* row, int c, int n, const float (&f)[V]) {
  if constexpr (V > 1) {
    if (c + V <= n) {
      u32x4_a4 u;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4)
          u[i] = __float_as_uint(f[i]);
        else
          u[i] = (uint32_t)f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
      }
      *reinterpret_cast<u32x4_a4*>(row + c) = u;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i++)
    if (c + i < n) from_f32(f[i], row[c + i]);
}

}  // namespace moe
