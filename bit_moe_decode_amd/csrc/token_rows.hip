// token_rows.hip -- tokens sorted by expert and back: the stable sort of a
// batch's picks, the gather of the tokens' rows into sorted order, the
// weighted combination of the sorted rows back into token order, and the
// gradients of both movements.
//
// With ids [T, k] (the picks; flat pick i = t k + j) and E groups:
//   sort      order = the flat picks with 0 <= id < E by (id, i), offsets[e] =
//             the picks with an id below e, pos = order's inverse (-1 for a
//             pick that is in no group)
//   gather    xs[pos[t,j]] = x[t]
//     its gradient     dx[t] = sum_j dxs[pos[t,j]]
//   combine   out[t] = sum_j g[t,j] y[pos[t,j]] (+ add[t])
//     its gradients    dy[pos[t,j]] = g[t,j] dout[t],
//                      dg[t,j] = sum_h dout[t,h] y[pos[t,j],h]
// All sums run in fp32 in pick order, and are rounded once.
#include "token_rows.h"

#include "device_common.h"

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

// The block's picks: id (or -1) and rank among the wave's picks of that id;
// cnt [waves][groups] ends as the waves' counts.
__device__ __forceinline__ void rank_chunk(const SortArgs& a, int chunk, uint16_t* cnt, int tid,
                                           int (&id)[kSortSteps], int (&rk)[kSortSteps]) {
  const int lane = tid & 63, wv = tid >> 6;
  const int64_t i0 = (int64_t)chunk * (kSortThreads * a.steps) + (int64_t)wv * (kWave * a.steps) + lane;
  const int other = a.spill ? a.groups - 1 : -1;
  // the loads carry no condition of the lane's (past the last pick they repeat
  // it), so that all of them are under way at once
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    id[s] = -1;
    if (s >= a.steps) continue;
    const int64_t i = i0 + 64 * s;
    id[s] = a.ids[i < a.picks ? i : a.picks - 1];
  }
#pragma unroll
  for (int s = 0; s < kSortSteps; s++) {
    const int e = (uint32_t)id[s] < (uint32_t)(a.groups - a.spill) ? id[s] : other;
    id[s] = s < a.steps && i0 + 64 * s < a.picks ? e : -1;
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
__global__ __launch_bounds__(kSortThreads) void moe_sort_one_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk(a, 0, cnt, tid, id, rk);
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
      a.pos[i] = p;
      if (p >= 0) a.order[p] = (int)i;
    }
  }
  write_tiles(a, first, total, at.y, all.y, tid);
}

// More chunks: each chunk's counts [chunk][group], ...
__global__ __launch_bounds__(kSortThreads) void moe_sort_count_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk(a, blockIdx.x, cnt, tid, id, rk);
  for (int g = tid; g < a.groups; g += kSortThreads) {
    int total = 0;
    for (int w = 0; w < kSortWaves; w++) total += cnt[w * a.groups + g];
    a.counts[(size_t)blockIdx.x * a.groups + g] = total;
  }
}

// ... and the places, every block summing the counts it needs: of its group
// over the chunks before its own, and of the groups before over all chunks.
__global__ __launch_bounds__(kSortThreads) void moe_sort_place_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  const int tid = threadIdx.x;
  int id[kSortSteps], rk[kSortSteps];
  rank_chunk(a, blockIdx.x, cnt, tid, id, rk);
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
      a.pos[i] = p;
      if (p >= 0) a.order[p] = (int)i;
    }
  }
  if (blockIdx.x == 0) write_tiles(a, first, total, at.y, all.y, tid);
}

// Picks a thread: all of them in one block up to kSortChunk picks; above that
// two launches, of at least 2 picks a thread and blocks enough that 32 of them
// hold the picks, up to 8 a thread (32768 picks of 256 groups: 10.7 + 13.6 us
// in 4 blocks of 8 a thread).
static int sort_steps(int64_t picks) {
  if (picks <= kSortChunk) return (int)((picks + kSortThreads - 1) / kSortThreads);
  const int64_t s = picks / (32 * kSortThreads);
  return s < 2 ? 2 : (s > kSortSteps ? kSortSteps : (int)s);
}
static int sort_chunks(int64_t picks) {
  const int64_t per = (int64_t)kSortThreads * sort_steps(picks);
  return picks > 0 ? (int)((picks + per - 1) / per) : 0;
}

size_t sort_workspace(int64_t picks, int groups) {
  const int c = sort_chunks(picks);
  return c > 1 ? (size_t)c * groups * sizeof(int32_t) : 0;
}

hipError_t launch_sort(SortArgs a, hipStream_t stream) {
  a.chunks = sort_chunks(a.picks);
  a.steps = sort_steps(a.picks);
  a.bits = 0;
  while ((1 << a.bits) < a.groups) a.bits++;
  const size_t lds = (size_t)kSortWaves * a.groups * sizeof(uint16_t);  // at most 32 KB
  if (a.chunks <= 1) {
    hipLaunchKernelGGL(moe_sort_one_kernel, dim3(1), dim3(kSortThreads), lds, stream, a);
  } else {
    hipLaunchKernelGGL(moe_sort_count_kernel, dim3(a.chunks), dim3(kSortThreads), lds, stream, a);
    hipLaunchKernelGGL(moe_sort_place_kernel, dim3(a.chunks), dim3(kSortThreads), lds, stream, a);
  }
  return hipGetLastError();
}

// -------------------------------------------------------------- row movement
// Rows are taken 16 bytes a lane where every row starts on a 4-byte boundary
// (gfx950 loads and stores 16 bytes at any dword alignment), element by
// element otherwise (an odd number of bf16).  All of them are bound by memory:
// a row is read once and written once, several rows under way a lane, a row's
// blocks next to each other so that its lines are used while they are open.
// At 6144 columns: gather of 8192 tokens to 65536 rows of bf16 170 us, 5.3
// TB/s; combine of 8191 tokens' 2 of 8 picks (those of a quarter of the experts)
// in fp32 109 us, 5.5 TB/s; combine's gradient of 4096 tokens in bf16 168 us,
// gather's 110 us.  A few rows take the launch
// and one pass of latency: 16 tokens gathered 3.5 us, 32 combined 4.3 us.
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

// The rows of picks j0 .. j0 + 7 of token t: -1 for a pick without one, for
// one behind the buffer and past the last pick.  The eight loads carry no
// condition (past the last pick they repeat it), so they are under way at once.
__device__ __forceinline__ void pick_rows(const RowArgs& a, int64_t t, int j0, int (&p)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) p[j] = a.pos[t * a.top_k + (j0 + j < a.top_k ? j0 + j : a.top_k - 1)];
#pragma unroll
  for (int j = 0; j < 8; j++) p[j] = j0 + j < a.top_k && (uint32_t)p[j] < (uint32_t)a.rows ? p[j] : -1;
}
__device__ __forceinline__ void pick_gates(const RowArgs& a, const float* gates, int64_t t, int j0,
                                           float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++)
    w[j] = gates ? gates[t * a.top_k + (j0 + j < a.top_k ? j0 + j : a.top_k - 1)] : 1.f;
}

// xs[pos[t,j]] = x[t]: a block reads its part of one token's row once and
// writes it to the token's places.
template <typename T, int V>
__global__ void moe_gather_kernel(RowArgs a, const T* __restrict__ x, T* __restrict__ xs) {
  const int64_t t = a.first + blockIdx.x / a.parts;
  const int c = ((int)(blockIdx.x % a.parts) * (int)blockDim.x + (int)threadIdx.x) * V;
  if (c >= a.hidden) return;
  const T* row = x + t * a.hidden;
  const bool whole = V > 1 && c + V <= a.hidden;
  u32x4_a4 u = {0u, 0u, 0u, 0u};
  if (whole) u = *reinterpret_cast<const u32x4_a4*>(row + c);
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    int p[8];
    pick_rows(a, t, j0, p);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (p[j] < 0) continue;
      T* to = xs + (int64_t)p[j] * a.hidden;
      if (whole)
        *reinterpret_cast<u32x4_a4*>(to + c) = u;
      else
        for (int i = c; i < c + V && i < a.hidden; i++) to[i] = row[i];
    }
  }
}

// out[t] = sum_j w[t,j] y[pos[t,j]] (+ add[t]), w = 1 without gates.  The
// rows of up to 8 picks are in flight at once; a pick without a row is not
// read, and its gate not used.
template <typename T, int V>
__global__ void moe_combine_kernel_t(RowArgs a, const T* __restrict__ y,
                                     const float* __restrict__ gates, const T* __restrict__ add,
                                     T* __restrict__ out) {
  const int64_t t = a.first + blockIdx.x / a.parts;
  const int c = ((int)(blockIdx.x % a.parts) * (int)blockDim.x + (int)threadIdx.x) * V;
  if (c >= a.hidden) return;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; i++) acc[i] = 0.f;
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    int p[8];
    float w[8], f[8][V];
    pick_rows(a, t, j0, p);
    pick_gates(a, gates, t, j0, w);
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (p[j] >= 0) load_row<T, V>(y + (int64_t)p[j] * a.hidden, c, a.hidden, f[j]);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (p[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < V; i++) acc[i] = fmaf(w[j], f[j][i], acc[i]);
    }
  }
  if (add) {
    float f[V];
    load_row<T, V>(add + t * a.hidden, c, a.hidden, f);
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] += f[i];
  }
  store_row<T, V>(out + t * a.hidden, c, a.hidden, acc);
}

// dy and dgates of one token a block: dout[t] is read once for up to 8 picks,
// each lane keeps its part of their dots, which the waves then add.
template <typename T, int V>
__global__ __launch_bounds__(256) void moe_combine_bwd_kernel(
    RowArgs a, const T* __restrict__ dout, const T* __restrict__ y,
    const float* __restrict__ gates, T* __restrict__ dy, float* __restrict__ dgates) {
  __shared__ float part[4][8];
  const int64_t t = a.first + blockIdx.x;
  const int tid = threadIdx.x;
  const T* d = dout + t * a.hidden;
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    int p[8];
    float w[8], dot[8];
    pick_rows(a, t, j0, p);
    pick_gates(a, gates, t, j0, w);
#pragma unroll
    for (int j = 0; j < 8; j++) dot[j] = 0.f;
    for (int c = tid * V; c < a.hidden; c += 256 * V) {
      float f[V], v[8][V];
      load_row<T, V>(d, c, a.hidden, f);
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (p[j] >= 0) load_row<T, V>(y + (int64_t)p[j] * a.hidden, c, a.hidden, v[j]);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (p[j] < 0) continue;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
          dot[j] = fmaf(f[i], v[j][i], dot[j]);
          o[i] = w[j] * f[i];
        }
        store_row<T, V>(dy + (int64_t)p[j] * a.hidden, c, a.hidden, o);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      float s = dot[j];
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
      if ((tid & 63) == 0) part[tid >> 6][j] = s;
    }
    __syncthreads();
    if (tid < 8 && j0 + tid < a.top_k) {  // 0 for a pick without a row: its dots stayed 0
      dgates[t * a.top_k + j0 + tid] = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
    }
    __syncthreads();
  }
}

// Threads of a block (whole waves, at most 256); sets the blocks a row
// (consecutive ones, so that a row is read in one go) for `vec` elements a lane.
static int row_threads(RowArgs* a, int vec) {
  const int lanes = (a->hidden + vec - 1) / vec;
  const int threads = lanes >= 256 ? 256 : (lanes + 63) / 64 * 64;
  a->parts = (uint32_t)((lanes + threads - 1) / threads);
  return threads;
}

// Calls launch(blocks) for tokens from a->first on: one launch, or several of
// at most 2^23 blocks (2^31 threads) each.
template <typename F>
static hipError_t for_tokens(RowArgs* a, F launch) {
  const int64_t most = ((int64_t)1 << 23) / a->parts > 0 ? ((int64_t)1 << 23) / a->parts : 1;
  for (a->first = 0; a->first < a->tokens; a->first += most) {
    const int64_t n = a->tokens - a->first < most ? a->tokens - a->first : most;
    launch(dim3((uint32_t)(n * a->parts)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
static bool rows_on_dwords(const RowArgs& a) {
  return a.hidden * sizeof(T) % 4 == 0;
}

template <typename T, int V>
static hipError_t gather_v(RowArgs a, const void* x, void* xs, hipStream_t stream) {
  const int th = row_threads(&a, V);
  return for_tokens(&a, [&](dim3 g) {
    hipLaunchKernelGGL((moe_gather_kernel<T, V>), g, dim3(th), 0, stream, a, (const T*)x, (T*)xs);
  });
}
template <typename T, int V>
static hipError_t combine_v(RowArgs a, const void* y, const float* gates, const void* add, void* out,
                            hipStream_t stream) {
  const int th = row_threads(&a, V);
  return for_tokens(&a, [&](dim3 g) {
    hipLaunchKernelGGL((moe_combine_kernel_t<T, V>), g, dim3(th), 0, stream, a, (const T*)y, gates,
                       (const T*)add, (T*)out);
  });
}
template <typename T, int V>
static hipError_t combine_bwd_v(RowArgs a, const void* dout, const void* y, const float* gates,
                                void* dy, float* dgates, hipStream_t stream) {
  a.parts = 1;
  return for_tokens(&a, [&](dim3 g) {
    hipLaunchKernelGGL((moe_combine_bwd_kernel<T, V>), g, dim3(256), 0, stream, a, (const T*)dout,
                       (const T*)y, gates, (T*)dy, dgates);
  });
}

template <typename T>
static hipError_t gather_t(const RowArgs& a, const void* x, void* xs, hipStream_t stream) {
  return rows_on_dwords<T>(a) ? gather_v<T, kVec<T>>(a, x, xs, stream) : gather_v<T, 1>(a, x, xs, stream);
}
template <typename T>
static hipError_t combine_t(const RowArgs& a, const void* y, const float* gates, const void* add,
                            void* out, hipStream_t stream) {
  return rows_on_dwords<T>(a) ? combine_v<T, kVec<T>>(a, y, gates, add, out, stream)
                              : combine_v<T, 1>(a, y, gates, add, out, stream);
}
template <typename T>
static hipError_t combine_bwd_t(const RowArgs& a, const void* dout, const void* y,
                                const float* gates, void* dy, float* dgates, hipStream_t stream) {
  return rows_on_dwords<T>(a) ? combine_bwd_v<T, kVec<T>>(a, dout, y, gates, dy, dgates, stream)
                              : combine_bwd_v<T, 1>(a, dout, y, gates, dy, dgates, stream);
}

hipError_t launch_gather(const RowArgs& a, bool f32, const void* x, void* xs, hipStream_t stream) {
  return f32 ? gather_t<float>(a, x, xs, stream) : gather_t<uint16_t>(a, x, xs, stream);
}
hipError_t launch_combine_rows(const RowArgs& a, bool f32, const void* y, const float* gates,
                               const void* add, void* out, hipStream_t stream) {
  return f32 ? combine_t<float>(a, y, gates, add, out, stream)
             : combine_t<uint16_t>(a, y, gates, add, out, stream);
}
hipError_t launch_combine_bwd(const RowArgs& a, bool f32, const void* dout, const void* y,
                              const float* gates, void* dy, float* dgates, hipStream_t stream) {
  return f32 ? combine_bwd_t<float>(a, dout, y, gates, dy, dgates, stream)
             : combine_bwd_t<uint16_t>(a, dout, y, gates, dy, dgates, stream);
}

}  // namespace moe
