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
#include "sort_rows.h"

namespace moe {

// ---------------------------------------------------------------------- sort
// (sort_rows.h)
__global__ __launch_bounds__(kSortThreads) void moe_sort_one_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  sort_one<false>(a, cnt, sh, base);
}
__global__ __launch_bounds__(kSortThreads) void moe_sort_count_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  sort_count<false>(a, cnt);
}
__global__ __launch_bounds__(kSortThreads) void moe_sort_place_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  sort_place<false>(a, cnt, sh, base);
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

void plan_sort(SortArgs* a) {
  a->chunks = sort_chunks(a->picks);
  a->steps = sort_steps(a->picks);
  a->bits = 0;
  while ((1 << a->bits) < a->groups) a->bits++;
}

hipError_t launch_sort(SortArgs a, hipStream_t stream) {
  plan_sort(&a);
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
