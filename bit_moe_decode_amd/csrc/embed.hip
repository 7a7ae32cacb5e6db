// embed.hip -- the embedding lookup with a scale and its gradient:
//   out[r]    = scale table[ids[r]]                       (0 for an id outside)
//   dtable[v] (+)= scale sum_{r: ids[r] = v} dout[r]
// Sums in fp32, rounded once; no atomics, so that every result is the same bits
// again.
#include "embed.h"

#include "device_common.h"
#include "sort_rows.h"

namespace moe {

// Eight columns of a row, from c on (those below n), as fp32: 16 bytes a load
// where rows start on 4-byte boundaries (VEC).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int n, float (&f)[8]) {
  if constexpr (VEC && sizeof(T) == 4) {
    float a[4], b[4];
    load_row<T, 4>(row, c, n, a);
    load_row<T, 4>(row, c + 4, n, b);
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = a[i], f[4 + i] = b[i];
  } else if constexpr (VEC) {
    load_row<T, 8>(row, c, n, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = c + i < n ? to_f32(row[c + i]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int c, int n, const float (&f)[8]) {
  if constexpr (VEC && sizeof(T) == 4) {
    const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
    store_row<T, 4>(row, c, n, a);
    store_row<T, 4>(row, c + 4, n, b);
  } else if constexpr (VEC) {
    store_row<T, 8>(row, c, n, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (c + i < n) from_f32(f[i], row[c + i]);
  }
}

// --------------------------------------------------------------------- lookup
// A wave takes 512 columns of a row: 8192 rows of 2560 in bf16 13 us, 4.9 TB/s.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a, const T* __restrict__ table, T* __restrict__ out) {
  const int r = blockIdx.x * 4 + (threadIdx.x >> 6), c = blockIdx.y * 512 + (threadIdx.x & 63) * 8;
  if (r >= a.rows || c >= a.hidden) return;
  const int id = a.ids[r];
  float f[8] = {};
  if ((uint32_t)id < (uint32_t)a.vocab) {
    load8<T, VEC>(table + (int64_t)id * a.hidden, c, a.hidden, f);
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] *= a.scale;
  }
  store8<T, VEC>(out + (int64_t)r * a.hidden, c, a.hidden, f);
}

// ------------------------------------------------------------------- gradient
struct EmbedGrad {
  EmbedGradArgs a;
  // many rows: the rows by id, their number, and the sums of tokens whose rows
  // pass the border of a chunk
  int32_t* order;
  const int32_t* kept;
  float* part;  // [chunks][2][hidden]
  int chunk;    // rows of a chunk
};

template <typename T, bool VEC, bool ADD>
__device__ __forceinline__ void put_sum(const EmbedGrad& g, int v, int c, float (&f)[8]) {
  const int n = g.a.e.hidden;
  T* row = static_cast<T*>(g.a.dtable) + (int64_t)v * n;
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] *= g.a.e.scale;
  if constexpr (ADD) {
    float o[8];
    load8<T, VEC>(row, c, n, o);
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] += o[i];
  }
  store8<T, VEC>(row, c, n, f);
}

// A few rows, whose ids a wave holds in registers, 64 K of them: it goes through
// tokens of the vocabulary (ADD: those of the rows, at the first row of each)
// and sums each one's rows.  61 rows of 257 into 1000 tokens, fp32: 4.8 us, one
// launch's latency.
constexpr int kEmbedFewK = 16;

template <typename T, typename TO, bool VEC, bool ADD>
__global__ __launch_bounds__(256) void embed_grad_few_kernel(EmbedGrad g) {
  const EmbedArgs& e = g.a.e;
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = blockIdx.y * 512 + lane * 8;
  const T* dout = static_cast<const T*>(g.a.dout);
  int id[kEmbedFewK];
#pragma unroll
  for (int k = 0; k < kEmbedFewK; k++) {
    id[k] = -1;
    if (64 * k < e.rows) id[k] = e.ids[64 * k + lane < e.rows ? 64 * k + lane : e.rows - 1];
    if (64 * k + lane >= e.rows) id[k] = -1;
  }
  const int end = ADD ? e.rows : e.vocab;
  for (int i = wave; i < end; i += 4 * gridDim.x) {
    int v = i;
    if constexpr (ADD) {
      v = e.ids[i];
      if ((uint32_t)v >= (uint32_t)e.vocab) continue;
    }
    float sum[8] = {};
    bool first = true;
    bool hit = false;
#pragma unroll
    for (int k = 0; k < kEmbedFewK; k++)
      if (64 * k < e.rows) hit |= id[k] == v;
    const bool any = __ballot(hit) != 0;
    if (any) {
#pragma unroll
      for (int k = 0; k < kEmbedFewK; k++) {
        if (64 * k >= e.rows) continue;
        uint64_t m = __ballot(id[k] == v);
        if (ADD && first && m) {
          first = false;
          if (64 * k + __builtin_ctzll(m) != i) goto next;  // (an earlier row's)
        }
        while (m) {  // four rows under way at once
          int r[4];
          float f[4][8];
          const int n = __popcll(m) < 4 ? __popcll(m) : 4;
#pragma unroll
          for (int q = 0; q < 4; q++) {
            r[q] = m ? 64 * k + __builtin_ctzll(m) : 0;
            m &= m - 1;
          }
#pragma unroll
          for (int q = 0; q < 4; q++)
            if (q < n && c < e.hidden) load8<T, VEC>(dout + (int64_t)r[q] * e.hidden, c, e.hidden, f[q]);
#pragma unroll
          for (int q = 0; q < 4; q++)
            if (q < n && c < e.hidden) {
#pragma unroll
              for (int j = 0; j < 8; j++) sum[j] += f[q][j];
            }
        }
      }
    }
    if (c < e.hidden) {
      if (any)
        put_sum<TO, VEC, ADD>(g, v, c, sum);
      else  // 0, whatever the scale is
        store8<TO, VEC>(static_cast<TO*>(g.a.dtable) + (int64_t)v * e.hidden, c, e.hidden, sum);
    }
  next:;
  }
}

__device__ __forceinline__ void fill_zero(void* p, size_t bytes, size_t block, size_t blocks, int threads) {
  u32x4* q = static_cast<u32x4*>(p);
  const size_t n = bytes / 16;
  for (size_t i = block * threads + threadIdx.x; i < n; i += blocks * threads) q[i] = u32x4{0u, 0u, 0u, 0u};
  if (block == 0 && threadIdx.x < (bytes & 15) / 2)
    reinterpret_cast<uint16_t*>(p)[n * 8 + threadIdx.x] = 0;
}

// The rows sorted by id, digit by digit, in one block, while the others clear
// the table (778 MB 138 us, 5.6 TB/s; the sort of 8192 rows, 20 us, runs beside).
struct EmbedSort {
  SortArgs low, high;  // high.groups 0: one digit
  void* table;         // null: not cleared
  size_t bytes;
};

__global__ __launch_bounds__(kSortThreads) void embed_sort_one_kernel(EmbedSort s) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  if (blockIdx.x > 0) {
    fill_zero(s.table, s.bytes, blockIdx.x - 1, gridDim.x - 1, kSortThreads);
    return;
  }
  const int kept = sort_one<true>(s.low, cnt, sh, base);
  if (s.high.groups == 0) return;
  __threadfence();
  __syncthreads();
  s.high.kept = nullptr;
  s.high.kept_here = kept;
  sort_one<true>(s.high, cnt, sh, base);
}

// The same in several blocks; the others of the first launch clear the table.
__global__ __launch_bounds__(kSortThreads) void embed_sort_count_kernel(SortArgs a, void* table, size_t bytes) {
  extern __shared__ uint16_t cnt[];
  if ((int)blockIdx.x >= a.chunks) {
    fill_zero(table, bytes, blockIdx.x - a.chunks, gridDim.x - a.chunks, kSortThreads);
    return;
  }
  sort_count<true>(a, cnt);
}
__global__ __launch_bounds__(kSortThreads) void embed_sort_place_kernel(SortArgs a) {
  extern __shared__ uint16_t cnt[];
  __shared__ SortShared sh;
  __shared__ int32_t base[kSortMaxGroups];
  sort_place<true>(a, cnt, sh, base);
}

// A wave takes 512 columns of a chunk of sorted rows, eight rows under way at
// once, and sums each token's.  A token whose rows lie in the chunk is done; of
// one that comes from the chunk before, the sum goes to part[chunk][0], of one
// that begins here and goes on, to part[chunk][1].  8192 rows of 2560 in bf16 33
// us behind the clearing, whose writes are still under way (chunks of 8 or 24
// rows, 16 rows under way at once: no less).
template <typename T, typename TO, bool VEC, bool ADD>
__global__ __launch_bounds__(256) void embed_grad_chunk_kernel(EmbedGrad g) {
  const EmbedArgs& e = g.a.e;
  const int chunk = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = blockIdx.y * 512 + (threadIdx.x & 63) * 8;
  const int n = *g.kept, lo = chunk * g.chunk;
  if (lo >= n || c >= e.hidden) return;
  const int hi = lo + g.chunk < n ? lo + g.chunk : n;
  const int before = lo > 0 ? e.ids[g.order[lo - 1]] : -1, after = hi < n ? e.ids[g.order[hi]] : -1;
  const T* dout = static_cast<const T*>(g.a.dout);
  int cur = -1;
  bool begins = true;
  float sum[8] = {};
  auto put = [&](bool ends) {
    if (begins && ends) {
      put_sum<TO, VEC, ADD>(g, cur, c, sum);
    } else {
      float* p = g.part + ((size_t)chunk * 2 + (begins ? 1 : 0)) * e.hidden;
      store8<float, true>(p, c, e.hidden, sum);
    }
  };
  for (int i0 = lo; i0 < hi; i0 += 8) {
    int r[8], id[8];
    float f[8][8];
#pragma unroll
    for (int q = 0; q < 8; q++) r[q] = g.order[i0 + q < hi ? i0 + q : hi - 1];
#pragma unroll
    for (int q = 0; q < 8; q++) {
      id[q] = e.ids[r[q]];
      load8<T, VEC>(dout + (int64_t)r[q] * e.hidden, c, e.hidden, f[q]);
    }
#pragma unroll
    for (int q = 0; q < 8; q++) {
      if (i0 + q >= hi) continue;
      if (id[q] != cur) {
        if (cur >= 0) put(true);
        begins = !(i0 + q == lo && id[q] == before);
        cur = id[q];
#pragma unroll
        for (int j = 0; j < 8; j++) sum[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += f[q][j];
    }
  }
  put(cur != after);
}

// The tokens that begin in a chunk and go on behind it: their parts added in
// order.
template <typename TO, bool VEC, bool ADD>
__global__ __launch_bounds__(256) void embed_grad_join_kernel(EmbedGrad g) {
  const EmbedArgs& e = g.a.e;
  const int lane = threadIdx.x & 63;
  const int chunk = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = blockIdx.y * 512 + lane * 8;
  const int n = *g.kept, lo = chunk * g.chunk, hi = lo + g.chunk;
  if (hi >= n) return;
  const int v = e.ids[g.order[hi - 1]];
  if (e.ids[g.order[hi]] != v) return;
  if (lo > 0 && e.ids[g.order[lo]] == v && e.ids[g.order[lo - 1]] == v) return;  // it began before
  int more = 0;  // chunks that it goes on through
  for (;;) {
    const int next = chunk + 1 + more + lane;  // (a chunk that starts with a row of v)
    const bool in = (int64_t)next * g.chunk < n && e.ids[g.order[next * g.chunk]] == v;
    const uint64_t m = ~__ballot(in);
    const int run = m ? __builtin_ctzll(m) : 64;
    more += run;
    if (run < 64) break;
  }
  if (c >= e.hidden) return;
  const float* p = g.part + (size_t)chunk * 2 * e.hidden;
  float sum[8];
  load8<float, true>(p + e.hidden, c, e.hidden, sum);
  for (int i0 = 1; i0 <= more; i0 += 8) {
    float f[8][8];
#pragma unroll
    for (int q = 0; q < 8; q++)
      load8<float, true>(p + (size_t)(i0 + q <= more ? i0 + q : more) * 2 * e.hidden, c, e.hidden, f[q]);
#pragma unroll
    for (int q = 0; q < 8; q++) {
      if (i0 + q > more) continue;
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += f[q][j];
    }
  }
  put_sum<TO, VEC, ADD>(g, v, c, sum);
}

struct IdSortPlan {
  int low_bits, low, high;  // digits: values of the low one, of the high one (0: none)
  size_t order_a, order_b, offsets, counts, total;
};

static IdSortPlan id_sort_plan(int rows, int vocab) {
  IdSortPlan p = {};
  int bits = 0;
  while ((1 << bits) < vocab) bits++;
  if (vocab <= kSortMaxGroups) {
    p.low_bits = bits;
    p.low = vocab;
  } else {
    p.low_bits = bits / 2;
    p.low = 1 << p.low_bits;
    p.high = (vocab + p.low - 1) >> p.low_bits;
  }
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  p.order_a = take((size_t)rows * 4);
  p.order_b = take((size_t)rows * 4);
  p.offsets = take((size_t)(kSortMaxGroups + 1) * 4 * 2);
  const size_t ca = sort_workspace(rows, p.low), cb = p.high ? sort_workspace(rows, p.high) : 0;
  p.counts = take(ca > cb ? ca : cb);
  p.total = o;
  return p;
}

size_t id_sort_workspace(int rows, int vocab) { return id_sort_plan(rows, vocab).total; }

hipError_t launch_id_sort(const int32_t* ids, int rows, int vocab, void* workspace, void* clear, size_t clear_bytes,
                          int32_t** order, const int32_t** kept, hipStream_t stream) {
  const IdSortPlan p = id_sort_plan(rows, vocab);
  char* b = static_cast<char*>(workspace);
  EmbedSort s = {};
  s.low.ids = ids;
  s.low.picks = rows;
  s.low.ids_below = vocab;
  s.low.counts = reinterpret_cast<int32_t*>(b + p.counts);
  s.high = s.low;
  s.low.groups = p.low;
  s.low.order = reinterpret_cast<int32_t*>(b + p.order_a);
  s.low.offsets = reinterpret_cast<int32_t*>(b + p.offsets);
  s.high.groups = p.high;
  s.high.shift = p.low_bits;
  s.high.by = s.low.order;
  s.high.kept = s.low.offsets + p.low;
  s.high.order = reinterpret_cast<int32_t*>(b + p.order_b);
  s.high.offsets = s.low.offsets + kSortMaxGroups + 1;
  *order = p.high ? s.high.order : s.low.order;
  *kept = s.high.kept;
  plan_sort(&s.low);
  if (p.high) plan_sort(&s.high);
  s.table = clear;
  s.bytes = clear_bytes;
  const size_t per = (size_t)kSortThreads * 16 * 4;  // bytes of a clearing block, at least
  const size_t most = (s.bytes + per - 1) / per;
  const int fill = clear ? (int)(most < 512 ? most : 512) : 0;
  const size_t lds_low = (size_t)kSortWaves * p.low * 2, lds_high = (size_t)kSortWaves * p.high * 2;
  if (s.low.chunks <= 1) {
    hipLaunchKernelGGL(embed_sort_one_kernel, dim3(1 + fill), dim3(kSortThreads), lds_low > lds_high ? lds_low : lds_high,
                       stream, s);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(embed_sort_count_kernel, dim3(s.low.chunks + fill), dim3(kSortThreads), lds_low, stream, s.low,
                     s.table, s.bytes);
  hipLaunchKernelGGL(embed_sort_place_kernel, dim3(s.low.chunks), dim3(kSortThreads), lds_low, stream, s.low);
  if (p.high) {
    hipLaunchKernelGGL(embed_sort_count_kernel, dim3(s.high.chunks), dim3(kSortThreads), lds_high, stream, s.high,
                       nullptr, (size_t)0);
    hipLaunchKernelGGL(embed_sort_place_kernel, dim3(s.high.chunks), dim3(kSortThreads), lds_high, stream, s.high);
  }
  return hipGetLastError();
}

// --------------------------------------------------------------------- launches
// Rows up to which every wave holds all ids, and one of them sums a token's in 512
// columns.  bf16 into 1000 x 2560: 1024 rows of different tokens 8.0 us, 1025, by the
// sort, 18.7; but all of one token 212 (with add 368) and 40.
constexpr int kEmbedFew = 64 * kEmbedFewK;

struct EmbedPlan {
  int chunk, chunks;
  size_t part, total;
};

static EmbedPlan embed_plan(int rows, int vocab, int hidden) {
  EmbedPlan p = {};
  if (rows <= kEmbedFew) return p;
  // chunks of 16 rows, longer ones above 32768 rows, so that a token of most rows
  // goes through few of them
  const int want = rows / 2048 / 8 * 8;
  p.chunk = want < 16 ? 16 : (want > 128 ? 128 : want);
  p.chunks = (rows + p.chunk - 1) / p.chunk;
  p.part = id_sort_workspace(rows, vocab);
  p.total = p.part + (size_t)p.chunks * 2 * hidden * 4;
  return p;
}

size_t embed_backward_workspace(int rows, int vocab, int hidden) { return embed_plan(rows, vocab, hidden).total; }

template <typename T, bool VEC>
static hipError_t embed_v(const EmbedArgs& a, const void* table, void* out, hipStream_t stream) {
  hipLaunchKernelGGL((embed_kernel<T, VEC>), dim3((a.rows + 3) / 4, (a.hidden + 511) / 512), dim3(256), 0, stream, a,
                     static_cast<const T*>(table), static_cast<T*>(out));
  return hipGetLastError();
}

hipError_t launch_embed(const EmbedArgs& a, const void* table, void* out, hipStream_t stream) {
  if (a.f32) return embed_v<float, true>(a, table, out, stream);
  return a.hidden % 2 ? embed_v<uint16_t, false>(a, table, out, stream)
                      : embed_v<uint16_t, true>(a, table, out, stream);
}

template <typename T, typename TO, bool VEC, bool ADD>
static hipError_t embed_backward_v(const EmbedGradArgs& a, char* b, hipStream_t stream) {
  const EmbedArgs& e = a.e;
  EmbedGrad g = {};
  g.a = a;
  const int parts = (e.hidden + 511) / 512;
  if (e.rows <= kEmbedFew) {
    const int64_t items = ADD ? e.rows : e.vocab;
    const int64_t most = 8192 / parts > 64 ? 8192 / parts : 64, want = (items + 3) / 4;
    hipLaunchKernelGGL((embed_grad_few_kernel<T, TO, VEC, ADD>), dim3((uint32_t)(want < most ? want : most), parts),
                       dim3(256), 0, stream, g);
    return hipGetLastError();
  }
  const EmbedPlan p = embed_plan(e.rows, e.vocab, e.hidden);
  const hipError_t st = launch_id_sort(e.ids, e.rows, e.vocab, b, ADD ? nullptr : a.dtable,
                                       (size_t)e.vocab * e.hidden * sizeof(TO), &g.order, &g.kept, stream);
  if (st != hipSuccess) return st;
  g.part = reinterpret_cast<float*>(b + p.part);
  g.chunk = p.chunk;
  const dim3 grid((p.chunks + 3) / 4, parts);
  hipLaunchKernelGGL((embed_grad_chunk_kernel<T, TO, VEC, ADD>), grid, dim3(256), 0, stream, g);
  hipLaunchKernelGGL((embed_grad_join_kernel<TO, VEC, ADD>), grid, dim3(256), 0, stream, g);
  return hipGetLastError();
}

template <typename T, typename TO>
static hipError_t embed_backward_t(const EmbedGradArgs& a, char* b, hipStream_t stream) {
  const bool vec = a.e.hidden % 2 == 0 || (sizeof(T) == 4 && sizeof(TO) == 4);
  if (a.add) return vec ? embed_backward_v<T, TO, true, true>(a, b, stream) : embed_backward_v<T, TO, false, true>(a, b, stream);
  return vec ? embed_backward_v<T, TO, true, false>(a, b, stream) : embed_backward_v<T, TO, false, false>(a, b, stream);
}

hipError_t launch_embed_backward(const EmbedGradArgs& a, void* workspace, hipStream_t stream) {
  char* b = static_cast<char*>(workspace);
  if (a.e.f32) return a.f32 ? embed_backward_t<float, float>(a, b, stream) : embed_backward_t<float, uint16_t>(a, b, stream);
  return a.f32 ? embed_backward_t<uint16_t, float>(a, b, stream) : embed_backward_t<uint16_t, uint16_t>(a, b, stream);
}

}  // namespace moe
