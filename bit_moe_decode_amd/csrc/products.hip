// products.hip -- matrix products of rows grouped by expert, for batches whose
// rows token_rows.hip has sorted: with rows offsets[e] .. offsets[e+1] of the
// buffers expert e's,
//   y[r]  = W_e x[r]                      (W_e [n, k])
//   dx[r] = W_e^T dy[r]
//   dW_e  = sum_r dy[r] x[r]^T            (0 for an expert without rows)
// bf16 operands, sums in fp32, rounded once.
//
// More than 48 rows of the buffers an expert, and tiles of 256 x 256 enough for the
// CUs: such tiles (tile_product.h), of fewer row tiles where an expert's rows end.
// Else y takes tiles of 64 x 64 that stream the weights (stream_product.h),
// dx of 64 x 128 and dW of 128 x 128.  Measured, of 256 experts [4096, 6144]: 16
// tokens x 8 picks 630 .. 720 us, the bytes of the 72 .. 84 experts in use at 5.4 ..
// 6.2 TB/s.  Of 64 experts [4096, 6144]: y of 65536 rows 2850 .. 3000 us (1.1
// PFLOP/s; 19 rounds of tiles where even experts would take 16), dx of 32768 1530 ..
// 1600 us (1.05), dW of 32768 2010 .. 2140 us (0.8 PFLOP/s: of it 600 us are the 3.2
// GB of its store, which 8 steps a tile do not hide; without the store 1410; added to
// an old dW, which is read behind the sums, 3650 .. 3710).
#include "products.h"

#include "device_common.h"
#include "stream_product.h"
#include "tile_product.h"

namespace moe {

// Expert e's rows, from offsets that may be anything: none reach out of the
// buffers.
__device__ __forceinline__ void rows_of_expert(const ProductArgs& a, int e, int64_t* lo, int64_t* hi) {
  const int64_t i = a.offsets[e], j = a.offsets[e + 1];
  *lo = i < 0 ? 0 : (i < a.rows ? i : a.rows);
  *hi = j < *lo ? *lo : (j < a.rows ? j : a.rows);
}

// first[e]: row tiles of the experts before e, and of all in first[experts].
// (A group of 4 experts a thread.)
struct ProductPlaces {
  int first[kProductMaxExperts + 1];
  int wave[4];
};
template <int TILE>
__device__ __forceinline__ void count_tiles(const ProductArgs& a, ProductPlaces& p) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int e = 4 * tid + i;
    n[i] = 0;
    if (e < a.experts) {
      int64_t lo, hi;
      rows_of_expert(a, e, &lo, &hi);
      n[i] = (int)((hi - lo + TILE - 1) / TILE);
    }
    sum += n[i];
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int t = __shfl_up(upto, o, kWave);
    if (lane >= o) upto += t;
  }
  if (lane == 63) p.wave[wv] = upto;
  __syncthreads();
  int at = upto - sum;
  for (int w = 0; w < wv; w++) at += p.wave[w];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (4 * tid + i <= a.experts) p.first[4 * tid + i] = at;
    at += n[i];
  }
  if (tid == 255 && a.experts == kProductMaxExperts) p.first[kProductMaxExperts] = at;
  __syncthreads();
}
// The expert whose row tile i is: the last e with first[e] <= i (16 experts a
// lane, then one of 16 a lane).
__device__ __forceinline__ int expert_of_tile(const ProductArgs& a, const ProductPlaces& p, int i) {
  const int lane = threadIdx.x & 63;
  const bool big = 16 * lane < a.experts && p.first[16 * lane] <= i;
  const int e0 = 16 * (__popcll(__ballot(big)) - 1);
  const int e = e0 + (lane & 15);
  const bool below = e < a.experts && p.first[e] <= i;
  return __builtin_amdgcn_readfirstlane(e0 + __popcll(__ballot(below) & 0xFFFFu) - 1);
}

// A tile: rows lo + .. to hi, columns j0 + .. of the output.
struct ProductTile {
  TileOperand m, j;
  int64_t lo, hi;
  int j0;
};

// y, or with DX dx, of tiles of 32 UMAX rows at most (fewer where a group's last
// tile holds fewer) and 32 V columns.
template <int UMAX, int V, bool DX, typename T>
__global__ __launch_bounds__(256) void moe_product_kernel(ProductArgs a) {
  using Pipe = TilePipe<UMAX, V, false, DX>;
  constexpr int TM = 32 * UMAX, TJ = 32 * V;
  __shared__ typename Pipe::Stage s0, s1;
  __shared__ typename Pipe::Last s2;
  __shared__ ProductPlaces places;
  count_tiles<TM>(a, places);
  const int cols = DX ? a.k : a.n, len = DX ? a.n : a.k;
  const int j_tiles = (cols + TJ - 1) / TJ;
  const int64_t total = (int64_t)places.first[a.experts] * j_tiles;
  T* out = reinterpret_cast<T*>(DX ? (void*)a.dx : a.y);
  auto tile_at = [&](int64_t t) TILE_INLINE {
    const int e = expert_of_tile(a, places, (int)(t / j_tiles));
    const int before = __builtin_amdgcn_readfirstlane(places.first[e]);
    const int mine = __builtin_amdgcn_readfirstlane(places.first[e + 1]) - before;
    int mt, jt;
    place_of((int)(t - (int64_t)before * j_tiles), mine, j_tiles, &mt, &jt);
    ProductTile p;
    rows_of_expert(a, e, &p.lo, &p.hi);
    p.lo += (int64_t)mt * TM;
    p.j0 = jt * TJ;
    const int rows = __builtin_amdgcn_readfirstlane((int)(p.hi - p.lo < TM ? p.hi - p.lo : TM));
    p.m = {(DX ? a.dy : a.x) + p.lo * len, (uint32_t)len * 2u, rows, len};
    p.j = {a.w + (int64_t)e * a.n * a.k + (DX ? (int64_t)p.j0 : (int64_t)p.j0 * a.k), (uint32_t)a.k * 2u,
           cols - p.j0 < TJ ? cols - p.j0 : TJ, len};
    return p;
  };
  int64_t t = first_tile();
  if (t >= total) return;
  Pipe pipe;
  ProductTile p = tile_at(t);
  pipe.start(p.m, p.j, s0, s1, s2);
  for (;;) {
    t += gridDim.x;
    const bool more = t < total;
    ProductTile next = p;
    if (more) next = tile_at(t);
    auto finish = [&](auto u) TILE_INLINE {
      TileSums<decltype(u)::value, V> sums;
      pipe.run(s0, s1, s2, sums);
      if (more) pipe.start(next.m, next.j, s0, s1, s2);
      store_tile<decltype(u)::value, V, T, false>(sums, out, p.lo, p.hi, p.j0, cols);
    };
    if (UMAX == 8 && p.m.own > 128)
      finish(std::integral_constant<int, UMAX>{});
    else if (UMAX >= 4 && p.m.own > 64)
      finish(std::integral_constant<int, UMAX < 4 ? UMAX : 4>{});
    else if (p.m.own > 32)
      finish(std::integral_constant<int, 2>{});
    else
      finish(std::integral_constant<int, 1>{});
    if (!more) return;
    p = next;
  }
}

__device__ __forceinline__ void put4(float* to, const v4f& s) { *reinterpret_cast<v4f*>(to) = s; }
__device__ __forceinline__ void put4(uint16_t* to, const v4f& s) {
  *reinterpret_cast<uint2*>(to) = uint2{(uint32_t)f32_to_bf16(s[0]) | ((uint32_t)f32_to_bf16(s[1]) << 16),
                                        (uint32_t)f32_to_bf16(s[2]) | ((uint32_t)f32_to_bf16(s[3]) << 16)};
}

// y of tiles of few rows: 64 rows and 64 columns.  Where these are fewer than the
// CUs, of parts of k, whose sums [parts][rows][n] of float are T's; they are then
// added in order.
template <typename T>
__global__ __launch_bounds__(256, 2) void moe_product_few_kernel(ProductArgs a) {
  __shared__ __align__(16) uint8_t lds[StreamPipe<kStreamU>::kLds];
  __shared__ ProductPlaces places;
  count_tiles<kStreamM>(a, places);
  const int j_tiles = (a.n + kStreamJ - 1) / kStreamJ;
  const int64_t total = (int64_t)places.first[a.experts] * j_tiles;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  for (int64_t i = blockIdx.x; i < total * a.parts; i += gridDim.x) {
    const int part = (int)(i / total), k0 = part * a.part, c = a.k - k0 < a.part ? a.k - k0 : a.part;
    const int64_t t = i - part * total;
    T* out = a.parts > 1 ? reinterpret_cast<T*>(a.space) + (int64_t)part * a.rows * a.n : reinterpret_cast<T*>(a.y);
    const int rt = (int)(t / j_tiles), e = expert_of_tile(a, places, rt);
    int64_t lo, hi;
    rows_of_expert(a, e, &lo, &hi);
    lo += (int64_t)(rt - __builtin_amdgcn_readfirstlane(places.first[e])) * kStreamM;
    const int j0 = (int)(t - (int64_t)rt * j_tiles) * kStreamJ;
    const int rows = __builtin_amdgcn_readfirstlane((int)(hi - lo < kStreamM ? hi - lo : kStreamM));
    const TileOperand om = {a.x + lo * a.k + k0, (uint32_t)a.k * 2u, rows, c};
    const TileOperand oj = {a.w + ((int64_t)e * a.n + j0) * a.k + k0, (uint32_t)a.k * 2u,
                            a.n - j0 < kStreamJ ? a.n - j0 : kStreamJ, c};
    auto done = [&](int u, int v, const v4f& s) TILE_INLINE {
      const int m = 16 * u + col, j = j0 + 16 * v + 4 * g;
      if (m >= rows || j >= a.n) return;
      put4(out + (lo + m) * a.n + j, s);
    };
    if (rows > 32) {
      StreamPipe<4> pipe;
      pipe.start(om, oj);
      pipe.run(lds);
      pipe.add(lds, done);
    } else if (rows > 16) {
      StreamPipe<2> pipe;
      pipe.start(om, oj);
      pipe.run(lds);
      pipe.add(lds, done);
    } else {
      StreamPipe<1> pipe;
      pipe.start(om, oj);
      pipe.run(lds);
      pipe.add(lds, done);
    }
  }
}

// y from the sums of k's parts.
template <typename T>
__global__ __launch_bounds__(256) void moe_product_add_kernel(ProductArgs a) {
  int64_t first, last, unused;
  rows_of_expert(a, 0, &first, &unused);
  rows_of_expert(a, a.experts - 1, &unused, &last);
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, r = i / a.n;
  if (r < first || r >= last) return;
  v4f s = *reinterpret_cast<const v4f*>(a.space + i);
  for (int p = 1; p < a.parts; p++) s += *reinterpret_cast<const v4f*>(a.space + p * a.rows * a.n + i);
  put4(reinterpret_cast<T*>(a.y) + i, s);
}

// dW of tiles of 32 U rows (of n) and 32 V columns (of k); where these are fewer
// than the CUs, of parts of the expert's rows, as above.
template <int U, int V, typename T, bool ADD>
__global__ __launch_bounds__(256) void moe_product_dw_kernel(ProductArgs a) {
  using Pipe = TilePipe<U, V, true, true>;
  constexpr int TM = 32 * U, TJ = 32 * V;
  __shared__ typename Pipe::Stage s0, s1;
  __shared__ typename Pipe::Last s2;
  const int m_tiles = (a.n + TM - 1) / TM, j_tiles = (a.k + TJ - 1) / TJ;
  const int per = m_tiles * j_tiles;
  const int64_t total = (int64_t)a.experts * per * a.parts;
  struct Tile {
    TileOperand m, j;
    int e, m0, j0;  // e: behind the experts, part by part, where there are several
  };
  auto tile_at = [&](int64_t t) TILE_INLINE {
    Tile p;
    p.e = (int)(t / per);
    int mt, jt;
    place_of((int)(t - (int64_t)p.e * per), m_tiles, j_tiles, &mt, &jt);
    int64_t lo, hi;
    const int part = p.e / a.experts;
    rows_of_expert(a, p.e - part * a.experts, &lo, &hi);
    if (a.parts > 1) {  // an expert's rows, in equal parts
      const int64_t one = ((hi - lo + a.parts - 1) / a.parts + kStepC - 1) / kStepC * kStepC;
      lo = lo + part * one < hi ? lo + part * one : hi;
      hi = hi - lo < one ? hi : lo + one;
    }
    const int c = __builtin_amdgcn_readfirstlane((int)(hi - lo));
    p.m0 = mt * TM;
    p.j0 = jt * TJ;
    p.m = {a.dy + lo * a.n + p.m0, (uint32_t)a.n * 2u, a.n - p.m0 < TM ? a.n - p.m0 : TM, c};
    p.j = {a.x + lo * a.k + p.j0, (uint32_t)a.k * 2u, a.k - p.j0 < TJ ? a.k - p.j0 : TJ, c};
    return p;
  };
  int64_t t = first_tile();
  if (t >= total) return;
  Pipe pipe;
  Tile p = tile_at(t);
  pipe.start(p.m, p.j, s0, s1, s2);
  for (;;) {
    t += gridDim.x;
    const bool more = t < total;
    Tile next = p;
    if (more) next = tile_at(t);
    TileSums<U, V> sums;
    pipe.run(s0, s1, s2, sums);
    if (more) pipe.start(next.m, next.j, s0, s1, s2);
    T* out = reinterpret_cast<T*>(a.parts > 1 ? (void*)a.space : a.dw) + (int64_t)p.e * a.n * a.k;
    if (!ADD || p.m.c > 0) store_tile<U, V, T, ADD>(sums, out, p.m0, a.n, p.j0, a.k);
    if (!more) return;
    p = next;
  }
}

// dW from the sums of the rows' parts.
template <typename T, bool ADD>
__global__ __launch_bounds__(256) void moe_product_dw_add_kernel(ProductArgs a) {
  const int64_t one = (int64_t)a.n * a.k, all = one * a.experts, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= all) return;
  T* to = reinterpret_cast<T*>(a.dw) + i;
  v4f s = *reinterpret_cast<const v4f*>(a.space + i);
  for (int p = 1; p < a.parts; p++) s += *reinterpret_cast<const v4f*>(a.space + p * all + i);
  if constexpr (ADD) {
    int64_t lo, hi;
    rows_of_expert(a, (int)(i / one), &lo, &hi);
    if (lo == hi) return;  // (no rows: left as it was)
    if constexpr (sizeof(T) == 4) {
      s += *reinterpret_cast<const v4f*>(to);
    } else {
      const uint2 o = *reinterpret_cast<const uint2*>(to);
      s += v4f{__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u), __uint_as_float(o.y << 16),
               __uint_as_float(o.y & 0xFFFF0000u)};
    }
  }
  put4(to, s);
}

// Upper bound of the tiles of `tm` rows by `tj` columns.
static int64_t most_tiles(const ProductArgs& a, int cols, int tm, int tj) {
  const int64_t m = a.rows / tm + (a.rows < a.experts ? a.rows : a.experts);
  return m * ((cols + tj - 1) / tj);
}

// Large tiles where there are enough of them and more than 48 rows an expert.  The
// offsets are the device's, so these are the buffers' rows, those of no expert here
// (another rank's) among them.  y and dx of 64 experts [4096, 6144], us, in large
// tiles and in small ones: 32 rows an expert 668, 635 and 589, 601; 48: 679, 644 and
// 645, 618; 64: 691, 647 and 681, 634; 96: 718 .. 752, 660 and 1245, 866; 128: 748,
// 677 and 1014, 923.  A quarter of the rows here, 16 of 64 an expert: 656, 630, where
// small tiles would take 555, 581.
static bool rows_large(const ProductArgs& a, int cols) {
  return a.rows > (int64_t)48 * a.experts && most_tiles(a, cols, 256, 256) >= 256;
}
// Parts of k of the small tiles, up to a block a CU, of 16 steps of 64 at least (8
// rows of 4 experts [512, 6144] 15.8 -> 10.2 us; two blocks a CU: 64 rows of 8
// experts [1024, 4096] 17.7 us, not split 14.5).
static void split_rows(ProductArgs* a) {
  const int64_t tiles = most_tiles(*a, a->n, kStreamM, kStreamJ), steps = (a->k + 63) / 64;
  int64_t parts = rows_large(*a, a->n) || tiles < 1 ? 1 : 256 / tiles;
  if (parts > steps / 16) parts = steps / 16;
  if (parts > 16) parts = 16;
  a->parts = parts < 2 ? 1 : (int)parts;
  a->part = (int)((steps + a->parts - 1) / a->parts) * 64;
}
// Tiles of dW, and parts of the rows up to two blocks a CU, of 512 rows at least
// if they are spread evenly (60000 rows of 8 experts, dW [128, 128] 51.7 -> 16.6
// us; 16384 of 4 experts [512, 512] 32.8 -> 29.7).
static int64_t dw_tiles(const ProductArgs& a, int side) {
  return (int64_t)a.experts * ((a.n + side - 1) / side) * ((a.k + side - 1) / side);
}
static void split_dw(ProductArgs* a) {
  int64_t parts = dw_tiles(*a, 256) >= 256 ? 1 : 512 / dw_tiles(*a, 128);
  const int64_t by_rows = a->rows / ((int64_t)a->experts * 512);
  if (parts > by_rows) parts = by_rows;
  if (parts > 32) parts = 32;
  a->parts = parts < 2 ? 1 : (int)parts;
}

size_t product_workspace(const ProductArgs& args) {
  ProductArgs a = args;
  split_rows(&a);
  return a.parts > 1 ? (size_t)a.parts * a.rows * a.n * 4 : 0;
}
size_t product_backward_workspace(const ProductArgs& args) {
  ProductArgs a = args;
  split_dw(&a);
  return a.parts > 1 ? (size_t)a.parts * a.experts * a.n * a.k * 4 : 0;
}

template <bool DX, typename T>
static hipError_t launch_large(const ProductArgs& a, hipStream_t stream) {
  int blocks;
  const hipError_t e = tile_blocks(most_tiles(a, DX ? a.k : a.n, 256, 256), 1, &blocks);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_product_kernel<8, 8, DX, T>), dim3(blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_few(const ProductArgs& a, hipStream_t stream) {
  int blocks;
  const hipError_t e = tile_blocks(most_tiles(a, a.n, kStreamM, kStreamJ) * a.parts, 2, &blocks);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_product_few_kernel<T>, dim3(blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_product(const ProductArgs& args, hipStream_t stream) {
  ProductArgs a = args;
  if (rows_large(a, a.n)) return a.f32 ? launch_large<false, float>(a, stream) : launch_large<false, uint16_t>(a, stream);
  split_rows(&a);
  if (a.parts == 1) return a.f32 ? launch_few<float>(a, stream) : launch_few<uint16_t>(a, stream);
  const hipError_t e = launch_few<float>(a, stream);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)((a.rows * a.n / 4 + 255) / 256));
  if (a.f32)
    hipLaunchKernelGGL(moe_product_add_kernel<float>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(moe_product_add_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_product_dx(const ProductArgs& a, hipStream_t stream) {
  if (rows_large(a, a.k)) return launch_large<true, uint16_t>(a, stream);
  int blocks;
  const hipError_t e = tile_blocks(most_tiles(a, a.k, 64, 128), 2, &blocks);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_product_kernel<2, 4, true, uint16_t>), dim3(blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T, bool ADD>
static hipError_t launch_dw(const ProductArgs& args, hipStream_t stream) {
  ProductArgs a = args;
  a.parts = 1;
  const int64_t large = dw_tiles(a, 256), small = dw_tiles(a, 128);
  int blocks;
  if (large >= 256) {
    const hipError_t e = tile_blocks(large, 1, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_product_dw_kernel<8, 8, T, ADD>), dim3(blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  split_dw(&a);
  const hipError_t e = tile_blocks(small * a.parts, 1, &blocks);
  if (e != hipSuccess) return e;
  if (a.parts == 1) {
    hipLaunchKernelGGL((moe_product_dw_kernel<4, 4, T, ADD>), dim3(blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((moe_product_dw_kernel<4, 4, float, false>), dim3(blocks), dim3(256), 0, stream, a);
  const int64_t n = (int64_t)a.experts * a.n * a.k / 4;
  hipLaunchKernelGGL((moe_product_dw_add_kernel<T, ADD>), dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_product_dw(const ProductArgs& a, hipStream_t stream) {
  if (a.f32) return a.add ? launch_dw<float, true>(a, stream) : launch_dw<float, false>(a, stream);
  return a.add ? launch_dw<uint16_t, true>(a, stream) : launch_dw<uint16_t, false>(a, stream);
}

}  // namespace moe
