// products.hip -- matrix products of rows grouped by expert, for batches whose
// rows token_rows.hip has sorted: with rows offsets[e] .. offsets[e+1] of the
// buffers expert e's,
//   y[r]  = W_e x[r]                      (W_e [n, k])
//   dx[r] = W_e^T dy[r]
//   dW_e  = sum_r dy[r] x[r]^T            (0 for an expert without rows)
// bf16 operands, sums in fp32, rounded once.
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
  bool stored = false;
  for (;;) {
    t += gridDim.x;
    const bool more = t < total;
    ProductTile next = p;
    if (more) next = tile_at(t);
    auto finish = [&](auto u) TILE_INLINE {
      TileSums<decltype(u)::value, V> sums;
      pipe.template run<kTileStores<UMAX, V, T>>(s0, s1, s2, sums, stored);
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
    stored = p.m.own > 16 * UMAX;  // (fewer stores of a tile of fewer rows)
    p = next;
  }
}

// y of tiles of few rows: 64 rows and 64 columns.
template <typename T>
__global__ __launch_bounds__(256, 2) void moe_product_few_kernel(ProductArgs a) {
  __shared__ __align__(16) uint8_t lds[StreamPipe<kStreamU>::kLds];
  __shared__ ProductPlaces places;
  count_tiles<kStreamM>(a, places);
  const int j_tiles = (a.n + kStreamJ - 1) / kStreamJ;
  const int64_t total = (int64_t)places.first[a.experts] * j_tiles;
  T* out = reinterpret_cast<T*>(a.y);
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int rt = (int)(t / j_tiles), e = expert_of_tile(a, places, rt);
    int64_t lo, hi;
    rows_of_expert(a, e, &lo, &hi);
    lo += (int64_t)(rt - __builtin_amdgcn_readfirstlane(places.first[e])) * kStreamM;
    const int j0 = (int)(t - (int64_t)rt * j_tiles) * kStreamJ;
    const int rows = __builtin_amdgcn_readfirstlane((int)(hi - lo < kStreamM ? hi - lo : kStreamM));
    const TileOperand om = {a.x + lo * a.k, (uint32_t)a.k * 2u, rows, a.k};
    const TileOperand oj = {a.w + ((int64_t)e * a.n + j0) * a.k, (uint32_t)a.k * 2u,
                            a.n - j0 < kStreamJ ? a.n - j0 : kStreamJ, a.k};
    auto done = [&](int u, int v, const v4f& s) TILE_INLINE {
      const int m = 16 * u + col, j = j0 + 16 * v + 4 * g;
      if (m >= rows || j >= a.n) return;
      T* to = out + (lo + m) * a.n + j;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<v4f*>(to) = s;
      else
        *reinterpret_cast<uint2*>(to) = uint2{(uint32_t)f32_to_bf16(s[0]) | ((uint32_t)f32_to_bf16(s[1]) << 16),
                                              (uint32_t)f32_to_bf16(s[2]) | ((uint32_t)f32_to_bf16(s[3]) << 16)};
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

// dW of tiles of 32 U rows (of n) and 32 V columns (of k).
template <int U, int V, typename T, bool ADD>
__global__ __launch_bounds__(256) void moe_product_dw_kernel(ProductArgs a) {
  using Pipe = TilePipe<U, V, true, true>;
  constexpr int TM = 32 * U, TJ = 32 * V;
  __shared__ typename Pipe::Stage s0, s1;
  __shared__ typename Pipe::Last s2;
  const int m_tiles = (a.n + TM - 1) / TM, j_tiles = (a.k + TJ - 1) / TJ;
  const int per = m_tiles * j_tiles;
  const int64_t total = (int64_t)a.experts * per;
  struct Tile {
    TileOperand m, j;
    int e, m0, j0;
  };
  auto tile_at = [&](int64_t t) TILE_INLINE {
    Tile p;
    p.e = (int)(t / per);
    int mt, jt;
    place_of((int)(t - (int64_t)p.e * per), m_tiles, j_tiles, &mt, &jt);
    int64_t lo, hi;
    rows_of_expert(a, p.e, &lo, &hi);
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
  bool stored = false;
  for (;;) {
    t += gridDim.x;
    const bool more = t < total;
    Tile next = p;
    if (more) next = tile_at(t);
    TileSums<U, V> sums;
    pipe.template run<ADD ? 0 : kTileStores<U, V, T>>(s0, s1, s2, sums, stored);
    if (more) pipe.start(next.m, next.j, s0, s1, s2);
    T* out = reinterpret_cast<T*>(a.dw) + (int64_t)p.e * a.n * a.k;
    if (!ADD || p.m.c > 0) store_tile<U, V, T, ADD>(sums, out, p.m0, a.n, p.j0, a.k);
    if (!more) return;
    p = next;
    stored = true;
  }
}

// Upper bound of the tiles of `tm` rows by `tj` columns.
static int64_t most_tiles(const ProductArgs& a, int cols, int tm, int tj) {
  const int64_t m = a.rows / tm + (a.rows < a.experts ? a.rows : a.experts);
  return m * ((cols + tj - 1) / tj);
}

template <bool DX, typename T>
static hipError_t launch_rows(const ProductArgs& a, hipStream_t stream) {
  const int cols = DX ? a.k : a.n;
  int blocks;
  const bool large = a.rows > (int64_t)48 * a.experts && most_tiles(a, cols, 256, 256) >= 256;
  if (large) {
    const hipError_t e = tile_blocks(most_tiles(a, cols, 256, 256), 1, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_product_kernel<8, 8, DX, T>), dim3(blocks), dim3(256), 0, stream, a);
  } else if constexpr (!DX) {
    const hipError_t e = tile_blocks(most_tiles(a, cols, kStreamM, kStreamJ), 2, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_product_few_kernel<T>, dim3(blocks), dim3(256), 0, stream, a);
  } else {
    const hipError_t e = tile_blocks(most_tiles(a, cols, 64, 128), 2, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_product_kernel<2, 4, DX, T>), dim3(blocks), dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

size_t product_workspace(const ProductArgs&) { return 0; }
size_t product_backward_workspace(const ProductArgs&) { return 0; }

hipError_t launch_product(const ProductArgs& a, hipStream_t stream) {
  return a.f32 ? launch_rows<false, float>(a, stream) : launch_rows<false, uint16_t>(a, stream);
}
hipError_t launch_product_dx(const ProductArgs& a, hipStream_t stream) {
  return launch_rows<true, uint16_t>(a, stream);
}

template <typename T, bool ADD>
static hipError_t launch_dw(const ProductArgs& a, hipStream_t stream) {
  const int64_t large = (int64_t)a.experts * ((a.n + 255) / 256) * ((a.k + 255) / 256);
  int blocks;
  if (large >= 256) {
    const hipError_t e = tile_blocks(large, 1, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_product_dw_kernel<8, 8, T, ADD>), dim3(blocks), dim3(256), 0, stream, a);
  } else {
    const hipError_t e = tile_blocks((int64_t)a.experts * ((a.n + 127) / 128) * ((a.k + 127) / 128), 2, &blocks);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_product_dw_kernel<4, 4, T, ADD>), dim3(blocks), dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_product_dw(const ProductArgs& a, hipStream_t stream) {
  if (a.f32) return a.add ? launch_dw<float, true>(a, stream) : launch_dw<float, false>(a, stream);
  return a.add ? launch_dw<uint16_t, true>(a, stream) : launch_dw<uint16_t, false>(a, stream);
}

}  // namespace moe
