// lora.hip -- low-rank adapters of many requests at once, beside a projection
// they share: row r with adapter i = ids[r] gets
//   y[r] = bf16( base[r] + scale_i * B_i (A_i x[r]) )
// with A_i [rank, K], B_i [N, rank].  Rows without an adapter keep base.  The
// inner product A x is summed and kept in fp32.
#include "lora.h"

namespace moe {

// ------------------------------------------------------------------ few rows
// scale A x of one row at one rank a block: its 4 waves split K, lanes take 8
// inputs at a time; the waves' sums are added in wave order.  A few hundred KB
// to a few MB: bound by the latency of one chain of loads, 3.5 us for 16 rows
// of 6144 at rank 16, 4.8 for 64 (8 ranks a block, which read x once for them:
// 5.6 and 7.1 us).
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs l, const uint16_t* __restrict__ x) {
  __shared__ float part[4];
  const int r = blockIdx.x, j = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int id = l.ids[r];
  if ((uint32_t)id >= (uint32_t)l.adapters) return;
  const int rank = lora_rank(l, id);
  const int chunks = l.k / 8;  // of 8 inputs
  const int c0 = chunks * wv / 4, c1 = chunks * (wv + 1) / 4;
  const uint16_t* px = x + (size_t)r * l.k;
  const uint16_t* pa = l.a + ((size_t)id * l.max_rank + j) * l.k;
  float s = 0.f;
  if (j < rank) {
#pragma unroll 4
    for (int c = c0 + lane; c < c1; c += 64) {
      const u32x4 xv = ld16(px + 8 * c), av = ld16(pa + 8 * c);
#pragma unroll
      for (int q = 0; q < 4; q++) {
        s = fmaf(__uint_as_float(av[q] << 16), __uint_as_float(xv[q] << 16), s);
        s = fmaf(__uint_as_float(av[q] & 0xFFFF0000u), __uint_as_float(xv[q] & 0xFFFF0000u), s);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
  if (lane == 0) part[wv] = s;
  __syncthreads();
  if (tid == 0)
    l.v[(size_t)r * l.max_rank + j] =
        j < rank ? (part[0] + part[1] + part[2] + part[3]) * l.scale[id] : 0.f;
}

// base + B v of one row, an output a thread: the adapter's row of B is the
// thread's own 16 to 256 bytes.  3.7 us for 16 rows of 6144 at rank 16, 5.1 for
// 64: latency.
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs l, const uint16_t* base,
                                                          uint16_t* y) {
  __shared__ LoraRows rows;
  const int r = blockIdx.x, tid = threadIdx.x;
  const int n = blockIdx.y * 256 + tid;
  const size_t at = (size_t)r * l.n + n;
  const uint16_t b = n < l.n ? base[at] : 0;
  LoraArgs one = l;
  one.ids = l.ids + r;
  one.v = l.v + (size_t)r * l.max_rank;
  rows.load(one, 1, tid, 256);
  __syncthreads();
  if (n >= l.n) return;
  if (rows.id[0] >= 0)
    y[at] = f32_to_bf16(bf16_to_f32(b) + rows.term(one, 0, n));
  else if (y != base)
    y[at] = b;
}

// ---------------------------------------------------------------- many rows
// Rows grouped by adapter (token_rows.hip), in tiles of 32: a tile reads its
// adapter once for 32 rows, in 16x16x32 bf16 MFMAs.  Memory is read and
// written row by row, 4 or 8 neighbouring lanes to a line (where lanes took
// their MFMA operand straight from memory, neighbours in different rows, each
// cost an access: the shrink of 6001 rows of 6144 at rank 64 45 against 36 us,
// the expand 60 against 47), and each wave turns what it loaded into operand
// order through an LDS area of its own.  LDS operations of one
// wave complete in order, so these need no barrier, only the compiler's order.
constexpr int kLoraM = kLoraTile / 16;
constexpr int kLoraParts = 8;  // parts of K at most

// 16 rows of 64 bytes in LDS, the 16-byte chunks permuted by the row so that
// neither 8 nor 16 lanes with one chunk of consecutive rows share a bank.
__device__ __forceinline__ int operand_at(int row, int chunk) {
  return row * 64 + (((chunk ^ (row >> 1) ^ (row >> 3)) & 3) << 4);
}
__device__ __forceinline__ void operand_put(uint8_t* tile, int lane, const u32x4& v) {
  *reinterpret_cast<u32x4*>(tile + operand_at(lane >> 2, lane & 3)) = v;
}
__device__ __forceinline__ v8bf operand_get(const uint8_t* tile, int lane) {
  return *reinterpret_cast<const v8bf*>(tile + operand_at(lane & 15, lane >> 4));
}
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// The tile of grid column b (a multiple of 8 columns, at least as many as
// tiles).  Consecutive blocks go to the 8 XCDs in turn, each with an L2 of its
// own: XCD b % 8 takes a run of consecutive tiles, so that the tiles of one
// adapter read it through one L2.
__device__ __forceinline__ bool xcd_tile(const LoraArgs& l, int b, RowTile* t) {
  const int n = *l.n_tiles, per = (n + 7) >> 3, i = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || i >= n) return false;
  *t = l.tiles[i];
  return true;
}

// The wave of a thread, as the scalar it is: an MFMA runs whatever EXEC says,
// so a branch around one has to be a scalar branch.
__device__ __forceinline__ int wave_of(int tid) {
  return __builtin_amdgcn_readfirstlane(tid >> 6);
}

// The part of K of wave `w` of `waves`, in steps of 32.
__device__ __forceinline__ void k_range(int k, int w, int waves, int* s0, int* s1) {
  const int steps = k / 32;
  *s0 = steps * w / waves;
  *s1 = steps * (w + 1) / waves;
}

// A x of a tile over one part of K; the block's 4 waves split the part
// further and add their sums through LDS in wave order.  RT: rank tiles of 16.
// 6001 rows of 6144, 24 adapters: 22 us at rank 16, 33 at rank 64 (x alone is
// 74 MB, 11 us of memory; every tile reads its adapter again, from L2).  Its
// waves wait for loads: a wave has 6 to 12 steps of 32, 4 of them under way (no
// other depth was measured).  Tiles of 64 rows halve A's traffic: 32 us here, but
// 85 against 48 in the expand.
template <int RT>
__global__ __launch_bounds__(256, 2) void lora_shrink_tile_kernel(
    LoraArgs l, const uint16_t* __restrict__ x) {
  // operand tiles of each wave, then its sums
  __shared__ __align__(16) uint8_t lds[4][(kLoraM + RT) * 1024];
  RowTile t;
  if (!xcd_tile(l, blockIdx.x, &t) || t.group == l.adapters) return;  // (rows without an adapter)
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_of(tid), col = lane & 15, g = lane >> 4;
  uint8_t* mine = lds[wv];
  const uint16_t* px[kLoraM];
#pragma unroll
  for (int i = 0; i < kLoraM; i++) {
    const int s = t.row + 16 * i + (lane >> 2);
    px[i] = x + (size_t)l.order[s < t.end ? s : t.end - 1] * l.k + 8 * (lane & 3);
  }
  const uint16_t* pa[RT];
#pragma unroll
  for (int j = 0; j < RT; j++) {
    const int r = 16 * j + (lane >> 2);
    pa[j] = l.a + ((size_t)t.group * l.max_rank + (r < l.max_rank ? r : l.max_rank - 1)) * l.k + 8 * (lane & 3);
  }
  int s0, s1;
  k_range(l.k, (int)blockIdx.y * 4 + wv, l.k_parts * 4, &s0, &s1);
  v4f acc[kLoraM][RT];
#pragma unroll
  for (int i = 0; i < kLoraM; i++)
#pragma unroll
    for (int j = 0; j < RT; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // kDepth steps in flight (steps past the end load the last one, unused)
  constexpr int kDepth = RT <= 4 ? 4 : 2;
  struct Step {
    u32x4 x[kLoraM], a[RT];
  } st[kDepth];
  auto issue = [&](Step& d, int s) {
    s = s < s1 ? s : s1 - 1;
#pragma unroll
    for (int i = 0; i < kLoraM; i++) d.x[i] = ld16(px[i] + 32 * s);
#pragma unroll
    for (int j = 0; j < RT; j++) d.a[j] = ld16(pa[j] + 32 * s);
  };
  auto multiply = [&](const Step& d) {
    lds_order();
#pragma unroll
    for (int i = 0; i < kLoraM; i++) operand_put(mine + 1024 * i, lane, d.x[i]);
#pragma unroll
    for (int j = 0; j < RT; j++) operand_put(mine + 1024 * (kLoraM + j), lane, d.a[j]);
    lds_order();
    v8bf xv[kLoraM];
#pragma unroll
    for (int i = 0; i < kLoraM; i++) xv[i] = operand_get(mine + 1024 * i, lane);
#pragma unroll
    for (int j = 0; j < RT; j++) {
      const v8bf av = operand_get(mine + 1024 * (kLoraM + j), lane);
#pragma unroll
      for (int i = 0; i < kLoraM; i++) acc[i][j] = mfma_bf16(av, xv[i], acc[i][j]);
    }
  };
  if (s0 < s1) {  // a part of few steps may leave a wave none
#pragma unroll
    for (int p = 0; p < kDepth; p++) issue(st[p], s0 + p);
    for (int s = s0; s < s1; s += kDepth) {
#pragma unroll
      for (int p = 0; p < kDepth; p++) {
        if (s + p < s1) multiply(st[p]);
        if (s + p + kDepth < s1) issue(st[p], s + p + kDepth);
      }
    }
  }
  // lane l holds ranks 16 j + 4 (l / 16) + v of row 16 i + l % 16: sums of rank
  // tile j at floats 512 j .. of the wave's area, a row's 16 ranks together.
  // Two rank tiles a pass fit every area.
#pragma unroll
  for (int j0 = 0; j0 < RT; j0 += 2) {
    if (j0 > 0) __syncthreads();
    lds_order();
#pragma unroll
    for (int j = j0; j < RT && j < j0 + 2; j++)
#pragma unroll
      for (int i = 0; i < kLoraM; i++) {
        pin4(acc[i][j]);
        *reinterpret_cast<v4f*>(mine + (((j - j0) * kLoraM + i) * 256 + col * 16 + 4 * g) * 4) = acc[i][j];
      }
    __syncthreads();
    const int tiles = (RT - j0 < 2 ? RT - j0 : 2) * kLoraM;
    for (int q = tid; q < tiles * 64; q += 256) {
      const int c = q >> 6, e = (q & 63) * 4;
      const int row = t.row + 16 * (c % kLoraM) + e / 16, r = 16 * (j0 + c / kLoraM) + e % 16;
      if (row >= t.end || r >= l.max_rank) continue;
      v4f s = *reinterpret_cast<const v4f*>(lds[0] + (c * 256 + e) * 4);
#pragma unroll
      for (int w = 1; w < 4; w++) s += *reinterpret_cast<const v4f*>(lds[w] + (c * 256 + e) * 4);
      *reinterpret_cast<v4f*>(l.v + ((size_t)blockIdx.y * l.rows + row) * l.max_rank + r) = s;
    }
  }
}

// v as two bf16 parts of its sign, v = hi + lo within 2^-16 of it: hi is v's
// leading 8 bits.  An infinity in B has to give v's infinity, so where nothing
// is left for lo (inf * 0 is a NaN) it is 2^-24 of hi, less than a rounding of
// v (0 for a v below 2^-102 at most, and for 0), and 1 beside an infinity.
__device__ __forceinline__ void split_bf16(float v, uint16_t* hi, uint16_t* lo) {
  *hi = (uint16_t)(__float_as_uint(v) >> 16);
  const float h = bf16_to_f32(*hi), left = v - h;
  *lo = f32_to_bf16(left == 0.f ? h * 0x1p-24f : left);
  if ((*hi & 0x7F80u) == 0x7F80u) *lo = (*hi & 0x8000u) | 0x3F80u;
}

// y = bf16(base + B v) of a tile's 32 rows over a part of N, 64 outputs a wave
// at a time.  v (its K parts added in order, times scale) is split into two
// bf16 parts (one part alone: 2^-8, as much as the result's own rounding): two
// MFMAs for one.  The products go back through
// the wave's LDS area to lanes that hold 8 outputs of one row.  RS: K steps of 32 ranks; the ranks
// past the adapter's are zero in both operands.
// 6001 rows of 6144, 24 adapters: 38 us at rank 16, 52 at rank 64; base and y
// are 148 MB, 29 us of memory at the rate of a copy.
constexpr int kOutStride = 68;  // floats of a row of products in LDS (64 used)

template <int RS>
__global__ __launch_bounds__(256, 2) void lora_expand_tile_kernel(
    LoraArgs l, const uint16_t* base, uint16_t* y, int n_part) {
  constexpr int JT = RS <= 2 ? 4 : 2;  // weight tiles in LDS at once
  __shared__ __align__(16) uint16_t sv[2][kLoraTile][32 * RS + 8];  // hi, lo
  __shared__ __align__(16) uint8_t lds[4][kLoraTile * kOutStride * 4];  // weights, then products
  static_assert(JT * RS * 1024 <= (int)sizeof(lds[0]), "the weight tiles fit the wave's area");
  RowTile t;
  if (!xcd_tile(l, blockIdx.x, &t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_of(tid), col = lane & 15, g = lane >> 4;
  const int n_lo = (int)blockIdx.y * n_part, n_hi = n_lo + n_part < l.n ? n_lo + n_part : l.n;
  if (t.group == l.adapters) {  // rows without an adapter: base as it is
    if (y == base) return;
    const int last = t.end < t.row + kLoraTile ? t.end : t.row + kLoraTile;
    const int chunks = (n_hi - n_lo) / 8, total = (last - t.row) * chunks;
#pragma unroll 4
    for (int q = tid; q < total; q += 256) {
      const int m = q / chunks, c = q - m * chunks;
      const size_t at = (size_t)l.order[t.row + m] * l.n + n_lo + 8 * c;
      *reinterpret_cast<u32x4*>(y + at) = ld16(base + at);
    }
    return;
  }
  uint8_t* mine = lds[wv];
  // this lane's rows of base and y: 8 i + lane / 8, outputs n0 + 8 (lane % 8) ..
  constexpr int NB = kLoraTile / 8;
  size_t at[NB];
  bool live[NB];
#pragma unroll
  for (int i = 0; i < NB; i++) {
    const int s = t.row + 8 * i + (lane >> 3);
    live[i] = s < t.end;
    at[i] = (size_t)l.order[live[i] ? s : t.end - 1] * l.n;
  }
  const int nc = 8 * (lane & 7);
  const uint16_t* wb = l.b + (size_t)t.group * l.n * l.max_rank;
  u32x4 w[4][RS];        // weight tile j: row lane / 4, ranks 32 s + 8 (lane % 4) ..
  u32x4 b[NB], bn[NB];   // base, and the next step's
  auto issue_w = [&](int n0) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      int n = n0 + 16 * j + (lane >> 2);
      n = n < l.n ? n : l.n - 1;
#pragma unroll
      for (int s = 0; s < RS; s++) {
        const int r = 32 * s + 8 * (lane & 3);
        w[j][s] = ld16(wb + (size_t)n * l.max_rank + (r < l.max_rank ? r : 0));
      }
    }
  };
  auto issue_b = [&](u32x4 (&d)[NB], int n0) {
    const int n = n0 + nc < l.n ? n0 + nc : l.n - 8;
#pragma unroll
    for (int i = 0; i < NB; i++) d[i] = ld16(base + at[i] + n);
  };
  // the first step's loads run while v is summed
  int n0 = n_lo + 64 * wv;
  issue_b(b, n0 < n_hi ? n0 : n_lo);
  issue_w(n0 < n_hi ? n0 : n_lo);
  const int rank = lora_rank(l, t.group);
  const float scale = l.scale[t.group];
  for (int q = tid; q < kLoraTile * 8 * RS; q += 256) {
    const int m = q / (8 * RS), r = 4 * (q - m * (8 * RS));
    v4f s = {0.f, 0.f, 0.f, 0.f};
    if (t.row + m < t.end && r < rank) {
      const float* p0 = l.v + ((size_t)t.row + m) * l.max_rank + r;
#pragma unroll
      for (int p = 0; p < kLoraParts; p++)
        if (p < l.k_parts)
          s += *reinterpret_cast<const v4f*>(p0 + (size_t)p * l.rows * l.max_rank);
    }
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const float v = r + c < rank ? s[c] * scale : 0.f;
      split_bf16(v, &hi[c], &lo[c]);
    }
    *reinterpret_cast<uint2*>(&sv[0][m][r]) =
        uint2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
    *reinterpret_cast<uint2*>(&sv[1][m][r]) =
        uint2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
  }
  __syncthreads();
  for (; n0 < n_hi; n0 += 256) {
    if (n0 + 256 < n_hi) issue_b(bn, n0 + 256);
    if (rank < 32 * RS) {
#pragma unroll
      for (int s = 0; s < RS; s++) {
        const int left = rank - (32 * s + 8 * (lane & 3));
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const uint32_t keep = left >= 2 * q + 2 ? ~0u : (left == 2 * q + 1 ? 0xFFFFu : 0u);
#pragma unroll
          for (int j = 0; j < 4; j++) w[j][s][q] &= keep;
        }
      }
    }
    v4f acc[kLoraM][4];
#pragma unroll
    for (int i = 0; i < kLoraM; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += JT) {
      lds_order();
#pragma unroll
      for (int j = 0; j < JT; j++)
#pragma unroll
        for (int s = 0; s < RS; s++) operand_put(mine + 1024 * (j * RS + s), lane, w[j0 + j][s]);
      lds_order();
#pragma unroll
      for (int s = 0; s < RS; s++)
#pragma unroll
        for (int j = 0; j < JT; j++) {
          const v8bf wv8 = operand_get(mine + 1024 * (j * RS + s), lane);
#pragma unroll
          for (int i = 0; i < kLoraM; i++)
#pragma unroll
            for (int h = 1; h >= 0; h--)
              acc[i][j0 + j] = mfma_bf16(
                  wv8, *reinterpret_cast<const v8bf*>(&sv[h][16 * i + col][32 * s + 8 * g]),
                  acc[i][j0 + j]);
        }
    }
    if (n0 + 256 < n_hi) issue_w(n0 + 256);
    lds_order();
#pragma unroll
    for (int i = 0; i < kLoraM; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        pin4(acc[i][j]);  // outputs 16 j + 4 g + v of row 16 i + col
        *reinterpret_cast<v4f*>(mine + ((16 * i + col) * kOutStride + 16 * j + 4 * g) * 4) = acc[i][j];
      }
    lds_order();
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const float* p = reinterpret_cast<const float*>(mine) + (8 * i + (lane >> 3)) * kOutStride + nc;
      const v4f d0 = *reinterpret_cast<const v4f*>(p), d1 = *reinterpret_cast<const v4f*>(p + 4);
      const float d[8] = {d0[0], d0[1], d0[2], d0[3], d1[0], d1[1], d1[2], d1[3]};
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; q++)
        o[q] = (uint32_t)f32_to_bf16(__uint_as_float(b[i][q] << 16) + d[2 * q]) |
               ((uint32_t)f32_to_bf16(__uint_as_float(b[i][q] & 0xFFFF0000u) + d[2 * q + 1]) << 16);
      if (live[i] && n0 + nc < n_hi) *reinterpret_cast<u32x4*>(y + at[i] + n0 + nc) = o;
      b[i] = bn[i];
    }
  }
}

// Above rows * max_rank = 2048 the rows are grouped (measured at this n and k
// alone; more distinct adapters move the crossing up).  Kernels of one call at n
// = k = 6144, one by one and grouped, with 128 adapters and with 4: 16 rows at
// rank 128 18.5 and 25.6, 18.1 and 21.2 us; 64 rows at rank 32 15.1 and 21.6,
// 12.9 and 13.5; 128 at rank 16 15.0 and 23.4, 12.0 and 14.1; 256 at rank 16
// 21.1 and 24.5, 16.0 and 14.9; 64 at rank 64 52 and 30, 25 and 17.
constexpr int kLoraDirect = 2048;

size_t lora_plan(LoraArgs* l, void* base) {
  char* b = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = b + o;
    o = (o + bytes + 255) / 256 * 256;
    return p;
  };
  const bool grouped = (int64_t)l->rows * l->max_rank > kLoraDirect;
  l->max_tiles = 0;
  if (grouped) {
    const int groups = l->adapters + 1;
    l->max_tiles = (int)sort_max_tiles(l->rows, groups, kLoraTile);
    // K parts of at least 8 steps of 32, about 2048 blocks (512 where a rank
    // above 64 takes more registers and longer sums): shrink and expand of 6001
    // rows of 6144 61 us at rank 16 and 82 at rank 64, 64 and 83 with half as many
    int parts = (l->max_rank <= 64 ? 2048 : 512) / l->max_tiles;
    if (parts < 1) parts = 1;
    int most = l->k / 256 > 1 ? l->k / 256 : 1;
    if (most > kLoraParts) most = kLoraParts;
    l->k_parts = parts < most ? parts : most;
    l->order = (int32_t*)take((size_t)l->rows * 4);
    l->pos = (int32_t*)take((size_t)l->rows * 4);
    l->offsets = (int32_t*)take(((size_t)groups + 1) * 4);
    l->counts = (int32_t*)take(sort_workspace(l->rows, groups));
    l->n_tiles = (int32_t*)take(4);
    l->tiles = (RowTile*)take((size_t)l->max_tiles * sizeof(RowTile));
  } else {
    l->k_parts = 1;
  }
  l->v = (float*)take((size_t)l->k_parts * l->rows * l->max_rank * sizeof(float));
  return o;
}

hipError_t launch_lora_shrink(const LoraArgs& l, const uint16_t* x, hipStream_t stream) {
  hipLaunchKernelGGL(lora_shrink_kernel, dim3(l.rows, l.max_rank), dim3(256), 0, stream, l, x);
  return hipGetLastError();
}

static hipError_t launch_lora_grouped(const LoraArgs& l, const uint16_t* x, const uint16_t* base,
                                      uint16_t* y, hipStream_t stream) {
  SortArgs s = {};
  s.ids = l.ids;
  s.picks = l.rows;
  s.groups = l.adapters + 1;
  s.spill = 1;
  s.offsets = l.offsets;
  s.order = l.order;
  s.pos = l.pos;
  s.counts = l.counts;
  s.tiles = l.tiles;
  s.n_tiles = l.n_tiles;
  s.tile_rows = kLoraTile;
  hipError_t e = launch_sort(s, stream);
  if (e != hipSuccess) return e;
  const int cols = (l.max_tiles + 7) / 8 * 8;  // xcd_tile
  const dim3 gs(cols, l.k_parts);
  switch ((l.max_rank + 15) / 16) {
#define LORA_RT(R) \
  case R: hipLaunchKernelGGL(lora_shrink_tile_kernel<R>, gs, dim3(256), 0, stream, l, x); break;
    LORA_RT(1) LORA_RT(2) LORA_RT(3) LORA_RT(4) LORA_RT(5) LORA_RT(6) LORA_RT(7) LORA_RT(8)
#undef LORA_RT
  }
  // parts of N: about 1024 blocks, of 256 outputs or more (6001 rows of 6144 at
  // rank 16: 38.5 us with 5 parts, 42.6 with 4, 44.9 with 6)
  int parts = (1024 + l.max_tiles - 1) / l.max_tiles;
  const int steps = (l.n + 255) / 256;
  parts = parts < steps ? parts : steps;
  const int n_part = (steps + parts - 1) / parts * 256;
  const dim3 ge(cols, (l.n + n_part - 1) / n_part);
  switch ((l.max_rank + 31) / 32) {
#define LORA_RS(R) \
  case R: hipLaunchKernelGGL(lora_expand_tile_kernel<R>, ge, dim3(256), 0, stream, l, base, y, n_part); break;
    LORA_RS(1) LORA_RS(2) LORA_RS(3) LORA_RS(4)
#undef LORA_RS
  }
  return hipGetLastError();
}

hipError_t launch_lora(LoraArgs l, const uint16_t* x, const uint16_t* base, uint16_t* y,
                       hipStream_t stream) {
  if (l.max_tiles > 0) return launch_lora_grouped(l, x, base, y, stream);
  hipError_t e = launch_lora_shrink(l, x, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_expand_kernel, dim3(l.rows, (l.n + 255) / 256), dim3(256), 0, stream, l,
                     base, y);
  return hipGetLastError();
}

}  // namespace moe
