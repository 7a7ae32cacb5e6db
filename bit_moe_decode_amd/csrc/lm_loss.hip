// lm_loss.hip -- the LM head's softmax cross entropy over a large vocabulary and
// its gradients, without keeping the logits: with z[r, v] = w[v] . h[r],
//   lse[r]  = log sum_v exp z[r, v]
//   loss[r] = lse[r] - z[r, t_r]             (0 for a row without a target)
//   d[r, v] = (exp(z[r, v] - lse[r]) - [v = t_r]) dloss[r]     (0 without one)
//   dh[r]   = sum_v d[r, v] w[v],   dw[v] = sum_r d[r, v] h[r]
// bf16 operands; logits, exponentials and sums in fp32.
//
// Measured at 151936 tokens of 2560: the loss of 4096 rows 2510 .. 2670 us, 1.24
// PFLOP/s, of 8 rows 140 us (134 of them the weights at 5.8 TB/s).  The gradients
// of 4096 rows 7.7 .. 8.2 ms, 1.2 PFLOP/s: in ten pieces d 306 us (1.04 PFLOP/s;
// the exponentials of a tile take as long as 5 of its 40 steps and nothing runs
// beside them), dh and dw 420 .. 470 (1.4).  Of 333 rows of 32003 x 1000 145 us: 5
// for the places, 55 d, 80 dh and dw, whose tiles of 5 to 35 steps wait for their
// loads, 8 dh's sum.
#include "lm_loss.h"

#include <math.h>

#include "device_common.h"
#include "embed.h"
#include "stream_product.h"
#include "tile_product.h"

namespace moe {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The largest and the sum of a value over the four lanes of a row of sums.
__device__ __forceinline__ float over_lanes_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float over_lanes_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// A tile of the logits of rows m0 + .. and tokens j0 + ..
struct HeadTile {
  TileOperand m, j;
  int m0, j0;
};

// Calls done(sums, tile) for this block's tiles of `total`.
template <typename Stage, typename Last, typename TileAt, typename Done>
__device__ __forceinline__ void head_tiles(int total, TileAt tile_at, Stage& s0, Stage& s1, Last& s2,
                                           Done done) {
  int t = first_tile();
  if (t >= total) return;
  TilePipe<8, 8, false, false> pipe;
  HeadTile p = tile_at(t);
  pipe.start(p.m, p.j, s0, s1, s2);
  for (;;) {
    t += gridDim.x;
    const bool more = t < total;
    HeadTile next = p;
    if (more) next = tile_at(t);
    auto finish = [&](auto u) TILE_INLINE {
      TileSums<decltype(u)::value, 8> sums;
      pipe.run(s0, s1, s2, sums);
      if (more) pipe.start(next.m, next.j, s0, s1, s2);
      done(sums, p);
    };
    if (p.m.own > 128)
      finish(std::integral_constant<int, 8>{});
    else if (p.m.own > 64)
      finish(std::integral_constant<int, 4>{});
    else if (p.m.own > 32)
      finish(std::integral_constant<int, 2>{});
    else
      finish(std::integral_constant<int, 1>{});
    if (!more) return;
    p = next;
  }
}

// Rows h [rows][hidden] against `columns` rows of w in tiles of 16 U x 64: calls
// done(m, j, part, z) with the logits of row m and columns j .. j + 3, of the
// part-th 16 columns.
template <int U, typename Done>
__device__ __forceinline__ void few_tiles(const uint16_t* h, int rows, const uint16_t* w, int columns, int hidden,
                                          uint8_t* lds, Done done) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int m_tiles = (rows + 16 * U - 1) / (16 * U), j_tiles = (columns + kStreamJ - 1) / kStreamJ;
  const int tiles = m_tiles * j_tiles;
  const uint32_t pitch = (uint32_t)hidden * 2u;
  auto start = [&](StreamPipe<U>& pipe, int t) TILE_INLINE {
    const int jt = t / m_tiles, m0 = (t - jt * m_tiles) * 16 * U, j0 = jt * kStreamJ;
    pipe.start(TileOperand{h + (int64_t)m0 * hidden, pitch, rows - m0 < 16 * U ? rows - m0 : 16 * U, hidden},
               TileOperand{w + (int64_t)j0 * hidden, pitch, columns - j0 < kStreamJ ? columns - j0 : kStreamJ, hidden});
  };
  int t = blockIdx.x;
  if (t >= tiles) return;
  StreamPipe<U> pipe;
  start(pipe, t);
  for (;;) {
    const int jt = t / m_tiles, m0 = (t - jt * m_tiles) * 16 * U;
    t += gridDim.x;
    pipe.run(lds);
    if (t < tiles) start(pipe, t);
    pipe.add(lds, [&](int u, int v, const v4f& z) TILE_INLINE {
      done(m0 + 16 * u + col, jt * kStreamJ + 16 * v + 4 * g, jt * kStreamV + v, z);
    });
    if (t >= tiles) return;
  }
}

// ------------------------------------------------------------------- the loss
// A tile's logits stay in its sums: each wave leaves a row's largest logit of
// its columns and the sum of the exponentials below it, [rows][parts] of
// float2, and the logit of the row's target where it is among them.
struct LossTiles {
  LossArgs a;
  int first, count;  // rows of this launch
  int parts;         // a row's: two a column tile
  float2* part;      // [count][parts]
  float* at_target;  // [count]
};

template <int U, int V>
__device__ __forceinline__ void loss_epilogue(const LossTiles& l, TileSums<U, V>& sums, int m0, int j0, int part) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tile_wave(tid);
  const int col = lane & 15, g = lane >> 4;
  m0 += (wv & 1) * 16 * U + col;
  j0 += (wv >> 1) * 16 * V;
  part += wv >> 1;
  const bool edge = j0 + 16 * V > l.a.vocab;  // columns of the tile that are not there
#pragma unroll
  for (int u = 0; u < U; u++) {
    tile_hold(sums.s[u]);
    float z[V][4];
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        z[v][i] = sums.s[u][v][i];
        if (edge && j0 + 16 * v + 4 * g + i >= l.a.vocab) z[v][i] = -INFINITY;
      }
    float big = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; v++) big = fmaxf(big, fmaxf(fmaxf(z[v][0], z[v][1]), fmaxf(z[v][2], z[v][3])));
    big = over_lanes_max(big);
    float sum = 0.f;
    if (__ballot(fabsf(big) == INFINITY)) {  // a largest of +-inf is not subtracted from itself
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 4; i++) sum += z[v][i] == big ? 1.f : exp_of(z[v][i] - big);
    } else {
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 4; i++) sum += exp_of(z[v][i] - big);
    }
    sum = over_lanes_sum(sum);
    const int m = m0 + 16 * u;
    const bool live = m < l.count;
    if (live && g == 0) l.part[(size_t)m * l.parts + part] = float2{big, sum};
    const int t = live ? l.a.targets[l.first + m] : -1;
    const int at = t - j0;  // the target's column here
    if (__ballot((uint32_t)t < (uint32_t)l.a.vocab && (uint32_t)at < 16u * V)) {
      float f = 0.f;
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (16 * v + 4 * g + i == at) f = z[v][i];
      if ((uint32_t)t < (uint32_t)l.a.vocab && (uint32_t)at < 16u * V && ((at >> 2) & 3) == g) l.at_target[m] = f;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

__global__ __launch_bounds__(256) void lm_loss_kernel(LossTiles l) {
  using Pipe = TilePipe<8, 8, false, false>;
  constexpr int TM = 256, TJ = 256;
  __shared__ typename Pipe::Stage s0, s1;
  __shared__ typename Pipe::Last s2;
  const int m_tiles = (l.count + TM - 1) / TM, j_tiles = (l.a.vocab + TJ - 1) / TJ, H = l.a.hidden;
  auto tile_at = [&](int t) TILE_INLINE {
    int mt, jt;
    place_of(t, m_tiles, j_tiles, &mt, &jt);
    HeadTile p;
    p.m0 = mt * TM;
    p.j0 = jt * TJ;
    p.m = {l.a.h + (int64_t)(l.first + p.m0) * H, (uint32_t)H * 2u, l.count - p.m0 < TM ? l.count - p.m0 : TM, H};
    p.j = {l.a.w + (int64_t)p.j0 * H, (uint32_t)H * 2u, l.a.vocab - p.j0 < TJ ? l.a.vocab - p.j0 : TJ, H};
    return p;
  };
  head_tiles(m_tiles * j_tiles, tile_at, s0, s1, s2, [&](auto& sums, const HeadTile& p) TILE_INLINE {
    loss_epilogue(l, sums, p.m0, p.j0, p.j0 / TJ * 2);
  });
}

// In small tiles: a part is 16 columns of a row.
template <int U>
__global__ __launch_bounds__(256, 2) void lm_loss_few_kernel(LossTiles l) {
  __shared__ __align__(16) uint8_t lds[StreamPipe<U>::kLds];
  few_tiles<U>(l.a.h + (int64_t)l.first * l.a.hidden, l.count, l.a.w, l.a.vocab, l.a.hidden, lds,
               [&](int m, int j, int part, v4f z) TILE_INLINE {
    float big = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (j + i >= l.a.vocab) z[i] = -INFINITY;
      big = fmaxf(big, z[i]);
    }
    big = over_lanes_max(big);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) sum += z[i] == big ? 1.f : exp_of(z[i] - big);
    sum = over_lanes_sum(sum);
    if (m >= l.count) return;
    if ((threadIdx.x & 63) < 16) l.part[(size_t)m * l.parts + part] = float2{big, sum};
    const int t = l.a.targets[l.first + m];
    if ((uint32_t)t < (uint32_t)l.a.vocab && (uint32_t)(t - j) < 4u)
      l.at_target[m] = t - j == 0 ? z[0] : (t - j == 1 ? z[1] : (t - j == 2 ? z[2] : z[3]));
  });
}

// A row's parts joined, a block a row: the largest, then the sums below it.
__global__ __launch_bounds__(1024) void lm_loss_join_kernel(LossTiles l) {
  __shared__ float s_big[16], s_sum[16];
  const int m = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, waves = blockDim.x >> 6;
  const float2* p = l.part + (size_t)m * l.parts;
  float big = -INFINITY, sum = 0.f;
  for (int i0 = tid; i0 < l.parts; i0 += 4 * blockDim.x) {
    float2 q[4];
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const int i = i0 + n * (int)blockDim.x;
      q[n] = p[i < l.parts ? i : l.parts - 1];
      if (i >= l.parts) q[n] = float2{-INFINITY, 0.f};
    }
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const float b = fmaxf(big, q[n].x);
      sum = (big == b ? sum : sum * exp_of(big - b)) + (q[n].x == b ? q[n].y : q[n].y * exp_of(q[n].x - b));
      big = b;
    }
  }
  const float mine = big;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, kWave));
  if (lane == 0) s_big[wv] = big;
  __syncthreads();
  big = s_big[0];
  for (int w = 1; w < waves; w++) big = fmaxf(big, s_big[w]);
  sum = mine == big ? sum : sum * exp_of(mine - big);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane == 0) s_sum[wv] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = s_sum[0];
    for (int w = 1; w < waves; w++) sum += s_sum[w];
    const float lse = big + logf(sum);
    const int r = l.first + m;
    l.a.lse[r] = lse;
    l.a.loss[r] = (uint32_t)l.a.targets[r] < (uint32_t)l.a.vocab ? lse - l.at_target[m] : 0.f;
  }
}

// -------------------------------------------------------------- its gradients
// The rows that have a target, by target: the rest take no part, whatever they
// hold.  Then, for one piece of the vocabulary after the other: d of the piece in
// bf16, and from it the piece's dw and its part of dh, which is kept in fp32.
//
// d's rounding moves each term of a sum by up to 2^-8 of it.  Where a sum has
// many terms these go their own ways; but at the targets d is near -dloss, and a
// mean's dloss is the same for all rows: rounded alike, they moved all of dw and
// dh by up to 2^-8 (error 0.0026 of the gradients' size for their own rounding's
// 0.0017).  So what the rounding takes from d at a row's target is kept too, and
// added: to dh by its last kernel, to dw as more rows of the product.  In the
// order by target the rows of 256 tokens are neighbours, so that their remainders
// are a dense [rows][256] matrix of one entry a row.  An fp32 dw is to be as near
// as fp32 sums are: there the remainders of all of d are kept, and dw is a product
// of twice the rows, whose d is within 2^-16 (333 rows of 16000 tokens of 512, those
// that are no target: error 0.0017 by d in one bf16, 2.6e-6 by two, where sums in
// fp32 of an fp32 d give 1.4e-6; the gradients of 4096 rows of 151936 x 2560 take
// 11.4 ms for 8.3).  Where a weight or a row holds
// an infinity, d itself has given the infinity or NaN that the result is: it takes
// no remainder, whose 0 or other sign would make it a NaN.
struct LossGrad {
  LossGradArgs a;
  uint16_t* h;       // [rows][hidden] of the rows with a target
  uint16_t* h_rest;  // the same with 0 for what is not finite: the remainders' factor
  float2* row;       // their lse and dloss,
  int32_t* target;   // target,
  float* rest;       // d at the target less its rounding
  // the same at column target % 256 of [rows][256]; ALL: all of d less its rounding,
  // [rows][pitch]
  uint16_t* rests;
  int32_t* place;    // [rows] each row's place among them, or -1
  const int32_t* order;  // [live] the row at each place
  const int32_t* live;   // [1] their number
  int32_t* first_of;     // [ceil(vocab / 256) + 1] the first place of each 256 tokens
  int32_t* next;     // [8] an XCD's next tile of the second products
  uint16_t* d;       // [rows][pitch]
  float* acc;        // [splits][rows][hidden] of dh
  void* sort;
  int pitch, splits;
  int first, count;  // this piece's part of the vocabulary
  bool all;          // dw is fp32: the kernels' ALL
};

// Eight bf16 with 0 for those that are not finite.
__device__ __forceinline__ u32x4 finite8(u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if ((v[i] & 0x7F80u) == 0x7F80u) v[i] &= 0xFFFF0000u;
    if ((v[i] & 0x7F800000u) == 0x7F800000u) v[i] &= 0xFFFFu;
  }
  return v;
}

// The row r of place b, from h: its part in all that the places hold.
// `before`: the target at the place before, -1 without one; `live`: all places.
__device__ __forceinline__ void take_place(const LossGrad& l, int r, int b, int t, int before, int live) {
  const int tid = threadIdx.x, last = (l.a.vocab + 255) / 256;
  const u32x4* from = reinterpret_cast<const u32x4*>(l.a.h + (size_t)r * l.a.hidden);
  u32x4* to = reinterpret_cast<u32x4*>(l.h + (size_t)b * l.a.hidden);
  u32x4* to_rest = reinterpret_cast<u32x4*>(l.h_rest + (size_t)b * l.a.hidden);
  for (int i = tid; i < l.a.hidden / 8; i += 256) {
    const u32x4 v = from[i];
    to[i] = v;
    to_rest[i] = finite8(v);
  }
  if (tid < 32 && !l.all) reinterpret_cast<u32x4*>(l.rests + (size_t)b * 256)[tid] = u32x4{0u, 0u, 0u, 0u};
  for (int i = (before < 0 ? 0 : before / 256 + 1) + tid; i <= t / 256; i += 256) l.first_of[i] = b;
  if (b == live - 1)
    for (int i = t / 256 + 1 + tid; i <= last; i += 256) l.first_of[i] = live;
  if (tid == 0) {
    l.place[r] = b;
    l.target[b] = t;
    l.row[b] = float2{l.a.lse[r], l.a.dloss[r]};
  }
}
__device__ __forceinline__ void take_no_place(const LossGrad& l, int r, int live) {
  if (threadIdx.x == 0) l.place[r] = -1;
  if (r == 0 && live == 0)
    for (int i = threadIdx.x; i <= (l.a.vocab + 255) / 256; i += 256) l.first_of[i] = 0;
}

// Up to kLossRanked rows, without a sort: a block counts what its row comes
// behind, reading all targets.
__global__ __launch_bounds__(256) void lm_loss_rank_kernel(LossGrad l, int32_t* count) {
  __shared__ int s_behind[4], s_live[4], s_before[4];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const uint32_t t = (uint32_t)l.a.targets[r];
  int behind = 0, live = 0, before = -1;
  for (int i0 = tid; i0 < l.a.rows; i0 += 4 * 256) {
    uint32_t o[4];
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const int i = i0 + 256 * n;
      o[n] = (uint32_t)l.a.targets[i < l.a.rows ? i : l.a.rows - 1];
      if (i >= l.a.rows) o[n] = ~0u;
    }
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const bool in = o[n] < (uint32_t)l.a.vocab, less = in && (o[n] < t || (o[n] == t && i0 + 256 * n < r));
      live += in;
      behind += less;
      if (less) before = max(before, (int)o[n]);
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    live += __shfl_xor(live, s, kWave);
    behind += __shfl_xor(behind, s, kWave);
    before = max(before, __shfl_xor(before, s, kWave));
  }
  if (lane == 0) s_behind[wv] = behind, s_live[wv] = live, s_before[wv] = before;
  __syncthreads();
  live = s_live[0] + s_live[1] + s_live[2] + s_live[3];
  behind = s_behind[0] + s_behind[1] + s_behind[2] + s_behind[3];
  before = max(max(s_before[0], s_before[1]), max(s_before[2], s_before[3]));
  if (r == 0 && tid == 0) *count = live;
  if (t < (uint32_t)l.a.vocab)
    take_place(l, r, behind, (int)t, before, live);
  else
    take_no_place(l, r, live);
}

// More rows, sorted: block b takes row b, if it has no target, and the row at
// place b.
__global__ __launch_bounds__(256) void lm_loss_gather_kernel(LossGrad l) {
  const int b = blockIdx.x, live = *l.live;
  if ((uint32_t)l.a.targets[b] >= (uint32_t)l.a.vocab) take_no_place(l, b, live);
  if (b >= live) return;
  const int r = l.order[b];
  take_place(l, r, b, l.a.targets[r], b > 0 ? l.a.targets[l.order[b - 1]] : -1, live);
}

// What d's rounding takes from it (nothing of an infinity or NaN).
__device__ __forceinline__ float rest_of(float d) {
  const float near = bf16_to_f32(f32_to_bf16(d));
  return fabsf(near) < INFINITY ? d - near : 0.f;
}

// d at a logit z of the row at place m, whose lse and dloss are q and target t;
// what its rounding takes at the target is kept.  0 past the vocabulary.
template <bool ALL>
__device__ __forceinline__ float d_of(const LossGrad& l, float z, const float2& q, int m, int t, bool hit, bool past) {
  float p = exp_of(z - q.x);
  if (hit) {
    p = (p - 1.f) * q.y;
    const float rest = rest_of(p);
    l.rest[m] = rest;
    if constexpr (!ALL) l.rests[(size_t)m * 256 + (t & 255)] = f32_to_bf16(rest);
  } else {
    p *= q.y;
  }
  return past ? 0.f : p;
}

// d of a tile; columns past the vocabulary are 0.
template <bool ALL, int U, int V>
__device__ __forceinline__ void grad_epilogue(const LossGrad& l, TileSums<U, V>& sums, int live, int m0, int j0) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tile_wave(tid);
  const int col = lane & 15, g = lane >> 4;
  m0 += (wv & 1) * 16 * U + col;
  j0 += (wv >> 1) * 16 * V;
  const bool edge = j0 + 16 * V > l.count;
#pragma unroll
  for (int u = 0; u < U; u++) {
    tile_hold(sums.s[u]);
    const int m = m0 + 16 * u, row = m < live ? m : live - 1;
    const float2 q = l.row[row];
    const int t = l.target[row], at = t - l.first - j0;
    const bool hit = __ballot((uint32_t)at < 16u * V) != 0;
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int c = 16 * v + 4 * g + i;
        sums.s[u][v][i] = d_of<ALL>(l, sums.s[u][v][i], q, m, t, hit && c == at && m < live, edge && j0 + c >= l.count);
      }
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const size_t at_d = (size_t)m * l.pitch + j0 + 16 * v + tile_pair_at(lane);
      const u32x4 o = tile_pair(sums.s[u][v], sums.s[u][v + 1]);
      if (m < live) *reinterpret_cast<u32x4*>(l.d + at_d) = o;
      if constexpr (ALL) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          sums.s[u][v][i] = rest_of(sums.s[u][v][i]);
          sums.s[u][v + 1][i] = rest_of(sums.s[u][v + 1][i]);
        }
        const u32x4 rest = tile_pair(sums.s[u][v], sums.s[u][v + 1]);
        if (m < live) *reinterpret_cast<u32x4*>(l.rests + at_d) = rest;
      }
    }
  }
}

template <bool ALL>
__global__ __launch_bounds__(256) void lm_loss_d_kernel(LossGrad l) {
  using Pipe = TilePipe<8, 8, false, false>;
  constexpr int TM = 256, TJ = 256;
  __shared__ typename Pipe::Stage s0, s1;
  __shared__ typename Pipe::Last s2;
  if (blockIdx.x == 0 && threadIdx.x < 8) l.next[threadIdx.x] = 0;
  const int live = __builtin_amdgcn_readfirstlane(*l.live);
  const int m_tiles = (live + TM - 1) / TM, j_tiles = (l.count + TJ - 1) / TJ, H = l.a.hidden;
  auto tile_at = [&](int t) TILE_INLINE {
    int mt, jt;
    place_of(t, m_tiles, j_tiles, &mt, &jt);
    HeadTile p;
    p.m0 = mt * TM;
    p.j0 = jt * TJ;
    p.m = {l.h + (int64_t)p.m0 * H, (uint32_t)H * 2u, live - p.m0 < TM ? live - p.m0 : TM, H};
    p.j = {l.a.w + (int64_t)(l.first + p.j0) * H, (uint32_t)H * 2u, l.count - p.j0 < TJ ? l.count - p.j0 : TJ, H};
    return p;
  };
  head_tiles(m_tiles * j_tiles, tile_at, s0, s1, s2,
             [&](auto& sums, const HeadTile& p) TILE_INLINE { grad_epilogue<ALL>(l, sums, live, p.m0, p.j0); });
}

__device__ __forceinline__ void put4_bf16(uint16_t* to, const v4f& s) {
  *reinterpret_cast<uint2*>(to) = uint2{(uint32_t)f32_to_bf16(s[0]) | ((uint32_t)f32_to_bf16(s[1]) << 16),
                                        (uint32_t)f32_to_bf16(s[2]) | ((uint32_t)f32_to_bf16(s[3]) << 16)};
}

// d in small tiles.
template <int U, bool ALL>
__global__ __launch_bounds__(256, 2) void lm_loss_d_few_kernel(LossGrad l) {
  __shared__ __align__(16) uint8_t lds[StreamPipe<U>::kLds];
  if (blockIdx.x == 0 && threadIdx.x < 8) l.next[threadIdx.x] = 0;
  const int live = __builtin_amdgcn_readfirstlane(*l.live);
  if (live == 0) return;
  few_tiles<U>(l.h, live, l.a.w + (int64_t)l.first * l.a.hidden, l.count, l.a.hidden, lds,
               [&](int m, int j, int, v4f z) TILE_INLINE {
    if (m >= live) return;
    const float2 q = l.row[m];
    const int t = l.target[m];
#pragma unroll
    for (int i = 0; i < 4; i++) z[i] = d_of<ALL>(l, z[i], q, m, t, t - l.first == j + i, j + i >= l.count);
    put4_bf16(l.d + (size_t)m * l.pitch + j, z);
    if constexpr (ALL) {
#pragma unroll
      for (int i = 0; i < 4; i++) z[i] = rest_of(z[i]);
      put4_bf16(l.rests + (size_t)m * l.pitch + j, z);
    }
  });
}

// The two products of a piece's d, in one launch: the tiles of dh, which are
// long (the piece's columns), first, then those of dw (the rows).  Each XCD has
// its eighth of either, whose tiles its blocks take one after the other, so that
// tiles under way at once share operands in its L2; then those left of others.
struct GradTile {
  TileOperand m, j;
  int m0, j0, split;  // split -1: of dw
};

template <int SIDE, bool ALL>
struct GradTiles {
  int h_tiles, v_tiles, m_tiles, dh, dw;  // tiles a side, and in all
  int part;                               // columns of a split
  __device__ __forceinline__ GradTiles(const LossGrad& l, int live) {
    h_tiles = (l.a.hidden + SIDE - 1) / SIDE;
    v_tiles = (l.count + SIDE - 1) / SIDE;
    m_tiles = (live + SIDE - 1) / SIDE;
    dh = l.a.dh ? m_tiles * h_tiles * l.splits : 0;
    dw = l.a.dw ? v_tiles * h_tiles : 0;
    part = ((l.count + kStepC - 1) / kStepC + l.splits - 1) / l.splits * kStepC;
  }
  __device__ __forceinline__ GradTile dh_at(const LossGrad& l, int live, int t) const {
    const int H = l.a.hidden;
    GradTile p;
    p.split = t / (m_tiles * h_tiles);
    int mt, jt;
    place_of(t - p.split * (m_tiles * h_tiles), m_tiles, h_tiles, &mt, &jt);
    p.m0 = mt * SIDE;
    p.j0 = jt * SIDE;
    const int c0 = p.split * part, left = l.count - c0, c = left < 0 ? 0 : (left < part ? left : part);
    // (d's columns past the vocabulary are 0, to a multiple of 8)
    p.m = {l.d + (int64_t)p.m0 * l.pitch + (c ? c0 : 0), (uint32_t)l.pitch * 2u, live - p.m0 < SIDE ? live - p.m0 : SIDE,
           (c + 7) / 8 * 8};
    p.j = {l.a.w + (int64_t)(l.first + (c ? c0 : 0)) * H + p.j0, (uint32_t)H * 2u, H - p.j0 < SIDE ? H - p.j0 : SIDE, c};
    return p;
  }
  __device__ __forceinline__ GradTile dw_at(const LossGrad& l, int live, int t) const {
    const int H = l.a.hidden;
    GradTile p;
    p.split = -1;
    int mt, jt;
    place_of(t, v_tiles, h_tiles, &mt, &jt);
    p.m0 = mt * SIDE;
    p.j0 = jt * SIDE;
    const int own = l.count - p.m0 < SIDE ? (l.count - p.m0 + 7) / 8 * 8 : SIDE, cols = H - p.j0 < SIDE ? H - p.j0 : SIDE;
    if constexpr (ALL) {  // all rows, and all of them again with d's remainders
      p.m = {l.d + p.m0, (uint32_t)l.pitch * 2u, own, live, l.rests + p.m0, (uint32_t)l.pitch * 2u, live};
      p.j = {l.h + p.j0, (uint32_t)H * 2u, cols, live, l.h_rest + p.j0, (uint32_t)H * 2u, live};
      return p;
    }
    const int r0 = __builtin_amdgcn_readfirstlane(l.first_of[(l.first + p.m0) / 256]);
    const int more = __builtin_amdgcn_readfirstlane(l.first_of[(l.first + p.m0) / 256 + 1]) - r0;
    p.m = {l.d + p.m0, (uint32_t)l.pitch * 2u, own, live, l.rests + (int64_t)r0 * 256 + p.m0 % 256, 512u, more};
    p.j = {l.h + p.j0, (uint32_t)H * 2u, cols, live, l.h_rest + (int64_t)r0 * H + p.j0, (uint32_t)H * 2u, more};
    return p;
  }
};

template <int U, typename T, bool ADD>
__global__ __launch_bounds__(256) void lm_loss_products_kernel(LossGrad l) {
  using Long = TilePipe<U, U, false, true>;
  using Wide = TilePipe<U, U, true, true, true>;
  static_assert(sizeof(typename Long::Stage) == sizeof(typename Wide::Stage), "both take the same stages");
  __shared__ typename Long::Stage s0, s1;
  __shared__ typename Long::Last s2;
  __shared__ int s_next;
  const int live = __builtin_amdgcn_readfirstlane(*l.live), tid = threadIdx.x;
  const GradTiles<32 * U, sizeof(T) == 4> g(l, live);
  // a tile's number: those of dh, then those of dw; each XCD has an eighth of either
  TileQueues queues{l.next};
  auto redeem = [&](int ticket) TILE_INLINE {
    return queues.redeem(
        ticket, &s_next,
        [&](int q) TILE_INLINE { return eighth(g.dh, q + 1) - eighth(g.dh, q) + eighth(g.dw, q + 1) - eighth(g.dw, q); },
        [&](int q, int i) TILE_INLINE {
          const int n = eighth(g.dh, q + 1) - eighth(g.dh, q);
          return i < n ? eighth(g.dh, q) + i : g.dh + eighth(g.dw, q) + i - n;
        });
  };
  int t = redeem(tid == 0 ? queues.ticket() : 0);
  if (t < 0) return;
  Long dh;
  Wide dw;
  int m0, j0, split, own;  // the tile that is under way
  auto begin = [&](int n) TILE_INLINE {
    const GradTile p = n < g.dh ? g.dh_at(l, live, n) : g.dw_at(l, live, n - g.dh);
    m0 = __builtin_amdgcn_readfirstlane(p.m0);
    j0 = __builtin_amdgcn_readfirstlane(p.j0);
    split = __builtin_amdgcn_readfirstlane(p.split);
    own = __builtin_amdgcn_readfirstlane(p.m.own);
    if (n < g.dh)
      dh.start(p.m, p.j, s0, s1, s2);
    else
      dw.start(p.m, p.j, s0, s1, s2);
  };
  begin(t);
  while (t >= 0) {
    const int ticket = tid == 0 ? queues.ticket() : 0;
    const int m = m0, j = j0;
    if (split < 0) {
      TileSums<U, U> sums;
      dw.run(s0, s1, s2, sums);
      t = redeem(ticket);
      if (t >= 0) begin(t);
      store_tile<U, U, T, ADD>(sums, reinterpret_cast<T*>(l.a.dw) + (int64_t)l.first * l.a.hidden, m, l.count, j,
                               l.a.hidden);
    } else {
      float* acc = l.acc + (int64_t)split * l.a.rows * l.a.hidden;
      auto finish = [&](auto u) TILE_INLINE {
        TileSums<decltype(u)::value, U> sums;
        dh.run(s0, s1, s2, sums);
        const bool none = dh.halves == 0;
        t = redeem(ticket);
        if (t >= 0) begin(t);
        if (l.first == 0)  // kept, or added to what earlier pieces left
          store_tile<decltype(u)::value, U, float, false>(sums, acc, m, live, j, l.a.hidden);
        else if (!none)
          store_tile<decltype(u)::value, U, float, true>(sums, acc, m, live, j, l.a.hidden);
      };
      if (U == 8 && own > 128)
        finish(std::integral_constant<int, U>{});
      else if (own > 64)
        finish(std::integral_constant<int, 4>{});
      else if (own > 32)
        finish(std::integral_constant<int, 2>{});
      else
        finish(std::integral_constant<int, 1>{});
    }
  }
}

// dh from its parts, in order, and what d's rounding took at the target; 0 for a
// row without a target.
__global__ __launch_bounds__(256) void lm_loss_dh_kernel(LossGrad l) {
  const int r = blockIdx.x, at = l.place[r], H = l.a.hidden;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= H) return;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  if (at >= 0) {
    const float rest = l.rest[at];
    const uint2 w = *reinterpret_cast<const uint2*>(l.a.w + (size_t)l.target[at] * H + c);
    for (int i = 0; i < l.splits; i++)
      s += *reinterpret_cast<const v4f*>(l.acc + ((size_t)i * l.a.rows + at) * H + c);
    const float f[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u)};
#pragma unroll
    for (int i = 0; i < 4; i++) s[i] = fabsf(f[i]) < INFINITY ? fmaf(rest, f[i], s[i]) : s[i];
  }
  put4_bf16(l.a.dh + (size_t)r * H + c, s);
}

// --------------------------------------------------------------------- launches
// Rows of a launch of the loss, for its parts' memory.
constexpr int kLossRows = 16384;
// Tiles of 256 x 256 where three quarters of the CUs or more have one, of 64 x 64
// else (158 rows of 4353 tokens x 2304 20 us, in large tiles 55; 115 of 23056 x 3200
// 58 and 78; but 1656 of 3222 x 328 33 and 24).
constexpr int kLossTiles = 192;
static bool loss_large(int rows, int columns) {
  return rows > kStreamM && (int64_t)((rows + 255) / 256) * ((columns + 255) / 256) >= kLossTiles;
}
static int64_t small_tiles(int rows, int columns) {
  return (int64_t)((rows + kStreamM - 1) / kStreamM) * ((columns + kStreamJ - 1) / kStreamJ);
}

template <typename Args>
static void launch_few(void (*u1)(Args), void (*u2)(Args), void (*u4)(Args), int rows, int blocks, const Args& l,
                       hipStream_t stream) {
  hipLaunchKernelGGL((rows > 32 ? u4 : rows > 16 ? u2 : u1), dim3(blocks), dim3(256), 0, stream, l);
}

static int loss_parts(int rows, int vocab) {
  return loss_large(rows, vocab) ? 2 * ((vocab + 255) / 256) : kStreamV * ((vocab + kStreamJ - 1) / kStreamJ);
}
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Parts of all rows of a launch, at most: the last of several may have fewer rows,
// and take the small tiles.
static size_t all_parts(int rows, int vocab) {
  if (rows <= kLossRows) return (size_t)rows * loss_parts(rows, vocab);
  int few = kLossTiles / ((vocab + 255) / 256) * 256;  // rows that may take the small tiles
  few = few < kStreamM ? kStreamM : (few < kLossRows ? few : kLossRows);
  const size_t large = (size_t)kLossRows * loss_parts(kLossRows, vocab), small = (size_t)few * loss_parts(1, vocab);
  return large > small ? large : small;
}

size_t loss_workspace(int rows, int vocab, int) {
  return up256(all_parts(rows, vocab) * sizeof(float2)) + up256((size_t)(rows < kLossRows ? rows : kLossRows) * 4);
}

hipError_t launch_loss(const LossArgs& a, void* workspace, hipStream_t stream) {
  LossTiles l = {};
  l.a = a;
  l.part = static_cast<float2*>(workspace);
  l.at_target = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(all_parts(a.rows, a.vocab) * sizeof(float2)));
  for (l.first = 0; l.first < a.rows; l.first += kLossRows) {
    l.count = a.rows - l.first < kLossRows ? a.rows - l.first : kLossRows;
    l.parts = loss_parts(l.count, a.vocab);
    int blocks;
    const bool few = !loss_large(l.count, a.vocab);
    const int64_t tiles = few ? small_tiles(l.count, a.vocab)
                              : (int64_t)((l.count + 255) / 256) * ((a.vocab + 255) / 256);
    hipError_t e = tile_blocks(tiles, few ? 2 : 1, &blocks);
    if (e != hipSuccess) return e;
    if (few)
      launch_few(lm_loss_few_kernel<1>, lm_loss_few_kernel<2>, lm_loss_few_kernel<4>, l.count, blocks, l, stream);
    else
      hipLaunchKernelGGL(lm_loss_kernel, dim3(blocks), dim3(256), 0, stream, l);
    hipLaunchKernelGGL(lm_loss_join_kernel, dim3(l.count), dim3(l.parts > 2048 ? 1024 : 256), 0, stream, l);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Rows up to which each one's place is counted (4096 rows of 2560 21 us, sorted and
// gathered 38; 333 of 1000 5.1 and 17).
constexpr int kLossRanked = 4096;

// Columns of a piece: d of at most 128 MB, in multiples of 256, and room for as much
// again, the remainders of an fp32 dw's.
constexpr size_t kLossPieceBytes = (size_t)128 << 20;

// Side of the second products' tiles: 256 where dw has one for each CU, 128 else
// (with the small tiles of d, 529 rows of 2661 tokens x 864 118 -> 53 us).
static int grad_side(const LossGradArgs& a) {
  return (int64_t)((a.vocab + 255) / 256) * ((a.hidden + 255) / 256) >= 256 ? 256 : 128;
}

static size_t loss_grad_plan(LossGrad* l, char* base) {
  const LossGradArgs& a = l->a;
  const int whole = (a.vocab + 255) / 256;
  int64_t most = (int64_t)(kLossPieceBytes / ((size_t)a.rows * 512));
  most = most < 1 ? 1 : (most < whole ? most : whole);
  const int pieces = (int)((whole + most - 1) / most);
  l->pitch = (whole + pieces - 1) / pieces * 256;
  l->all = a.f32 && a.dw;
  // dh's products split over a piece's columns where its tiles are fewer than the
  // CUs: parts of at least 32 steps (16 of small tiles), 32 of them at most
  const int side = grad_side(a);
  const int64_t tiles = (int64_t)((a.rows + side - 1) / side) * ((a.hidden + side - 1) / side);
  int64_t splits = 256 / tiles;
  const int64_t by_steps = l->pitch / ((side / 8) * kStepC);
  if (splits > by_steps) splits = by_steps;
  l->splits = splits < 1 ? 1 : (splits > 32 ? 32 : (int)splits);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = base + o;
    o += up256(bytes);
    return p;
  };
  const size_t R = a.rows;
  l->h = reinterpret_cast<uint16_t*>(take(R * a.hidden * 2));
  l->h_rest = reinterpret_cast<uint16_t*>(take(R * a.hidden * 2));
  l->row = reinterpret_cast<float2*>(take(R * sizeof(float2)));
  l->target = reinterpret_cast<int32_t*>(take(R * 4));
  l->place = reinterpret_cast<int32_t*>(take(R * 4));
  l->rest = reinterpret_cast<float*>(take(R * 4));
  l->first_of = reinterpret_cast<int32_t*>(take(((size_t)whole + 1) * 4));
  l->sort = take(a.rows <= kLossRanked ? 4 : id_sort_workspace(a.rows, a.vocab));
  l->next = reinterpret_cast<int32_t*>(take(8 * 4));
  l->d = reinterpret_cast<uint16_t*>(take(R * l->pitch * 2));
  l->rests = reinterpret_cast<uint16_t*>(take(R * l->pitch * 2));  // (pitch: 256 or more)
  l->acc = reinterpret_cast<float*>(take((size_t)l->splits * R * a.hidden * 4));
  return o;
}

size_t loss_backward_workspace(int rows, int vocab, int hidden) {
  LossGrad l = {};
  l.a.rows = rows;
  l.a.vocab = vocab;
  l.a.hidden = hidden;
  return loss_grad_plan(&l, nullptr);
}

template <bool ALL>
static void launch_d(const LossGrad& l, bool few, int blocks, hipStream_t stream) {
  if (few)
    launch_few(lm_loss_d_few_kernel<1, ALL>, lm_loss_d_few_kernel<2, ALL>, lm_loss_d_few_kernel<4, ALL>, l.a.rows, blocks, l,
               stream);
  else
    hipLaunchKernelGGL(lm_loss_d_kernel<ALL>, dim3(blocks), dim3(256), 0, stream, l);
}

template <int U>
static void launch_products(const LossGrad& l, int blocks, hipStream_t stream) {
  if (l.a.f32 && l.a.add)
    hipLaunchKernelGGL((lm_loss_products_kernel<U, float, true>), dim3(blocks), dim3(256), 0, stream, l);
  else if (l.a.f32)
    hipLaunchKernelGGL((lm_loss_products_kernel<U, float, false>), dim3(blocks), dim3(256), 0, stream, l);
  else if (l.a.add)
    hipLaunchKernelGGL((lm_loss_products_kernel<U, uint16_t, true>), dim3(blocks), dim3(256), 0, stream, l);
  else
    hipLaunchKernelGGL((lm_loss_products_kernel<U, uint16_t, false>), dim3(blocks), dim3(256), 0, stream, l);
}

hipError_t launch_loss_backward(const LossGradArgs& a, void* workspace, hipStream_t stream) {
  LossGrad l = {};
  l.a = a;
  loss_grad_plan(&l, static_cast<char*>(workspace));
  hipError_t e = hipSuccess;
  if (a.rows <= kLossRanked) {
    int32_t* count = static_cast<int32_t*>(l.sort);
    l.live = count;
    hipLaunchKernelGGL(lm_loss_rank_kernel, dim3(a.rows), dim3(256), 0, stream, l, count);
  } else {
    int32_t* order;
    e = launch_id_sort(a.targets, a.rows, a.vocab, l.sort, nullptr, 0, &order, &l.live, stream);
    if (e != hipSuccess) return e;
    l.order = order;
    hipLaunchKernelGGL(lm_loss_gather_kernel, dim3(a.rows), dim3(256), 0, stream, l);
  }
  for (l.first = 0; l.first < a.vocab; l.first += l.pitch) {
    l.count = a.vocab - l.first < l.pitch ? a.vocab - l.first : l.pitch;
    int blocks;
    const bool few = !loss_large(a.rows, l.count);
    const int64_t tiles = few ? small_tiles(a.rows, l.count)
                              : (int64_t)((a.rows + 255) / 256) * ((l.count + 255) / 256);
    e = tile_blocks(tiles, few ? 2 : 1, &blocks);
    if (e != hipSuccess) return e;
    if (l.all)
      launch_d<true>(l, few, blocks, stream);
    else
      launch_d<false>(l, few, blocks, stream);
    const int side = grad_side(a);
    const int64_t products = ((int64_t)((a.rows + side - 1) / side) * l.splits + (l.count + side - 1) / side) *
                             ((a.hidden + side - 1) / side);
    e = tile_blocks(products, 1, &blocks);
    if (e != hipSuccess) return e;
    if (side == 256)
      launch_products<8>(l, blocks, stream);
    else
      launch_products<4>(l, blocks, stream);
  }
  if (a.dh)
    hipLaunchKernelGGL(lm_loss_dh_kernel, dim3(a.rows, (a.hidden + 1023) / 1024), dim3(256), 0, stream, l);
  return hipGetLastError();
}

}  // namespace moe
