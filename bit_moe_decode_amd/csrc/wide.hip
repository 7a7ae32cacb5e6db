// wide.hip -- the experts' step for any number of token rows whose routing
// (picks and gates) is given: the FP8 activation blocks of every token, the
// sort of the picks by expert (token_rows.hip), the experts' up/gate and down
// products over the sorted rows, and the gate-weighted sum back.
//
// The arithmetic is the decode step's: u = bf16(x * gamma); FP8 E4M3 codes of
// u per 1x128 block with scale amax/448; gate and up as FP8 x FP8 products
// per 128 of K, scaled and summed in fp32; mid = silu(gate) * up, re-quantised
// per 1x128 block; down likewise; out = bf16(sum_j g_j y_j + y_shared).  The
// row's rstd is folded into its activation scales (one fp32 rounding; the
// decode step multiplies the finished sum).  y stays in fp32 between the down
// products and the sum: rounding it to bf16 would halve that traffic and add
// an error as large as the output's own rounding.
#include "wide.h"

#include "device_common.h"

namespace moe {

// ------------------------------------------------------- activation blocks
// A block takes one token: 8 columns a lane, a 1x128 block in 16 lanes.
__global__ __launch_bounds__(256) void moe_wide_act_kernel(WideArgs a, const uint16_t* __restrict__ x,
                                                           const uint16_t* __restrict__ gamma) {
  __shared__ float s_ss[4];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const uint16_t* row = x + t * a.H;
  float ss = 0.f, sc[8];
#pragma unroll
  for (int it = 0; it < 8; it++) {  // H <= 16384
    const int c = (it * 256 + tid) * 8;
    sc[it] = 0.f;
    if (c >= a.H) continue;  // whole rows of 16 lanes
    const u32x4 xv = ld16(row + c), gv = ld16(gamma + c);
    float u[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float xf = __uint_as_float(i & 1 ? xv[i >> 1] & 0xFFFF0000u : xv[i >> 1] << 16);
      const float gf = __uint_as_float(i & 1 ? gv[i >> 1] & 0xFFFF0000u : gv[i >> 1] << 16);
      ss = fmaf(xf, xf, ss);
      u[i] = bf16_to_f32(f32_to_bf16(xf * gf));
      m = fmaxf(m, fabsf(u[i]));
    }
    const float s = __uint_as_float(row16_umax(__float_as_uint(m))) / 448.0f;
    sc[it] = s;
    uint2 q = {0u, 0u};
    if (s > 0.f) {
      q.x = f32x2_to_e4m3(u[0] / s, u[1] / s) | (f32x2_to_e4m3(u[2] / s, u[3] / s) << 16);
      q.y = f32x2_to_e4m3(u[4] / s, u[5] / s) | (f32x2_to_e4m3(u[6] / s, u[7] / s) << 16);
    }
    *reinterpret_cast<uint2*>(a.act_q + t * a.H + c) = q;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o, kWave);
  if (lane == 0) s_ss[tid >> 6] = ss;
  __syncthreads();
  const float rstd = 1.0f / sqrtf((s_ss[0] + s_ss[1] + s_ss[2] + s_ss[3]) / (float)a.H + a.eps);
#pragma unroll
  for (int it = 0; it < 8; it++) {
    const int c = (it * 256 + tid) * 8;
    if (c < a.H && (tid & 15) == 0) a.act_s[t * (a.H / 128) + c / 128] = sc[it] * rstd;
  }
}

// ------------------------------------------------------------ the products
// A block computes BM sorted rows of one expert against 256 weight rows (the
// gate and up rows of 128 mid columns, or 256 down rows), K in steps of 128.
// Each step's codes go through LDS in rows of 128 bytes whose 16-byte chunks
// are permuted by the row, so that the 16 rows a wave reads at one chunk fall
// on distinct banks.  The weights are the MFMA's A operand (their 16 rows its
// output rows: a lane holds 4 consecutive columns of one sorted row), the
// sorted rows its B operand.  After each step the fp32 products are scaled by
// weight scale times row scale and added.
__device__ __forceinline__ int lds_at(int row, int chunk) {
  return row * 128 + ((chunk ^ row ^ (row >> 3)) & 7) * 16;
}

template <int MT, int WM>
struct WideTile {
  static constexpr int BM = 16 * MT * WM;    // sorted rows
  static constexpr int kThreads = 256 * WM;  // WM x 4 waves, MT x 4 MFMA tiles each
  static constexpr int kChunksA = BM * 8, kChunksW = 256 * 8;  // 16-byte chunks a step
  static constexpr int NA = (kChunksA + kThreads - 1) / kThreads, NW = kChunksW / kThreads;
  static constexpr int kLds = (BM + 256) * 128;
};

template <int MT, int WM, bool UG>
__global__ __launch_bounds__(256 * WM) void moe_wide_gemm_kernel(WideArgs a, WideWeights w) {
  using C = WideTile<MT, WM>;
  __shared__ __align__(16) uint8_t lds[C::kLds];
  __shared__ float s_as[C::BM];
  __shared__ float s_max[4][C::BM];
  if ((int)blockIdx.y >= *a.n_tiles) return;
  const RowTile tile = a.tiles[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int wn = wv & 3, wm = wv >> 2, col = lane & 15, g = lane >> 4;
  const bool sh = tile.group == a.E;
  const int K = UG ? a.H : a.I, N = UG ? a.I : a.H, nkb = K / 128;
  const int nb = blockIdx.x;  // UG: 128 mid columns; down: 256 output columns
  const int64_t ew = sh ? 0 : (int64_t)tile.group * N * K;
  const int64_t es = sh ? 0 : (int64_t)tile.group * (N / 128) * nkb;
  const uint8_t* w0 = (UG ? (sh ? w.sg_c : w.gate_c) : (sh ? w.sd_c : w.down_c)) + ew;
  const uint8_t* w1 = UG ? (sh ? w.su_c : w.up_c) + ew : w0;
  const float* s0 = (UG ? (sh ? w.sg_s : w.gate_s) : (sh ? w.sd_s : w.down_s)) + es;
  const float* s1 = UG ? (sh ? w.su_s : w.up_s) + es : s0;
  // weight rows of the block: half h (0, 1) starts at row n0[h]; a half past
  // the end of the down matrix repeats its last and is not stored
  const int n0 = UG ? nb * 128 : nb * 256;
  const int n1 = UG ? n0 : (n0 + 128 < N ? n0 + 128 : n0);
  const float* ps0 = s0 + (int64_t)(n0 / 128) * nkb;
  const float* ps1 = s1 + (int64_t)(n1 / 128) * nkb;

  // this thread's chunks of a step: weights, then sorted rows (those past the
  // tile's end repeat its last row)
  const uint8_t* pw[C::NW];
#pragma unroll
  for (int i = 0; i < C::NW; i++) {
    const int q = tid + i * C::kThreads, r = q >> 3;
    const uint8_t* base = r < 128 ? w0 + (int64_t)(n0 + r) * K : w1 + (int64_t)(n1 + r - 128) * K;
    pw[i] = base + (q & 7) * 16;
  }
  const uint8_t* pa[C::NA];
  auto source_row = [&](int i) -> int64_t {  // row of the activations for sorted row i of the tile
    int s = tile.row + i;
    if (s >= tile.end) s = tile.end - 1;
    if (!UG) return s;
    return s < a.picks ? a.order[s] >> 3 : s - a.picks;
  };
#pragma unroll
  for (int i = 0; i < C::NA; i++) {
    const int q = tid + i * C::kThreads;
    const int64_t r = q < C::kChunksA ? source_row(q >> 3) : 0;
    pa[i] = (UG ? a.act_q : a.mid_q) + r * K + (q & 7) * 16;
  }
  const float* psa = (UG ? a.act_s : a.mid_s) + (tid < C::BM ? source_row(tid) : 0) * nkb;

  u32x4 rw[C::NW], ra[C::NA];
  float rs = 0.f;
  auto issue = [&](int kb) {
#pragma unroll
    for (int i = 0; i < C::NW; i++) rw[i] = ld16(pw[i] + kb * 128);
#pragma unroll
    for (int i = 0; i < C::NA; i++)
      if (tid + i * C::kThreads < C::kChunksA) ra[i] = ld16(pa[i] + kb * 128);
    if (tid < C::BM) rs = psa[kb];
  };
  float acc[MT][4][4];  // [sorted-row tile][weight tile: 2 of half 0, 2 of half 1][4 columns]
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int v = 0; v < 4; v++) acc[i][j][v] = 0.f;

  issue(0);
  for (int kb = 0; kb < nkb; kb++) {
    __syncthreads();  // every wave is done with the last step's codes
#pragma unroll
    for (int i = 0; i < C::NW; i++) {
      const int q = tid + i * C::kThreads;
      *reinterpret_cast<u32x4*>(lds + lds_at(q >> 3, q & 7)) = rw[i];
    }
#pragma unroll
    for (int i = 0; i < C::NA; i++) {
      const int q = tid + i * C::kThreads;
      if (q < C::kChunksA) *reinterpret_cast<u32x4*>(lds + lds_at(256 + (q >> 3), q & 7)) = ra[i];
    }
    if (tid < C::BM) s_as[tid] = rs;
    const float sw[2] = {ps0[kb], ps1[kb]};
    if (kb + 1 < nkb) issue(kb + 1);
    __syncthreads();
    v8i op[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int r = (j >> 1) * 128 + wn * 32 + (j & 1) * 16 + col;
      op[j] = cat8(ld16(lds + lds_at(r, g)), ld16(lds + lds_at(r, g + 4)));
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const int m = (wm * MT + i) * 16 + col;
      const v8i b = cat8(ld16(lds + lds_at(256 + m, g)), ld16(lds + lds_at(256 + m, g + 4)));
      const float as = s_as[m];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const v4f c = mfma_fp8(op[j], b);
        const float s = as * sw[j >> 1];
#pragma unroll
        for (int v = 0; v < 4; v++) acc[i][j][v] = fmaf(c[v], s, acc[i][j][v]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) pin4(acc[i][j]);

  if constexpr (UG) {
    // mid of columns 32 wn + 16 j + 4 g + v, j < 2, then its 1x128 block's
    // largest value over the 4 waves of the row
#pragma unroll
    for (int i = 0; i < MT; i++) {
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
          const float gt = acc[i][j][v];
          const float mid = gt / (1.0f + __expf(-gt)) * acc[i][j + 2][v];
          acc[i][j][v] = mid;
          mx = fmaxf(mx, fabsf(mid));
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
      mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
      if (g == 0) s_max[wn][(wm * MT + i) * 16 + col] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const int m = (wm * MT + i) * 16 + col;
      const int row = tile.row + m;
      if (row >= tile.end) continue;
      const float s = fmaxf(fmaxf(s_max[0][m], s_max[1][m]), fmaxf(s_max[2][m], s_max[3][m])) / 448.0f;
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint32_t q = 0u;
        if (s > 0.f)
          q = f32x2_to_e4m3(acc[i][j][0] / s, acc[i][j][1] / s) |
              (f32x2_to_e4m3(acc[i][j][2] / s, acc[i][j][3] / s) << 16);
        *reinterpret_cast<uint32_t*>(a.mid_q + (int64_t)row * N + n0 + wn * 32 + j * 16 + 4 * g) = q;
      }
      if (wn == 0 && g == 0) a.mid_s[(int64_t)row * (N / 128) + nb] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const int row = tile.row + (wm * MT + i) * 16 + col;
      if (row >= tile.end) continue;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int n = n0 + (j >> 1) * 128 + wn * 32 + (j & 1) * 16 + 4 * g;
        if (n < N)
          *reinterpret_cast<v4f*>(a.y + (int64_t)row * N + n) =
              v4f{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      }
    }
  }
}

// out[t] = bf16( sum_j g[t,j] y[pos[t,j]] + y[picks + t] ), in pick order.
__global__ __launch_bounds__(256) void moe_wide_combine_kernel(WideArgs a,
                                                               const float* __restrict__ gates,
                                                               uint16_t* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= a.H) return;
  v4f f[9];
  float gw[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int p = a.pos[t * 8 + j];
    gw[j] = p >= 0 ? gates[t * 8 + j] : 0.f;
    f[j] = p >= 0 ? *reinterpret_cast<const v4f*>(a.y + (int64_t)p * a.H + c) : v4f{0.f, 0.f, 0.f, 0.f};
  }
  f[8] = a.shared ? *reinterpret_cast<const v4f*>(a.y + (a.picks + t) * a.H + c) : v4f{0.f, 0.f, 0.f, 0.f};
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int v = 0; v < 4; v++) {
#pragma unroll
    for (int j = 0; j < 8; j++) o[v] = fmaf(gw[j], f[j][v], o[v]);
    o[v] += f[8][v];
  }
  uint2 q;
  q.x = (uint32_t)f32_to_bf16(o[0]) | ((uint32_t)f32_to_bf16(o[1]) << 16);
  q.y = (uint32_t)f32_to_bf16(o[2]) | ((uint32_t)f32_to_bf16(o[3]) << 16);
  *reinterpret_cast<uint2*>(out + t * a.H + c) = q;
}

int wide_tile_rows(int64_t picks, int experts) {
  const int64_t per = picks / experts;
  return per <= 16 ? 16 : (per <= 48 ? 32 : (per <= 96 ? 64 : 128));
}

int wide_max_tiles(int64_t picks, int experts, int shared_rows, int tile_rows) {
  return (int)(sort_max_tiles(picks, experts, tile_rows) + (shared_rows + tile_rows - 1) / tile_rows);
}

template <int MT, int WM>
static void launch_products(const WideArgs& a, const WideWeights& w, hipStream_t stream) {
  hipLaunchKernelGGL((moe_wide_gemm_kernel<MT, WM, true>), dim3(a.I / 128, a.max_tiles),
                     dim3(256 * WM), 0, stream, a, w);
  hipLaunchKernelGGL((moe_wide_gemm_kernel<MT, WM, false>), dim3((a.H + 255) / 256, a.max_tiles),
                     dim3(256 * WM), 0, stream, a, w);
}

hipError_t launch_wide(const WideArgs& a, const WideWeights& w, const uint16_t* x,
                       const int32_t* ids, const float* gates, uint16_t* out, hipStream_t stream) {
  hipLaunchKernelGGL(moe_wide_act_kernel, dim3(a.tokens), dim3(256), 0, stream, a, x, w.gamma);
  SortArgs s = {};
  s.ids = ids;
  s.picks = a.picks;
  s.groups = a.E;
  s.offsets = a.offsets;
  s.order = a.order;
  s.pos = a.pos;
  s.counts = a.counts;
  s.tiles = a.tiles;
  s.n_tiles = a.n_tiles;
  s.tile_rows = a.tile_rows;
  s.extra = a.shared ? a.tokens : 0;
  hipError_t e = launch_sort(s, stream);
  if (e != hipSuccess) return e;
  switch (a.tile_rows) {
    case 16: launch_products<1, 1>(a, w, stream); break;
    case 32: launch_products<2, 1>(a, w, stream); break;
    case 64: launch_products<4, 1>(a, w, stream); break;
    default: launch_products<4, 2>(a, w, stream); break;
  }
  hipLaunchKernelGGL(moe_wide_combine_kernel, dim3(a.tokens, (a.H + 1023) / 1024), dim3(256), 0,
                     stream, a, gates, out);
  return hipGetLastError();
}

}  // namespace moe
