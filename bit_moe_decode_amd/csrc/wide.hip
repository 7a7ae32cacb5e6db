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
//
// How 128 products are added.  The FP8 MFMA aligns each group of 8 to its
// largest product and drops what lies 13 bits below (1.3e-5 of a result, rms).
// That is nothing in y, but it moves some of mid's values across a border
// between two FP8 codes, 2^-4 of the value apart: at 16 to 48 tokens of 6144
// the outputs' error went from the 0.00166 of their bf16 rounding to 0.0018 ..
// 0.0026.  Gate and up of the 64-row tiles therefore take the codes as bf16
// numbers, which they are, through the bf16 MFMA, whose sums are fp32's: twice
// the MFMA work and the conversions, for 558.7 -> 560.7 us at 16 tokens, 1598
// -> 1611 us at 300 and 2102 -> 2182 us at 1536, where the weights' bytes set
// the time.  In the 128-row tiles the products set it (4096 tokens: 2935 us
// with FP8 MFMAs, 6076 us with bf16, its operands spilling): they keep the FP8
// MFMA, and an error of 0.0020.
#include "wide.h"

#include "device_common.h"

namespace moe {

// ------------------------------------------------------- activation blocks
// A block takes one token: 8 columns a lane, a 1x128 block in 16 lanes.  Reads
// and writes 18 KB a token of 6144: 4096 tokens 23 us (3.3 TB/s; 0.8% of the
// step), 16 tokens 4.8 us, the latency of one pass.
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
//
// Measured at 256 experts of 6144 x 2048 and a shared one.  300 tokens: up/gate
// 1012 us, down 544, the weights' 9.7 GB at 6.2 TB/s, which bounds it.  4096
// tokens: 1805 .. 1870 and 911 .. 945 us, 1.0 PFLOP/s, bound by no single unit:
// the loads of the next step are under way during one step's products, yet the
// step's phases add up (MFMAs busy 24% of the cycles, LDS 25%; without any
// loads the up/gate still takes 1115 us, without the weights' 1160, and a loop
// of loads and LDS reads without any MFMA 1690).  Tried there: loads straight
// into three LDS stages, the products of one row tile issued before the last
// one's are scaled, in blocks of 4 waves and of 8 (1740 .. 1860 us, not taken:
// 3% for a second kernel whose waits count its loads); rows of 256 in two
// stages (2100); other orders of tiles over the XCDs, tiles of even size and
// staggered K (1760 .. 1990).
__device__ __forceinline__ int lds_at(int row, int chunk) {
  return row * 128 + ((chunk ^ (row >> 1)) & 7) * 16;
}

// Loads at a 32-bit offset from a block-uniform base: the base, the uniform
// part of the offset and the bound stay in scalar registers (as 64-bit
// addresses a lane's 12 loads a step took 24 vector registers).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_base(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 load_at(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t uniform) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, uniform, 0));
}
__device__ __forceinline__ float load_f32_at(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t uniform) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, lane, uniform, 0));
}

template <int MT>
struct WideLds {
  __align__(16) uint8_t codes[(16 * MT + 256) * 128];  // weight rows, then sorted rows
  float as[16 * MT];
  float mx[4][16 * MT];
};

// The tile's products and their epilogue, U of its MT row tiles holding rows.
template <int MT, int U, bool UG>
__device__ __forceinline__ void wide_tile(const WideArgs& a, const WideWeights& w,
                                          const RowTile& tile, int nb, WideLds<MT>& sh) {
  constexpr bool kExact = UG && MT == 4;  // sums in fp32: see the top of the file
  constexpr int NA = (U + 1) / 2;  // 16-byte chunks of sorted rows a thread loads a step
  const int tid = threadIdx.x, lane = tid & 63, wn = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const bool shared = tile.group == a.E;
  const int K = UG ? a.H : a.I, N = UG ? a.I : a.H, nkb = K / 128;
  const int64_t ew = shared ? 0 : (int64_t)tile.group * N * K;
  const int64_t es = shared ? 0 : (int64_t)tile.group * (N / 128) * nkb;
  const uint8_t* w0 = (UG ? (shared ? w.sg_c : w.gate_c) : (shared ? w.sd_c : w.down_c)) + ew;
  const uint8_t* w1 = UG ? (shared ? w.su_c : w.up_c) + ew : w0;
  const float* s0 = (UG ? (shared ? w.sg_s : w.gate_s) : (shared ? w.sd_s : w.down_s)) + es;
  const float* s1 = UG ? (shared ? w.su_s : w.up_s) + es : s0;
  // weight rows of the block: half h (0, 1) starts at row n0, n1; a half past
  // the end of the down matrix repeats its last and is not stored
  const int n0 = UG ? nb * 128 : nb * 256;
  const int n1 = UG ? n0 : (n0 + 128 < N ? n0 + 128 : n0);
  const float* ps0 = s0 + (int64_t)(n0 / 128) * nkb;
  const float* ps1 = s1 + (int64_t)(n1 / 128) * nkb;

  // this thread's chunks of a step: weight rows tid / 8 + 32 i (i < 4: half 0),
  // then sorted rows (those past the tile's end repeat its last row)
  const uint32_t ow = (uint32_t)(tid >> 3) * (uint32_t)K + (uint32_t)(tid & 7) * 16u;
  const auto bw0 = uniform_base(w0 + (int64_t)n0 * K, 128u * K);
  const auto bw1 = uniform_base(w1 + (int64_t)n1 * K, 128u * K);
  const int rows = UG ? a.tokens : (tile.end - tile.row < 16 * U ? tile.end - tile.row : 16 * U);
  const auto ba = uniform_base(UG ? a.act_q : a.mid_q + (int64_t)tile.row * K, (uint32_t)rows * K);
  const auto bs = uniform_base(UG ? a.act_s : a.mid_s + (int64_t)tile.row * nkb, (uint32_t)rows * nkb * 4u);
  auto source_row = [&](int i) -> uint32_t {  // row behind ba, bs of the tile's sorted row i
    int s = tile.row + i;
    if (s >= tile.end) s = tile.end - 1;
    if (!UG) return (uint32_t)(s - tile.row);
    return (uint32_t)(s < a.picks ? a.order[s] >> 3 : s - a.picks);
  };
  uint32_t oa[NA];
#pragma unroll
  for (int i = 0; i < NA; i++)
    oa[i] = source_row((tid >> 3) + 32 * i) * (uint32_t)K + (uint32_t)(tid & 7) * 16u;
  const uint32_t os = source_row(tid) * (uint32_t)nkb * 4u;
  // an odd number of row tiles: the last 16 rows are loaded by the first two waves
  auto loads = [&](int i) { return i + 1 < NA || U % 2 == 0 || wn < 2; };

  u32x4 rw[8], ra[NA];
  float rs = 0.f;
  auto issue = [&](uint32_t kb) {
#pragma unroll
    for (int i = 0; i < 4; i++) rw[i] = load_at(bw0, ow, 32u * i * K + kb * 128u);
#pragma unroll
    for (int i = 0; i < 4; i++) rw[4 + i] = load_at(bw1, ow, 32u * i * K + kb * 128u);
#pragma unroll
    for (int i = 0; i < NA; i++)
      if (loads(i)) ra[i] = load_at(ba, oa[i], kb * 128u);
    if (64 * wn < 16 * U) rs = load_f32_at(bs, os, kb * 4u);
  };
  float acc[U][4][4];  // [sorted-row tile][weight tile: 2 of half 0, 2 of half 1][4 columns]
#pragma unroll
  for (int i = 0; i < U; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int v = 0; v < 4; v++) acc[i][j][v] = 0.f;

  // Places in LDS.  The permutation depends on a row's last 4 bits alone, so
  // that 16 rows on (and 32, for the writes) are at a constant distance.
  uint8_t* const put = sh.codes + lds_at(tid >> 3, tid & 7);
  const uint8_t* const row0 = sh.codes + lds_at(col, g);      // K 16 g .. of row col
  const uint8_t* const row1 = sh.codes + lds_at(col, g + 4);  // K 64 + 16 g ..
  auto operand = [&](int row) { return cat8(ld16(row0 + row * 128), ld16(row1 + row * 128)); };

  issue(0);
  for (int kb = 0; kb < nkb; kb++) {
    __syncthreads();  // every wave is done with the last step's codes
#pragma unroll
    for (int i = 0; i < 8; i++) *reinterpret_cast<u32x4*>(put + i * 4096) = rw[i];
#pragma unroll
    for (int i = 0; i < NA; i++)
      if (loads(i)) *reinterpret_cast<u32x4*>(put + 32768 + i * 4096) = ra[i];
    if (tid < 16 * U) sh.as[tid] = rs;
    const float sw[2] = {ps0[kb], ps1[kb]};
    if (kb + 1 < nkb) issue(kb + 1);
    __syncthreads();
    v8i op[4];
    v8bf opx[4][4];  // (kExact) as bf16: 8 codes of every lane an MFMA
#pragma unroll
    for (int j = 0; j < 4; j++) {
      op[j] = operand((j >> 1) * 128 + wn * 32 + (j & 1) * 16);
      if constexpr (kExact) {
#pragma unroll
        for (int q = 0; q < 4; q++) opx[j][q] = fp8x8_to_bf16(uint2{(uint32_t)op[j][2 * q], (uint32_t)op[j][2 * q + 1]});
      }
    }
    // the scheduling barriers keep the compiler from hoisting every row tile's
    // reads (71 spilled registers at 8 row tiles without them)
    v8i b[2];
    float as[2];
    auto fetch = [&](int i) {
      b[i & 1] = operand(256 + 16 * i);
      as[i & 1] = sh.as[i * 16 + col];
    };
    fetch(0);
#pragma unroll
    for (int i = 0; i < U; i++) {
      v4f c[4];
      if constexpr (kExact) {
#pragma unroll
        for (int j = 0; j < 4; j++) c[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const v8bf bx = fp8x8_to_bf16(uint2{(uint32_t)b[i & 1][2 * q], (uint32_t)b[i & 1][2 * q + 1]});
#pragma unroll
          for (int j = 0; j < 4; j++) c[j] = mfma_bf16(opx[j][q], bx, c[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) c[j] = mfma_fp8(op[j], b[i & 1]);
      }
      const float ar = as[i & 1];
      if (i + 1 < U) fetch(i + 1);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float s = ar * sw[j >> 1];
#pragma unroll
        for (int v = 0; v < 4; v++) acc[i][j][v] = fmaf(c[j][v], s, acc[i][j][v]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < U; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) pin4(acc[i][j]);

  if constexpr (UG) {
    // mid of columns 32 wn + 16 j + 4 g + v, j < 2, then its 1x128 block's
    // largest value over the 4 waves of the row
#pragma unroll
    for (int i = 0; i < U; i++) {
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
      if (g == 0) sh.mx[wn][i * 16 + col] = mx;
    }
    __syncthreads();
    // the codes through LDS, so that 8 lanes store a row's 128 bytes
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int m = i * 16 + col;
      const float s = fmaxf(fmaxf(sh.mx[0][m], sh.mx[1][m]), fmaxf(sh.mx[2][m], sh.mx[3][m])) / 448.0f;
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint32_t q = 0u;
        if (s > 0.f)
          q = f32x2_to_e4m3(acc[i][j][0] / s, acc[i][j][1] / s) |
              (f32x2_to_e4m3(acc[i][j][2] / s, acc[i][j][3] / s) << 16);
        *reinterpret_cast<uint32_t*>(sh.codes + m * 128 + wn * 32 + j * 16 + 4 * g) = q;
      }
      if (wn == 0 && g == 0 && tile.row + m < tile.end)
        a.mid_s[(int64_t)(tile.row + m) * (N / 128) + nb] = s;
    }
    __syncthreads();
    for (int q = tid; q < 16 * U * 8; q += 256) {
      const int row = tile.row + (q >> 3);
      if (row < tile.end)
        *reinterpret_cast<u32x4*>(a.mid_q + (int64_t)row * N + n0 + (q & 7) * 16) = ld16(sh.codes + q * 16);
    }
  } else {
    // through LDS, so that 8 lanes store 32 consecutive outputs of a row: the
    // wave's 16 rows x 64 columns of one row tile at a time, in an area of its
    // own (rows of 68 floats; one wave's LDS operations complete in order)
    __syncthreads();  // every wave is done with the last step's codes
    float* mine = reinterpret_cast<float*>(sh.codes) + wn * 16 * 68;
    const int jn = lane & 15;  // columns 4 jn ..: half jn / 8
    const int n = n0 + (jn >> 3) * 128 + wn * 32 + (jn & 7) * 4;
#pragma unroll
    for (int i = 0; i < U; i++) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = 0; j < 4; j++)
        *reinterpret_cast<v4f*>(mine + col * 68 + j * 16 + 4 * g) =
            v4f{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      asm volatile("" ::: "memory");
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = 4 * q + (lane >> 4), row = tile.row + i * 16 + m;
        const v4f v = *reinterpret_cast<const v4f*>(mine + m * 68 + 4 * jn);
        if (row < tile.end && n < N) *reinterpret_cast<v4f*>(a.y + (int64_t)row * N + n) = v;
      }
    }
  }
}

template <int MT, bool UG>
__global__ __launch_bounds__(256, 2) void moe_wide_gemm_kernel(WideArgs a, WideWeights w) {
  __shared__ WideLds<MT> sh;
  // Column blocks (UG: 128 mid columns; down: 256 outputs) first: consecutive
  // blocks go to the 8 XCDs in turn, each with an L2 of its own, and where a
  // multiple of 8 column blocks makes up a row tile, one XCD's L2 serves all
  // the row tiles of a column block, so that an expert's tiles share its weights
  const uint32_t nbs = UG ? a.I / 128 : (a.H + 255) / 256;
  const int ti = (int)(blockIdx.x / nbs), nb = (int)(blockIdx.x % nbs);
  if (ti >= *a.n_tiles) return;
  const RowTile tile = a.tiles[ti];
  int used = (tile.end - tile.row + 15) >> 4;
  used = __builtin_amdgcn_readfirstlane(used < MT ? used : MT);
  // a loop for each number of row tiles that hold rows
  if constexpr (MT == 8) {
    if (used == 8) return wide_tile<MT, 8, UG>(a, w, tile, nb, sh);
    if (used == 7) return wide_tile<MT, 7, UG>(a, w, tile, nb, sh);
    if (used == 6) return wide_tile<MT, 6, UG>(a, w, tile, nb, sh);
    if (used == 5) return wide_tile<MT, 5, UG>(a, w, tile, nb, sh);
  }
  if (used == 4) return wide_tile<MT, 4, UG>(a, w, tile, nb, sh);
  if (used == 3) return wide_tile<MT, 3, UG>(a, w, tile, nb, sh);
  if (used == 2) return wide_tile<MT, 2, UG>(a, w, tile, nb, sh);
  wide_tile<MT, 1, UG>(a, w, tile, nb, sh);
}

// out[t] = bf16( sum_j g[t,j] y[pos[t,j]] + y[picks + t] ), in pick order.
// Nine fp32 rows read for one bf16 row written, all loads under way at once:
// 4096 tokens of 6144 196 us, 4.9 TB/s, bound by memory.
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

// Rows of a tile, by the rows an expert has in the mean.  256 experts of 6144
// x 2048, whole step in 64- and 128-row tiles: 1538 and 1616 us at 9 rows, 1990
// and 1969 at 32, 2176 and 2048 at 48, 2495 and 2202 at 64.  From 32 to 48 rows
// the 64-row tiles' sums in fp32 (top of the file) are taken for up to 6% of
// the time.
int wide_tile_rows(int64_t picks, int experts) {
  const int64_t per = picks / experts;
  return per <= 48 ? 64 : 128;
}

int wide_max_tiles(int64_t picks, int experts, int shared_rows, int tile_rows) {
  return (int)(sort_max_tiles(picks, experts, tile_rows) + (shared_rows + tile_rows - 1) / tile_rows);
}

template <int MT>
static void launch_products(const WideArgs& a, const WideWeights& w, hipStream_t stream) {
  hipLaunchKernelGGL((moe_wide_gemm_kernel<MT, true>), dim3(a.max_tiles * (a.I / 128)), dim3(256), 0,
                     stream, a, w);
  hipLaunchKernelGGL((moe_wide_gemm_kernel<MT, false>), dim3(a.max_tiles * ((a.H + 255) / 256)),
                     dim3(256), 0, stream, a, w);
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
    case 64: launch_products<4>(a, w, stream); break;
    default: launch_products<8>(a, w, stream); break;
  }
  hipLaunchKernelGGL(moe_wide_combine_kernel, dim3(a.tokens, (a.H + 1023) / 1024), dim3(256), 0,
                     stream, a, gates, out);
  return hipGetLastError();
}

}  // namespace moe
