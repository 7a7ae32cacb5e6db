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
// between two FP8 codes, 2^-4 of the value apart: the outputs' error against
// the definition is 0.00166 of their size where all sums are fp32's, which is
// their bf16 rounding, and 0.0020 where gate and up take the FP8 MFMA, with
// single tokens at 0.014.  The bf16 MFMA, which takes the codes as the bf16
// numbers they are, sums in fp32, at twice the time a product and with 192
// conversions a step of 128 rows.  While the weights' bytes set the time that
// costs little: of 256 experts and a shared one of 6144 x 2048, with the routed
// experts in fp32 and by the FP8 MFMA, 545 and 542 us at 16 tokens, 1560 and
// 1557 at 300, 1705 and 1700 at 512, 1842 and 1810 at 768, 1969 and 1909 at 1024,
// 2545 and 2201 at 2048, 3954 and 2915 at 4096; of 240 experts of 6144 x 256 362
// and 339 at 700.  So up to kWideExactRows picks an expert (512 tokens of 256
// experts) all products are summed in fp32.  Above, the shared expert's gate and
// up still are, its weight being 1 (the error at 4096 tokens 0.0020 -> 0.0017, the
// step 2850 -> 2915 us), and the rest is the FP8 MFMA's.
#include "wide.h"

#include <type_traits>

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
    float u[8];
    uint32_t m = 0u;  // largest |u| by its bits: a NaN is the largest, and stays one
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float xf = __uint_as_float(i & 1 ? xv[i >> 1] & 0xFFFF0000u : xv[i >> 1] << 16);
      const float gf = __uint_as_float(i & 1 ? gv[i >> 1] & 0xFFFF0000u : gv[i >> 1] << 16);
      ss = fmaf(xf, xf, ss);
      u[i] = bf16_to_f32(f32_to_bf16(xf * gf));
      m = max(m, __float_as_uint(fabsf(u[i])));
    }
    const float s = __uint_as_float(row16_umax(m)) / 448.0f;
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

// The tokens' scales once more, by K block and sorted row: a step of a tile
// reads 512 bytes in a row instead of 4 from each of 128 places, each of which
// costs a request as a line of codes does (4096 tokens: 110 us of the up/gate
// for the 7 that this takes).
__global__ __launch_bounds__(256) void moe_wide_sorted_scales_kernel(WideArgs a) {
  const int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x;
  // (sorted rows behind the last pick of a group: none)
  if (s >= a.rows || (s < a.picks && s >= a.offsets[a.E])) return;
  const int64_t t = s < a.picks ? a.order[s] >> 3 : s - a.picks;
  const int nkb = a.H / 128, k0 = blockIdx.y * 4;
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; k++) v[k] = a.act_s[t * nkb + (k0 + k < nkb ? k0 + k : nkb - 1)];
#pragma unroll
  for (int k = 0; k < 4; k++)
    if (k0 + k < nkb) a.act_t[(int64_t)(k0 + k) * a.rows + s] = v[k];
}

// ------------------------------------------------------------ the products
// A block computes up to 128 sorted rows of one expert against 256 weight rows
// (the gate and up rows of 128 mid columns, or 256 down rows), K in steps of
// 128; one block holds a CU.  The weights are the MFMA's A operand (their 16
// rows its output rows: a lane holds 4 consecutive columns of one sorted row),
// the sorted rows its B operand; each of the 4 waves takes 64 weight rows and
// all the sorted ones.  The fp32 products of a step are scaled by weight scale
// times row scale and added.
//
// Codes are loaded straight into LDS, into a ring of three stages, and each
// operand is replaced by the next one right after its last use, so that a
// wave's loads, LDS reads, MFMAs and scaling run beside each other: the products
// of one row tile are issued before the last one's are scaled, and the ring's
// next loads are spread between the MFMAs (in one go they stall the wave that
// issues them: up/gate of 4096 tokens 1790 against 1740 us).
//
// Measured at 256 experts of 6144 x 2048 and a shared one.  300 tokens: up/gate
// 950 us, down 524: the bytes of the weights in use (5.8 and 2.9 GB, counted as
// 5.87 and 2.92) at 6.2 and 5.6 TB/s, which bounds it.  4096 tokens: up/gate 1726
// us, down 938, 1.1 PFLOP/s; the matrix units of the up/gate are busy for 28% of
// the time.  Before the shared expert's fp32 sums it took 1630 .. 1680; then
// without any loads 955, with half the weights' 1352, and a loop of the loads
// and LDS reads without any MFMA 1690: bound by the loads, 16.1 GB a launch from
// L2 to the CUs, 8.8 of them from memory.  A form with the next step in
// registers and two blocks a CU took 1830 and 920 us, and 4 to 10% more time
// from 16 tokens on; other orders of tiles over the XCDs, tiles of even size and
// K started at other places were no faster (1760 .. 1890 where this order took
// 1760), nor were row scales read from 128 places a step (1740 for 1630).

// Loads at a 32-bit offset from a block-uniform base: the base, the uniform
// part of the offset and the bound stay in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_base(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}

// A block's weights and columns: half h (0, 1) of its 256 weight rows starts at
// row n0, n1 of w0, w1, with scales from s0, s1 on; a half past the end of the
// down matrix repeats its last and is not stored.
struct WideBlock {
  const uint8_t *w0, *w1;
  const float *s0, *s1;
  int K, N, nkb, n0;
};
template <bool UG>
__device__ __forceinline__ WideBlock wide_block(const WideArgs& a, const WideWeights& w,
                                                const RowTile& tile, int nb) {
  const bool shared = tile.group == a.E;
  WideBlock o;
  o.K = UG ? a.H : a.I;
  o.N = UG ? a.I : a.H;
  o.nkb = o.K / 128;
  const int64_t ew = shared ? 0 : (int64_t)tile.group * o.N * o.K;
  const int64_t es = shared ? 0 : (int64_t)tile.group * (o.N / 128) * o.nkb;
  o.w0 = (UG ? (shared ? w.sg_c : w.gate_c) : (shared ? w.sd_c : w.down_c)) + ew;
  o.w1 = UG ? (shared ? w.su_c : w.up_c) + ew : o.w0;
  o.s0 = (UG ? (shared ? w.sg_s : w.gate_s) : (shared ? w.sd_s : w.down_s)) + es;
  o.s1 = UG ? (shared ? w.su_s : w.up_s) + es : o.s0;
  o.n0 = UG ? nb * 128 : nb * 256;
  const int n1 = UG ? o.n0 : (o.n0 + 128 < o.N ? o.n0 + 128 : o.n0);
  o.w0 += (int64_t)o.n0 * o.K;
  o.w1 += (int64_t)n1 * o.K;
  o.s0 += (int64_t)(o.n0 / 128) * o.nkb;
  o.s1 += (int64_t)(n1 / 128) * o.nkb;
  return o;
}

// The row behind act_q (UG: a token) or behind the tile's first of mid_q that
// is the tile's sorted row i; rows past the tile's end repeat its last.
template <bool UG>
__device__ __forceinline__ uint32_t source_row(const WideArgs& a, const RowTile& tile, int i) {
  int s = tile.row + i;
  if (s >= tile.end) s = tile.end - 1;
  if (!UG) return (uint32_t)(s - tile.row);
  return (uint32_t)(s < a.picks ? a.order[s] >> 3 : s - a.picks);
}

// Stores a tile's sums.  codes: 17408 bytes of the block's LDS, mx: 4 words a
// row, which no wave uses any more.
template <int U, bool UG>
__device__ __forceinline__ void wide_store(const WideArgs& a, const RowTile& tile, int nb,
                                           const WideBlock& bl, float (&acc)[U][4][4],
                                           uint8_t* codes, uint32_t* mx) {
  const int tid = threadIdx.x, lane = tid & 63, wn = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int N = bl.N, n0 = bl.n0;
#pragma unroll
  for (int i = 0; i < U; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) pin4(acc[i][j]);

  if constexpr (UG) {
    // mid of columns 32 wn + 16 j + 4 g + v, j < 2, then its 1x128 block's
    // largest value over the 4 waves of the row
#pragma unroll
    for (int i = 0; i < U; i++) {
      uint32_t big = 0u;  // by its bits, as for the activations
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int v = 0; v < 4; v++) {
          const float gt = acc[i][j][v];
          const float mid = gt / (1.0f + __expf(-gt)) * acc[i][j + 2][v];
          acc[i][j][v] = mid;
          big = max(big, __float_as_uint(fabsf(mid)));
        }
      big = max(big, (uint32_t)__shfl_xor((int)big, 16, kWave));
      big = max(big, (uint32_t)__shfl_xor((int)big, 32, kWave));
      if (g == 0) mx[wn * 16 * U + i * 16 + col] = big;
    }
    __syncthreads();
    // the codes through LDS, so that 8 lanes store a row's 128 bytes
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int m = i * 16 + col;
      const float s = __uint_as_float(max(max(mx[m], mx[16 * U + m]), max(mx[32 * U + m], mx[48 * U + m]))) / 448.0f;
      if (s < 0x1p-126f) {  // a rounded subnormal: values up to 1.5 * 448 of them
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
          for (int v = 0; v < 4; v++) acc[i][j][v] = fminf(fmaxf(acc[i][j][v], -448.f * s), 448.f * s);
      }
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint32_t q = 0u;
        if (s > 0.f)
          q = f32x2_to_e4m3(acc[i][j][0] / s, acc[i][j][1] / s) |
              (f32x2_to_e4m3(acc[i][j][2] / s, acc[i][j][3] / s) << 16);
        *reinterpret_cast<uint32_t*>(codes + m * 128 + wn * 32 + j * 16 + 4 * g) = q;
      }
      if (wn == 0 && g == 0 && tile.row + m < tile.end)
        a.mid_s[(int64_t)nb * a.rows + tile.row + m] = s;
    }
    __syncthreads();
    for (int q = tid; q < 16 * U * 8; q += 256) {
      const int row = tile.row + (q >> 3);
      if (row < tile.end)
        *reinterpret_cast<u32x4*>(a.mid_q + (int64_t)row * N + n0 + (q & 7) * 16) = ld16(codes + q * 16);
    }
  } else {
    // through LDS, so that 8 lanes store 32 consecutive outputs of a row: the
    // wave's 16 rows x 64 columns of one row tile at a time, in an area of its
    // own (rows of 68 floats; one wave's LDS operations complete in order)
    float* mine = reinterpret_cast<float*>(codes) + wn * 16 * 68;
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

// A block's tile, column block, and number of row tiles that hold rows; false:
// none.  All of it in scalars: an MFMA runs whatever EXEC says, so that the
// branches that lead to one have to be scalar.
//
// The shared expert's tiles, the last of the list, are taken first: nearly all
// of them are full, and would outlast the others (90 tokens of 32 experts of
// 1024 x 1024: 73 -> 60 us).  Column blocks (UG: 128 mid columns; down: 256
// outputs) before tiles: consecutive blocks go to the 8 XCDs in turn, each with
// an L2 of its own, and where a multiple of 8 column blocks makes up a row tile,
// one XCD's L2 serves all the row tiles of a column block, so that an expert's
// tiles share its weights.
template <bool UG, bool EXACT>
__device__ __forceinline__ bool wide_place(const WideArgs& a, RowTile* tile, int* nb, int* used) {
  const uint32_t nbs = UG ? a.I / 128 : (a.H + 255) / 256;
  const int shared = a.shared ? (a.tokens + kWideExactTile - 1) / kWideExactTile : 0;
  const int ti = (int)(blockIdx.x / nbs), end = __builtin_amdgcn_readfirstlane(*a.n_tiles);
  if (ti >= end) return false;
  *nb = (int)(blockIdx.x % nbs);
  const RowTile t = a.tiles[ti < shared ? end - shared + ti : ti - shared];
  *tile = RowTile{__builtin_amdgcn_readfirstlane(t.group), __builtin_amdgcn_readfirstlane(t.row),
                  __builtin_amdgcn_readfirstlane(t.end)};
  const int most = (EXACT || tile->group == a.E ? kWideExactTile : kWideTile) / 16;
  const int rows = (tile->end - tile->row + 15) >> 4;
  *used = rows < most ? rows : most;
  return true;
}

// A load to LDS puts 16 bytes a lane at consecutive places, 1 KB in all, and
// reads memory a line at a time only where neighbouring lanes read ascending
// addresses.  So a kilobyte holds 8 pieces of 128 bytes, each of another row,
// and starts 1056 bytes behind the one before.  The LDS reads lanes 0-3, 12-15
// and 20-27 of a wave together (and so on): the chunks that these take, of rows
// in 8 kilobytes in turn, or in 4 kilobytes and neighbouring pieces, lie in
// distinct banks (1040 bytes apart, two and two shared one: up/gate 1817 against
// 1774 us).
constexpr int kKilo = 1056;

// A wave's own 64 weight rows: kilobyte 8 wn + 4 h + q holds rows 32 wn + 16 j +
// 4 p + q of half h, its piece 4 j + p.
struct RingWeights {
  __align__(16) uint8_t b[32 * kKilo];
};
// Sorted rows: kilobyte i holds row i of each row tile.  Behind them their
// scales, and a place for loads of nothing.
struct RingRows {
  static constexpr int kScales = 16 * kKilo, kNone = kScales + 512;
  __align__(16) uint8_t b[kNone + 256];
};
// (one LDS object for each: while a load to an object is under way, the
// compiler lets reads of that object wait for all loads)
struct RingStage {
  RingWeights& w;
  RingRows& r;
};

typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t lane,
                                            uint32_t uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, lane, uniform, 0, 0);
}
__device__ __forceinline__ void load_f32_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t lane,
                                                uint32_t uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, lane, uniform, 0, 0);
}

// Waits for this wave's LDS operations, and until at most VM of its loads are
// under way.  No memory operation moves across.
template <int VM>
__device__ __forceinline__ void wait_own() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
  asm volatile("" ::: "memory");
}
// The same, then for the other waves.
template <int VM>
__device__ __forceinline__ void wait_and_meet() {
  wait_own<VM>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int U, bool UG, bool kExact>
__device__ __forceinline__ void wide_tile(const WideArgs& a, const WideWeights& w, const RowTile& tile,
                                          int nb, const RingStage& st0, const RingStage& st1,
                                          const RingStage& st2) {
  // a wave's loads of a step: 8 of weights, then 4 of sorted rows and 1 of their
  // scales.  A wave (or lane) without any loads from past the buffer's end,
  // which touches no memory: every step of every wave has as many loads.
  constexpr int NW = 8, NR = 5, ND = NW + NR;
  constexpr uint32_t kNothing = 0xFFFFFF00u;
  const int tid = threadIdx.x, lane = tid & 63, wn = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const WideBlock bl = wide_block<UG>(a, w, tile, nb);
  const int K = bl.K, nkb = bl.nkb;
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  const scalar_ptr ps0 = (scalar_ptr)bl.s0, ps1 = (scalar_ptr)bl.s1;  // scalar loads
  const int left = tile.end - tile.row < 16 * U ? tile.end - tile.row : 16 * U;
  const auto bw0 = uniform_base(bl.w0, 128u * K);
  const auto bw1 = uniform_base(bl.w1, 128u * K);
  const auto ba = uniform_base(UG ? a.act_q : a.mid_q + (int64_t)tile.row * K, (uint32_t)(UG ? a.tokens : left) * K);
  const uint32_t sb = 4u * (uint32_t)a.rows;  // bytes from one K block's scales to the next
  const auto bs = uniform_base((UG ? a.act_t : a.mid_s) + tile.row, (uint32_t)(nkb - 1) * sb + 4u * (uint32_t)left);
  const uint32_t ow = (uint32_t)(32 * wn + 16 * (lane >> 5) + 4 * ((lane >> 3) & 3)) * (uint32_t)K + 16u * (lane & 7);
  uint32_t oa[4];
#pragma unroll
  for (int n = 0; n < 4; n++)
    oa[n] = (lane >> 3) < U ? source_row<UG>(a, tile, 4 * wn + n + 16 * (lane >> 3)) * (uint32_t)K + 16u * (uint32_t)(lane & 7)
                            : kNothing;
  const int srow = 64 * wn + lane;  // whose scale this lane loads
  const uint32_t os = srow < 16 * U ? 4u * (uint32_t)(srow < left ? srow : left - 1) : kNothing;
  const int ls = wn < 2 ? RingRows::kScales + wn * 256 : RingRows::kNone;
  // load n of step kb; wq, rq, sq: where the wave's parts of a stage start
  auto issue = [&](const RingStage& st, int kb, int n, int wq, int rq, int sq) {
    const uint32_t k0 = (uint32_t)kb * 128u;
    if (n < NW)
      load_to_lds(n < 4 ? bw0 : bw1, st.w.b + wq + n * kKilo, ow, k0 + (uint32_t)(n & 3) * K);
    else if (n < NW + 4)
      load_to_lds(ba, st.r.b + rq + (n - NW) * kKilo, oa[n - NW], k0);
    else
      load_f32_to_lds(bs, st.r.b + sq, os, (uint32_t)kb * sb);
  };
  const int wq0 = 8 * wn * kKilo, rq0 = 4 * wn * kKilo;

  // operands: chunks g and g + 4 of weight row 16 j + col, of sorted row 16 i + col
  const int ow0 = (8 * wn + (col & 3)) * kKilo + (col >> 2) * 128 + 16 * g, oa0 = col * kKilo + 16 * g;
  auto half_weights = [&](const RingStage& st, int wo, int j, int h) {
    return ld16(st.w.b + (j >> 1) * (4 * kKilo) + (j & 1) * 512 + wo + 64 * h);
  };
  auto weights = [&](const RingStage& st, int wo, int j) {
    return cat8(half_weights(st, wo, j, 0), half_weights(st, wo, j, 1));
  };
  auto rows_of = [&](const RingStage& st, int ro, int i) {
    const uint8_t* p = st.r.b + i * 128 + ro;
    return cat8(ld16(p), ld16(p + 64));
  };
  auto scale_of = [&](const RingStage& st, int so, int i) {
    return *reinterpret_cast<const float*>(st.r.b + RingRows::kScales + i * 64 + so);
  };

  // Row tile i of a step uses slot (first + i) % 3 of b and as; the one D tiles
  // on is read meanwhile.  At row tile M the wave meets the others: they have
  // then read all of this step's rows, whose stage may be loaded again, and the
  // next step's have arrived, from which the reads go on.
  constexpr int D = U > 1 ? 2 : 1, M = U > 2 ? U - 2 : 0;
  // The wave's own weights of this step are in registers from its first row
  // tile on: with 4 row tiles or more their place is loaded again from the
  // second on, before the meeting.
  constexpr bool kAhead = U >= 4;
  // kExact: sums in fp32 by the bf16 MFMA (top of the file).  Two vector
  // operations run beside one of these MFMAs for nothing (18 cycles for 17), each
  // more takes 6 cycles, so the scaling and the codes' conversion are spread
  // over them.  A row tile's 16 MFMAs are 4, one a weight tile, for each of 4
  // pieces of K (8 codes of every lane); a piece's bf16 values are replaced
  // once used, the rows' by the next row tile's, the weights' from the last row
  // tile on by the next step's (1623 -> 1558 us at 300 tokens against converting
  // before a row tile's MFMAs).  One row tile: each piece just before its MFMAs.
  constexpr bool kSpread = kExact && U > 1;
  v8i op[4], b[3];
  u32x4 raw[2][4];             // (kExact) the next weights' codes: pieces 2 h, 2 h + 1 of tile j
  u32x4 opx[4][4], bx[4];      // (kExact) weights and a row tile as bf16, by piece
  auto weights_pair = [&](int f) {  // pair f % 4 of piece f / 16 of weight tile f / 4 % 4
    const int p = f >> 4, j = (f >> 2) & 3, r = f & 3;
    opx[j][p][r] = fp8x2_to_bf16(raw[p >> 1][j][2 * (p & 1) + (r >> 1)], r & 1);
  };
  auto rows_pair = [&](const v8i& o, int p, int r) {
    bx[p][r] = fp8x2_to_bf16((uint32_t)o[2 * p + (r >> 1)], r & 1);
  };
  float as[3] = {0.f, 0.f, 0.f}, sw[2], sw_last[2] = {0.f, 0.f};
  v4f c[4] = {};  // the products not yet scaled: of the row tile before
  float acc[U][4][4];
#pragma unroll
  for (int i = 0; i < U; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int v = 0; v < 4; v++) acc[i][j][v] = 0.f;
  auto at = [&](int k) { return k < nkb ? k : nkb - 1; };  // (loads past the last step repeat it)
  auto step = [&](auto first, const RingStage& cur, const RingStage& nx, int k) {
    constexpr int P = decltype(first)::value;
    const int kl = at(k + 3);
    float sw_next[2];
    // (opaque, or the addresses in all three stages are kept in registers)
    int wq = wq0, rq = rq0, sq = ls, wo = ow0, ro = oa0, so = 4 * col;
    asm volatile("" : "+s"(wq), "+s"(rq), "+s"(sq), "+v"(wo), "+v"(ro), "+v"(so));
#pragma unroll
    for (int i = 0; i < U; i++) {
      const float ap = as[(P + i + 2) % 3];
      const float s[2] = {ap * (i ? sw[0] : sw_last[0]), ap * (i ? sw[1] : sw_last[1])};
      if (kAhead && i == 1) wait_own<63>();  // the operands read from cur's weights are here
      if (i == M) {
        // step k + 1 has arrived when at most these are under way: all of step
        // k + 2, and the weights of k + 3 where they have been issued
        wait_and_meet<kAhead ? ND + NW : ND>();
        sw_next[0] = ps0[at(k + 1)];
        sw_next[1] = ps1[at(k + 1)];
      }
      b[(P + i + D) % 3] = i + D < U ? rows_of(cur, ro, i + D) : rows_of(nx, ro, i + D - U);
      as[(P + i + D) % 3] = i + D < U ? scale_of(cur, so, i + D) : scale_of(nx, so, i + D - U);
      const int t = i ? i - 1 : U - 1;
      auto scale = [&](int j) {  // the products of the row tile before
#pragma unroll
        for (int v = 0; v < 4; v++) acc[t][j][v] = fmaf(c[j][v], s[j >> 1], acc[t][j][v]);
      };
      v4f d[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if constexpr (kExact) {
          if constexpr (!kSpread) {
#pragma unroll
            for (int f = 0; f < 16; f++) weights_pair(16 * j + f);
#pragma unroll
            for (int f = 0; f < 4; f++) rows_pair(b[P % 3], j, f);
          }
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const int n = 4 * j + q;
            d[q] = mfma_bf16(__builtin_bit_cast(v8bf, opx[q][j]), __builtin_bit_cast(v8bf, bx[j]),
                             j ? d[q] : v4f{0.f, 0.f, 0.f, 0.f});
            acc[t][j][q] = fmaf(c[j][q], s[j >> 1], acc[t][j][q]);
            if (i == U - 1 && j == (kSpread ? 0 : 1)) raw[0][q] = half_weights(nx, wo, q, 0);
            if (i == U - 1 && j == 3) raw[1][q] = half_weights(nx, wo, q, 1);
            if constexpr (kSpread) {
              rows_pair(b[(P + i + (j > 0)) % 3], (j + 3) & 3, q);  // of the next row tile, once used
#pragma unroll
              for (int e = 0; e < 3; e++) {
                const int f = 3 * n + e;
                if (i == U - 1 && f >= 12 && f < 44) weights_pair(f - 12);
                if (i == 0 && f < 32) weights_pair(32 + f);
              }
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
          scale(j);
          c[j] = mfma_fp8(op[j], b[(P + i) % 3]);
          if (i == U - 1) op[j] = weights(nx, wo, j);
        }
        // step k + 3's loads, evenly over the MFMAs that they may follow
        if constexpr (kAhead) {
          constexpr int QW = 4 * (M - 1), QR = 4 * (U - M);
          const int qw = (i - 1) * 4 + j, qr = (i - M) * 4 + j;
          if (qw >= 0 && qw < QW) {
#pragma unroll
            for (int n = NW * qw / QW; n < NW * (qw + 1) / QW; n++) issue(cur, kl, n, wq, rq, sq);
          }
          if (qr >= 0) {
#pragma unroll
            for (int n = NW + NR * qr / QR; n < NW + NR * (qr + 1) / QR; n++) issue(cur, kl, n, wq, rq, sq);
          }
        } else {
          constexpr int Q = 4 * (U - M);
          const int q = (i - M) * 4 + j;
          if (q >= 0) {
#pragma unroll
            for (int n = ND * q / Q; n < ND * (q + 1) / Q; n++) issue(cur, kl, n, wq, rq, sq);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (kExact) {
#pragma unroll
        for (int q = 0; q < 4; q++) c[q] = d[q];
      }
    }
    sw_last[0] = sw[0];
    sw_last[1] = sw[1];
    sw[0] = sw_next[0];
    sw[1] = sw_next[1];
  };
#pragma unroll
  for (int n = 0; n < ND; n++) issue(st0, at(0), n, wq0, rq0, ls);
#pragma unroll
  for (int n = 0; n < ND; n++) issue(st1, at(1), n, wq0, rq0, ls);
#pragma unroll
  for (int n = 0; n < ND; n++) issue(st2, at(2), n, wq0, rq0, ls);
  sw[0] = ps0[0];
  sw[1] = ps1[0];
  wait_and_meet<2 * ND>();  // step 0 has arrived
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (kExact) {
      raw[0][j] = half_weights(st0, ow0, j, 0);
      raw[1][j] = half_weights(st0, ow0, j, 1);
    } else {
      op[j] = weights(st0, ow0, j);
    }
  }
#pragma unroll
  for (int i = 0; i < D; i++) {
    b[i] = rows_of(st0, oa0, i);
    as[i] = scale_of(st0, 4 * col, i);
  }
  if constexpr (kSpread) {  // what a step finds of the one before: see there
#pragma unroll
    for (int f = 0; f < 32; f++) weights_pair(f);
#pragma unroll
    for (int f = 0; f < 12; f++) rows_pair(b[0], f >> 2, f & 3);
  }
  using p0 = std::integral_constant<int, 0>;
  using p1 = std::integral_constant<int, U % 3>;
  using p2 = std::integral_constant<int, 2 * U % 3>;
  int k = 0, next = 0;  // next: the slot of the row tile behind the last
  for (; k + 3 <= nkb; k += 3) {
    step(p0{}, st0, st1, k);
    step(p1{}, st1, st2, k + 1);
    step(p2{}, st2, st0, k + 2);
  }
  if (k < nkb) {
    step(p0{}, st0, st1, k);
    next = p1::value;
  }
  if (k + 1 < nkb) {
    step(p1{}, st1, st2, k + 1);
    next = p2::value;
  }
  const float ap = next == 0 ? as[2] : next == 1 ? as[0] : as[1];
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int v = 0; v < 4; v++) acc[U - 1][j][v] = fmaf(c[j][v], ap * sw_last[j >> 1], acc[U - 1][j][v]);
  wait_and_meet<0>();  // nothing under way into the LDS that the epilogue uses
  wide_store<U, UG>(a, tile, nb, bl, acc, st0.w.b, reinterpret_cast<uint32_t*>(st1.w.b));
}

// (256 threads a block; the bound of 512 keeps the compiler at 256 registers a
// thread.  With more it leaves the MFMAs' results in accumulation registers and
// moves each one before it is scaled: 1857 against 1818 us up/gate by the FP8
// MFMA.  The bf16 operands leave room for tiles of up to 80 rows; 96 spill
// registers beside the FP8 form, 16384 tokens 8765 against 8664 us.)
// EXACT: everything summed in fp32, else the shared expert's gate and up.
template <bool UG, bool EXACT>
__global__ __launch_bounds__(512) void moe_wide_gemm_kernel(WideArgs a, WideWeights w) {
  __shared__ RingWeights w0, w1, w2;
  __shared__ RingRows r0, r1, r2;
  RowTile tile;
  int nb, used;
  if (!wide_place<UG, EXACT>(a, &tile, &nb, &used)) return;
  const RingStage s0{w0, r0}, s1{w1, r1}, s2{w2, r2};
  if (EXACT || (UG && tile.group == a.E)) {
    if (used >= 5) return wide_tile<5, UG, true>(a, w, tile, nb, s0, s1, s2);
    if (used == 4) return wide_tile<4, UG, true>(a, w, tile, nb, s0, s1, s2);
    if (used == 3) return wide_tile<3, UG, true>(a, w, tile, nb, s0, s1, s2);
    if (used == 2) return wide_tile<2, UG, true>(a, w, tile, nb, s0, s1, s2);
    return wide_tile<1, UG, true>(a, w, tile, nb, s0, s1, s2);
  }
  if constexpr (!EXACT) {
    if (used >= 8) return wide_tile<8, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 7) return wide_tile<7, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 6) return wide_tile<6, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 5) return wide_tile<5, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 4) return wide_tile<4, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 3) return wide_tile<3, UG, false>(a, w, tile, nb, s0, s1, s2);
    if (used == 2) return wide_tile<2, UG, false>(a, w, tile, nb, s0, s1, s2);
    wide_tile<1, UG, false>(a, w, tile, nb, s0, s1, s2);
  }
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

// Picks an expert up to which a batch's products are all summed in fp32 (top of
// the file).
constexpr int kWideExactRows = 16;

static bool wide_exact(int64_t picks, int experts) {
  return picks <= (int64_t)kWideExactRows * experts;
}

int wide_max_tiles(int64_t picks, int experts, int shared_rows) {
  const int rows = wide_exact(picks, experts) ? kWideExactTile : kWideTile;
  return (int)(sort_max_tiles(picks, experts, rows) + (shared_rows + kWideExactTile - 1) / kWideExactTile);
}

hipError_t launch_wide(const WideArgs& a, const WideWeights& w, const uint16_t* x,
                       const int32_t* ids, const float* gates, uint16_t* out, hipStream_t stream) {
  const bool exact = wide_exact(a.picks, a.E);
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
  s.tile_rows = exact ? kWideExactTile : kWideTile;
  s.extra_rows = kWideExactTile;
  s.extra = a.shared ? a.tokens : 0;
  hipError_t e = launch_sort(s, stream);
  if (e != hipSuccess) return e;
  const dim3 gu(a.max_tiles * (a.I / 128)), gd(a.max_tiles * ((a.H + 255) / 256));
  hipLaunchKernelGGL(moe_wide_sorted_scales_kernel,
                     dim3((uint32_t)((a.rows + 255) / 256), (a.H / 128 + 3) / 4), dim3(256), 0, stream, a);
  if (exact) {
    hipLaunchKernelGGL((moe_wide_gemm_kernel<true, true>), gu, dim3(256), 0, stream, a, w);
    hipLaunchKernelGGL((moe_wide_gemm_kernel<false, true>), gd, dim3(256), 0, stream, a, w);
  } else {
    hipLaunchKernelGGL((moe_wide_gemm_kernel<true, false>), gu, dim3(256), 0, stream, a, w);
    hipLaunchKernelGGL((moe_wide_gemm_kernel<false, false>), gd, dim3(256), 0, stream, a, w);
  }
  hipLaunchKernelGGL(moe_wide_combine_kernel, dim3(a.tokens, (a.H + 1023) / 1024), dim3(256), 0,
                     stream, a, gates, out);
  return hipGetLastError();
}

}  // namespace moe
