// tile_product.h -- the tile of a bf16 matrix product that products.hip and
// lm_loss.hip build on: sum_c M(m, c) J(j, c) for a block's m and j, by
// 16x16x32 bf16 MFMAs with fp32 sums.
//
// Either operand lies in memory with c contiguous in a row of each m (j), or
// transposed, with m (j) contiguous in a row of each c.
//
// A block's four waves hold the tile as 2 x 2 parts of 16 U x 16 V sums a wave.
// c runs in steps of 64 through a ring of LDS stages that loads fill directly,
// and in halves of 32 through the MFMAs: while those of one half run, the wave
// reads the next half's operands into registers, and in a step's second half,
// when all waves have read its stage, the stage's next loads go out, one load or
// LDS read between MFMAs.  At 8 x 8 a half is 64 MFMAs of 16 cycles beside 64 KB
// read from LDS and 32 KB written to it, 768 cycles of its 128 bytes a cycle: one
// wave a SIMD with 256 sums a lane keeps the LDS below the MFMAs, where 8 waves of
// half the width would read 96 KB, as long as the MFMAs take.
//
// Loads take 128 bytes of a row, a line, in all cases: the L2 serves 64 bytes in
// the time of 128 (loads to LDS alone of 256 blocks that share their rows as these
// do, 15 against 25 TB/s; with steps of 32, which took a line in two halves, two
// steps apart, the loss of 4096 rows took 2717 us, 2400 of them without the MFMAs).
//
// What bounds it at 8 x 8 and long c is the chip's power more than any one path:
// 1.3 to 1.46 PFLOP/s at a clock that falls to 1.8 GHz, as a large library product
// does (1.18 to 1.55).  Taking tiles of unequal length from queues, which evens the
// blocks' ends, took longer (y of 65536 rows 3190 us for 3070), and so did tiles of
// 256 x 128 and, two blocks a CU, 128 x 128 in dW (with its dx 4005 and 4253 us for
// 3758).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"

namespace moe {

// One operand: `own` rows (transposed: columns) of the tile that exist and `c`
// contraction entries, in rows of `pitch` bytes from base on.  Where own or c
// end the operand is 0: a load past an end reads nothing and fills its place with
// zeros.  Not transposed: c a multiple of 8, own * pitch below 2^32; transposed:
// own a multiple of 8.
struct TileOperand {
  const uint16_t* base;
  uint32_t pitch;
  int own, c;
  // (TilePipe's LONGER, transposed operands) c2 more entries behind them,
  // from another place
  const uint16_t* base2 = nullptr;
  uint32_t pitch2 = 0;
  int c2 = 0;
};

// (on a lambda: a tile of it that is called and not inlined keeps its registers in
// memory)
#define TILE_INLINE __attribute__((always_inline))

constexpr int kStepC = 64, kHalfC = 32;
// A load to LDS puts 16 bytes a lane at consecutive places, 1 KB in all, and
// reads memory a line at a time only where neighbouring lanes read ascending
// addresses: a kilobyte holds whole pieces of rows, each of another row.  The
// next one starts 1056 bytes on, so that the 16 lanes whose LDS reads go
// together find their rows in distinct banks.
constexpr int kPiecesAt = 1056;

template <int KILOS>
struct TileStage {
  __align__(16) uint8_t b[KILOS > 0 ? KILOS * kPiecesAt : 16];
};

typedef __attribute__((address_space(3))) void tile_lds_void;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s tile_lds_v4s;

// Waits for this wave's LDS operations, and until at most VM of its loads are
// under way, then for the other waves.  No memory operation moves across.
template <int VM>
__device__ __forceinline__ void tile_meet() {
  static_assert(VM < 64, "what the counter holds");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An address that is the same in all lanes, as the scalar it is (a buffer whose
// base the compiler takes for a lane's own is read lane by lane).
__device__ __forceinline__ const uint8_t* tile_scalar(const void* p) {
  const uint64_t a = (uint64_t)p;
  return reinterpret_cast<const uint8_t*>(
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32);
}

// How an operand of P tiles of 16 (own) x 64 (c) lies in a stage: 2 P kilobytes of
// 8 pieces of 128 bytes.
//
// Not transposed: a piece is 64 c of one row.  Kilobyte r holds row r of each of 8
// row tiles (P = 16: 16 + r of the second 8); with P below 8 kilobyte q holds rows
// q, q + 2 P, .. of tile i in its pieces i, i + P, ..  A lane's operand of a half
// is 16 bytes of row lane % 16: one read.
// Transposed: a piece is 64 columns of one c: kilobyte 8 b + q holds c = q + 8 p of
// the b-th 64 columns in its pieces p.  A lane's operand of a half is the 8 c of
// column lane % 16: two transposing reads of 4 (in each, lane i of 16 names 8 bytes
// of c = i / 4, columns 4 (i % 4) .., and gets the 4 c of column i).
template <int P, bool T, bool LONGER>
struct TileLoader {
  static constexpr int kKilos = 2 * P, kLoads = kKilos / 4;  // of a stage, a wave's of them
  static_assert(P == 4 || P == 8 || P == 16, "tiles of an operand");
  static constexpr uint32_t kNothing = 0xFFFFFF00u;  // an offset behind every buffer's end
  __amdgpu_buffer_rsrc_t whole;  // not transposed: the tile's rows
  const uint8_t* base;
  uint32_t pitch, at[kLoads];    // this lane's offsets in a step
  int c, kc, q0;                 // entries, this lane's first of a step, the wave's first kilobyte
  const uint8_t* base2;          // LONGER: of the entries behind them
  uint32_t pitch2, at2[LONGER ? kLoads : 1];
  int c2, steps;                 // their number, the steps before them
  int read;                      // this lane's operands in a stage

  __device__ __forceinline__ void set(const TileOperand& o, int lane, int wv) {
    pitch = (uint32_t)__builtin_amdgcn_readfirstlane((int)o.pitch);
    c = __builtin_amdgcn_readfirstlane(o.c);
    base = tile_scalar(o.base);
    q0 = wv * kLoads;
    const int col = lane & 15, g = lane >> 4, p = lane >> 3;
    if constexpr (T) {
#pragma unroll
      for (int n = 0; n < kLoads; n++) {
        const int q = q0 + n, own0 = (q >> 3) * 64 + (lane & 7) * 8;
        const uint32_t row = (uint32_t)((q & 7) + 8 * p);
        at[n] = own0 < o.own ? row * pitch + (uint32_t)own0 * 2u : kNothing;
        if constexpr (LONGER) at2[n] = own0 < o.own ? row * o.pitch2 + (uint32_t)own0 * 2u : kNothing;
      }
      kc = 0;
      if constexpr (LONGER) {
        base2 = tile_scalar(o.base2);
        pitch2 = (uint32_t)__builtin_amdgcn_readfirstlane((int)o.pitch2);
        c2 = __builtin_amdgcn_readfirstlane(o.c2);
        steps = (c + kStepC - 1) / kStepC;
      }
      read = (col >> 2) * kPiecesAt + g * 128 + (col & 3) * 8;
    } else {
      whole = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0,
                                                (uint32_t)__builtin_amdgcn_readfirstlane(o.own) * pitch, 0x00027000);
#pragma unroll
      for (int n = 0; n < kLoads; n++) {
        const int q = q0 + n;
        const int row = P >= 8 ? ((q >> 4) * 8 + p) * 16 + (q & 15) : (p % P) * 16 + q + 2 * P * (p / P);
        at[n] = (uint32_t)row * pitch + 16u * (uint32_t)(lane & 7);
      }
      kc = 8 * (lane & 7);
      read = P >= 8 ? col * kPiecesAt + 16 * g : (col % kKilos) * kPiecesAt + (col / kKilos) * P * 128 + 16 * g;
    }
  }
  // Load n of the wave's of step k; lds: where the operand starts in the stage.
  // Past the last step it reads nothing (the part of an offset that is the same
  // for all lanes is kept inside the buffer: the check of its end subtracts it).
  __device__ __forceinline__ void issue(uint8_t* lds, int k, int n) const {
    const int c0 = k * kStepC;
    tile_lds_void* to = (tile_lds_void*)(lds + (q0 + n) * kPiecesAt);
    if constexpr (T) {
      const bool two = LONGER && k >= steps;
      const int c1 = two ? c0 - steps * kStepC : c0, most = (two ? c2 : c) - c1;
      const int left = most < kStepC ? most : kStepC;
      const uint32_t p = two ? pitch2 : pitch;
      const uint8_t* from = (two ? base2 : base) + (int64_t)(left > 0 ? c1 : 0) * p;
      const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(from), 0, left > 0 ? (uint32_t)left * p : 0u,
                                                       0x00027000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, LONGER && two ? at2[LONGER ? n : 0] : at[n], 0, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(whole, to, 16, c0 + kc < c ? at[n] : kNothing,
                                               c0 < c ? (uint32_t)c0 * 2u : 0u, 0, 0);
    }
  }
  // Tile i's operand of half h.
  __device__ __forceinline__ v8bf operand(const uint8_t* lds, int i, int h) const {
    if constexpr (T) {
      const uint8_t* p = lds + read + (i >> 2) * (8 * kPiecesAt) + (i & 3) * 32 + h * 512;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_lds_v4s*)p);
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_lds_v4s*)(p + 4 * kPiecesAt));
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const v8bf*>(lds + read + (i >> 3) * (16 * kPiecesAt) + (i & 7) * 128 + h * 64);
    }
  }
};

// sums += j m by one MFMA, in place: left to the compiler, 256 sums in 256
// accumulation registers are moved between them, 600 moves for 256 MFMAs.  Its
// hazards: the operands come from LDS reads (waited for as any use is) and are
// not written again before the next step; the sums are read again by the same
// MFMA of the next step, or, where a basic block ends and the compiler may copy
// them, behind tile_settle().
__device__ __forceinline__ void mfma_bf16_into(v4f& sums, const v8bf& j, const v8bf& m) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(sums) : "v"(j), "v"(m));
}
__device__ __forceinline__ void tile_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// Holds sums in accumulation registers up to this point: a store of one row tile
// at a time takes them from there, where the compiler would move all 256 first.
template <int V>
__device__ __forceinline__ void tile_hold(v4f (&sums)[V]) {
#pragma unroll
  for (int v = 0; v < V; v++) asm volatile("" : "+a"(sums[v]));
}

// The wave of a thread, as the scalar it is: an MFMA runs whatever EXEC says,
// so a branch around one has to be a scalar branch.
__device__ __forceinline__ int tile_wave(int tid) { return __builtin_amdgcn_readfirstlane(tid >> 6); }

// One wave's sums: s[u][v] of m tile wm U + u and j tile wj V + v (wm, wj: the
// wave's bits 0 and 1); a lane holds j = 4 (lane / 16) + 0..3 of m = lane % 16.
template <int U, int V>
struct TileSums {
  v4f s[U][V];
};

// The products of tiles of 32 UMAX m at most by 32 V j, one after the other:
//   pipe.start(..) the first tile's loads
//   for each tile: pipe.run<U>(.., sums) for its sums, U = UMAX or fewer row tiles
//     a wave where the tile's m are; then pipe.start(..) the next tile, whose
//     first loads run while the sums are stored.
// All of the block's threads call them, with the same arguments.  A tile lies in
// the stages as one of UMAX does.  The ring has two stages where they are large
// (67 KB), or three.
template <int UMAX, int V, bool MT, bool JT, bool LONGER = false>
struct TilePipe {
  static constexpr int PM = 2 * UMAX, PJ = 2 * V;
  static_assert(!LONGER || (MT && JT), "of transposed operands");
  using Rows = TileLoader<PM, MT, LONGER>;
  using Columns = TileLoader<PJ, JT, LONGER>;
  static constexpr int NM = Rows::kLoads, NJ = Columns::kLoads, NL = NM + NJ;
  static constexpr int kJ = Rows::kKilos * kPiecesAt;  // where J starts in a stage
  static constexpr int kKilos = Rows::kKilos + Columns::kKilos;
  static constexpr int kStages = kKilos > 48 ? 2 : 3;
  // (one LDS object a stage: while a load to an object is under way, the compiler
  // lets reads of that object wait for all loads)
  using Stage = TileStage<kKilos>;
  using Last = TileStage<kStages == 3 ? kKilos : 0>;
  Rows m;
  Columns j;
  int halves;

#ifdef __HIP_DEVICE_COMPILE__  // (the host's pass of the compiler refuses the bodies and needs none)
  __device__ __forceinline__ void issue(uint8_t* b, int k, int n) const {
    if (n < NM)
      m.issue(b, k, n);
    else
      j.issue(b + kJ, k, n - NM);
  }
  __device__ __forceinline__ void start(const TileOperand& om, const TileOperand& oj, Stage& s0, Stage& s1, Last& s2) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tile_wave(tid);
    m.set(om, lane, wv);
    j.set(oj, lane, wv);
    // (a step of the second part of LONGER begins where one of the first ends)
    halves = LONGER && m.c2 > 0 ? 2 * m.steps + (m.c2 + kHalfC - 1) / kHalfC : (m.c + kHalfC - 1) / kHalfC;
    if (halves <= 0) return;
#pragma unroll
    for (int n = 0; n < NL; n++) issue(s0.b, 0, n);
#pragma unroll
    for (int n = 0; n < NL; n++) issue(s1.b, 1, n);
    if constexpr (kStages == 3) {
#pragma unroll
      for (int n = 0; n < NL; n++) issue(s2.b, 2, n);
    }
  }

  template <int U>
  __device__ __forceinline__ void run(Stage& s0, Stage& s1, Last& s2, TileSums<U, V>& sums) const {
    const int wv = tile_wave(threadIdx.x), wm = wv & 1, wj = wv >> 1;
    auto& acc = sums.s;
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int v = 0; v < V; v++) acc[u][v] = v4f{0.f, 0.f, 0.f, 0.f};
    if (halves <= 0) return;
    constexpr int N = U * V, NR = U + V;
    struct Operands {
      v8bf m[U], j[V];
    };
    auto read = [&](Operands& o, const uint8_t* s, int h, int n) TILE_INLINE {
      if (n < V)
        o.j[n] = j.operand(s + kJ, wj * V + n, h);
      else
        o.m[n - V] = m.operand(s, wm * U + n - V, h);
    };
    // A half's MFMAs, of the operands in `now`.  READ: beside them the half h of
    // `from` is read into `then`; LOAD: and `to` is filled with step k.
    auto half = [&](auto read_too, auto load_too, Operands& now, Operands& then, const uint8_t* from, int h, uint8_t* to,
                    int k) TILE_INLINE {
      constexpr bool READ = decltype(read_too)::value, LOAD = decltype(load_too)::value;
      constexpr int kRead = N >= 16 ? N * 3 / 4 : N;  // reads end early: the next half waits for them
      constexpr int kLoad = N >= 16 ? N / 2 : N;      // and loads have the more time to arrive
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int n = v * U + u;
#pragma unroll
          for (int q = 0; q < NR; q++)
            if (READ && q * kRead / NR == n) read(then, from, h, q);
#pragma unroll
          for (int q = 0; q < NL; q++)
            if (LOAD && q * kLoad / NL == n) issue(to, k, q);
          mfma_bf16_into(acc[u][v], now.j[v], now.m[u]);
          __builtin_amdgcn_sched_barrier(0);
        }
    };
    using yes = std::true_type;
    using no = std::false_type;
    Operands a, b;
    // step k in stage cur, the next in nx
    auto step = [&](uint8_t* cur, uint8_t* nx, int k) TILE_INLINE {
      half(yes{}, no{}, a, b, cur, 1, nullptr, 0);
      // the next step has arrived when at most the one behind it is under way, and
      // all waves have read all of this one
      tile_meet<(kStages - 2) * NL>();
      half(yes{}, yes{}, b, a, nx, 0, cur, k + kStages);
    };
    tile_meet<(kStages - 1) * NL>();
#pragma unroll
    for (int q = 0; q < NR; q++) read(a, s0.b, 0, q);
    const int steps = halves >> 1;
    int k = 0;
    for (; k + kStages <= steps; k += kStages) {
      if constexpr (kStages == 3) {
        step(s0.b, s1.b, k);
        step(s1.b, s2.b, k + 1);
        step(s2.b, s0.b, k + 2);
      } else {
        step(s0.b, s1.b, k);
        step(s1.b, s0.b, k + 1);
      }
      tile_settle();
    }
    if (k < steps) {
      step(s0.b, s1.b, k);
      tile_settle();
    }
    if constexpr (kStages == 3) {
      if (k + 1 < steps) {
        step(s1.b, s2.b, k + 1);
        tile_settle();
      }
    }
    if (halves & 1) {
      half(no{}, no{}, a, b, nullptr, 0, nullptr, 0);
      tile_settle();
    }
    tile_meet<0>();  // nothing under way into a stage, and no wave reads one
    // (a branch that the lanes do not share may not draw the last MFMAs into it)
#pragma unroll
    for (int u = 0; u < U; u++) tile_hold(acc[u]);
  }
#else
  __device__ void start(const TileOperand&, const TileOperand&, Stage&, Stage&, Last&) {}
  template <int U>
  __device__ void run(Stage&, Stage&, Last&, TileSums<U, V>&) const {}
#endif
};

// Two neighbouring j tiles' sums of one m as bf16: 16 bytes, the 8 values at
// tile_pair_at() of the pair's first column.  (The lanes of j 4 .. 7 and 0 .. 3
// trade halves, so that four lanes store 64 bytes of a row.)
__device__ __forceinline__ u32x4 tile_pair(const v4f& x, const v4f& y) {
  u32x4 o;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const uint32_t a = (uint32_t)f32_to_bf16(x[2 * h]) | ((uint32_t)f32_to_bf16(x[2 * h + 1]) << 16);
    const uint32_t b = (uint32_t)f32_to_bf16(y[2 * h]) | ((uint32_t)f32_to_bf16(y[2 * h + 1]) << 16);
    const auto t = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    o[h] = t[0];
    o[2 + h] = t[1];
  }
  return o;
}
__device__ __forceinline__ int tile_pair_at(int lane) { return 16 * ((lane >> 4) & 1) + 8 * (lane >> 5); }

// The place of tile t of m_tiles x j_tiles: four row tiles in a run, then the
// next column tile, so that the 32 blocks of an XCD share few rows and columns.
__device__ __forceinline__ void place_of(int t, int m_tiles, int j_tiles, int* mt, int* jt) {
  const int band = t / (4 * j_tiles), m0 = 4 * band;
  const int high = m_tiles - m0 < 4 ? m_tiles - m0 : 4;
  const int r = t - band * 4 * j_tiles;
  *jt = r / high;
  *mt = m0 + (r - *jt * high);
}

// Blocks go to the 8 XCDs in turn, each with an L2 of its own: of every
// gridDim.x tiles (a multiple of 8) an XCD takes neighbouring ones.
__device__ __forceinline__ int first_tile() {
  return (int)(blockIdx.x & 7) * (int)(gridDim.x >> 3) + (int)(blockIdx.x >> 3);
}

// Tiles of unequal length, taken as blocks come free: XCD x's blocks take the
// tiles of queue x one after the other, then those left in the others.  Which
// block computes a tile changes no result.  A ticket is asked for before the tile
// that runs meanwhile, and looked at behind it.
struct TileQueues {
  int32_t* next;  // [8], zeros at the start
  int empty = 0;  // queues known to be (thread 0's)
  __device__ __forceinline__ int queue() const { return (int)(blockIdx.x + empty) & 7; }
  __device__ __forceinline__ int ticket() const { return atomicAdd(next + queue(), 1); }  // thread 0
  // The tile of thread 0's ticket, for all threads; -1: none is left.  size(q):
  // tiles of queue q; tile(q, i): its i-th.
  template <typename Size, typename Tile>
  __device__ __forceinline__ int redeem(int ticket_, int* shared, Size size, Tile tile) {
    if (threadIdx.x == 0) {
      int t = -1;
      while (empty < 8) {
        if (ticket_ < size(queue())) {
          t = tile(queue(), ticket_);
          break;
        }
        if (++empty < 8) ticket_ = ticket();
      }
      *shared = t;
    }
    tile_meet<63>();
    const int t = __builtin_amdgcn_readfirstlane(*shared);
    tile_meet<63>();
    return t;
  }
};
// An eighth of n tiles, in their order.
__device__ __forceinline__ int eighth(int n, int q) { return (int)((int64_t)n * q / 8); }

// Stores a wave's sums as rows m0 + .. of out, of `cols` columns (a multiple of
// 8); rows from m_end on and columns from cols on are not there.
template <int U, int V, typename T, bool ADD>
__device__ __forceinline__ void store_tile(TileSums<U, V>& sums, T* out, int64_t m0, int64_t m_end, int j0, int cols) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tile_wave(tid);
  const int col = lane & 15, g = lane >> 4;
  auto& acc = sums.s;
  m0 += (wv & 1) * 16 * U;
  j0 += (wv >> 1) * 16 * V;
  // this wave's rows, from column j0 on
  const int64_t rows = m_end - m0;
  const uint32_t pitch = (uint32_t)cols * (uint32_t)sizeof(T);
  const uint8_t* base = tile_scalar(out + (rows > 0 ? m0 : 0) * cols);
  const auto whole = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(base), 0,
      rows > 0 ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(rows < 16 * U ? rows : 16 * U)) * pitch : 0u, 0x00027000);
  constexpr uint32_t kNothing = 0xFFFFFF00u;
#pragma unroll
  for (int u = 0; u < U; u++) {
    tile_hold(acc[u]);
    const uint32_t row = (uint32_t)(16 * u + col) * pitch;
    const bool there = 16 * u + col < rows;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int v = 0; v < V; v++) {
        const int j = j0 + 16 * v + 4 * g;
        v4f s = acc[u][v];
        if constexpr (ADD) {
          if (there && j < cols) s += *reinterpret_cast<const v4f*>(base + row + 4u * (uint32_t)j);
        }
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, s), whole,
                                               j < cols ? row + 4u * (uint32_t)j : kNothing, 0, 0);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        if constexpr (ADD) {  // in place of the sums: a lane's own 4 columns
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const int j = j0 + 16 * (v + h) + 4 * g;
            if (there && j < cols) {
              const uint2 o = *reinterpret_cast<const uint2*>(base + row + 2u * (uint32_t)j);
              acc[u][v + h] += v4f{__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u),
                                   __uint_as_float(o.y << 16), __uint_as_float(o.y & 0xFFFF0000u)};
            }
          }
        }
        const u32x4 o = tile_pair(acc[u][v], acc[u][v + 1]);
        const int j = j0 + 16 * v + tile_pair_at(lane);
        __builtin_amdgcn_raw_buffer_store_b128(o, whole, j < cols ? row + 2u * (uint32_t)j : kNothing, 0, 0);
      }
    }
  }
}

// Blocks of a launch over `tiles` tiles: `a_cu` for each CU of the current device
// at most, a multiple of 8.
inline hipError_t tile_blocks(int64_t tiles, int a_cu, int* blocks) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  const int64_t most = (int64_t)(cus / 8 > 0 ? cus / 8 : 1) * 8 * a_cu;
  const int64_t want = (tiles + 7) / 8 * 8;
  *blocks = (int)(want < most ? want : most);
  return hipSuccess;
}

}  // namespace moe
