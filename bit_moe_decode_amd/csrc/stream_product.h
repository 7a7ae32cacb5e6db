// stream_product.h -- the tile of a bf16 matrix product with few rows, for
// products.hip and lm_loss.hip: sum_c M(m, c) J(j, c) for up to 64 m and 64 j,
// both with c contiguous, by 16x16x32 bf16 MFMAs with fp32 sums.
//
// With few rows the time is that of J's bytes, the weights', which are read once:
// what counts is how many of them are under way, and that a request is a whole
// line (halves of lines read at 5.1 TB/s where lines do at 6.0).  A block's four
// waves take steps of 64 c in turn, lines of 8 rows a load into registers, several
// steps ahead, without meetings: 8 KB a wave and step.  A step then goes through
// an LDS area of the wave's own into the order of the MFMA's operands.  The waves'
// sums are added in wave order at the end.
//
// 16 tokens x 8 of 256 experts [4096, 6144], one draw of the picks 633 us (several
// 630 .. 720, by the 72 .. 84 experts that they use), in halves of lines 738, with
// loads that the caches are told not to keep, which fetch a line twice, 850, in
// tiles that share LDS 760 .. 930.  The loss of 8 rows of 151936 x 2560 134 us, 5.8
// TB/s, where loads alone take 128.  Two steps under way a wave: 4 as good there
// (633 us), 161 against 153 us in the loss.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "tile_product.h"

namespace moe {

constexpr int kStreamU = 4, kStreamV = 4;          // tiles of 16 m at most, of 16 j
constexpr int kStreamM = 16 * kStreamU, kStreamJ = 16 * kStreamV;

// The products of tiles of 16 U m: start() a tile's first loads; run() it; start()
// the next, whose loads run while add() joins the waves' sums.
template <int U>
struct StreamPipe {
  static constexpr int V = kStreamV;
  static constexpr int kDepth = 2;  // steps under way, of a wave
  // bytes of LDS: the waves' operand tiles, and the sums that add() takes
  static constexpr int kWave = (U + V) * kTileBytes, kLds = 4 * kWave > 4096 * U * V ? 4 * kWave : 4096 * U * V;
  static constexpr uint32_t kNothing = 0xFFFFFF00u;
  struct Step {
    u32x4 m[U][2], j[V][2];
  };
  // 32 bytes of a row: 16 c, 8 in each of two MFMAs
  struct Operand {
    v8i both;
    __device__ __forceinline__ v8bf half(int h) const {
      return __builtin_bit_cast(v8bf, h ? __builtin_shufflevector(both, both, 4, 5, 6, 7)
                                        : __builtin_shufflevector(both, both, 0, 1, 2, 3));
    }
  };
  Step st[kDepth];
  v4f acc[U][V];
  __amdgpu_buffer_rsrc_t rm, rj;
  uint32_t pm, pj;
  int c, n;  // entries, and this wave's steps: wv, wv + 4, ..

#ifdef __HIP_DEVICE_COMPILE__
  __device__ __forceinline__ void load(Step& d, int s) const {
    const int lane = threadIdx.x & 63, wv = tile_wave(threadIdx.x), row = lane >> 3;
    const int k = 64 * (4 * s + wv) + 8 * (lane & 7);
    // behind c, as behind the last row, 0: by an offset of all ones (a choice
    // between two offsets becomes branches that each wait for their loads)
    uint32_t past = k < c ? 0u : kNothing;
    asm volatile("" : "+v"(past));
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int v = 0; v < V; v++)
        d.j[v][h] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rj, ((uint32_t)(16 * v + 8 * h + row) * pj + 2u * (uint32_t)k) | past, 0, 0));
#pragma unroll
      for (int u = 0; u < U; u++)
        d.m[u][h] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rm, ((uint32_t)(16 * u + 8 * h + row) * pm + 2u * (uint32_t)k) | past, 0, 0));
    }
  }
  __device__ __forceinline__ void start(const TileOperand& om, const TileOperand& oj) {
    c = __builtin_amdgcn_readfirstlane(om.c);
    pm = (uint32_t)__builtin_amdgcn_readfirstlane((int)om.pitch);
    pj = (uint32_t)__builtin_amdgcn_readfirstlane((int)oj.pitch);
    rm = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(tile_scalar(om.base)), 0,
                                           (uint32_t)__builtin_amdgcn_readfirstlane(om.own) * pm, 0x00027000);
    rj = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(tile_scalar(oj.base)), 0,
                                           (uint32_t)__builtin_amdgcn_readfirstlane(oj.own) * pj, 0x00027000);
    n = ((c + 63) / 64 - tile_wave(threadIdx.x) + 3) / 4;
#pragma unroll
    for (int p = 0; p < kDepth; p++) {
      load(st[p], p);
      __builtin_amdgcn_sched_barrier(0);  // (in the order of their use: the loop waits by their number)
    }
  }
  __device__ __forceinline__ void run(uint8_t* lds) {
    const int lane = threadIdx.x & 63;
    uint8_t* mine = lds + tile_wave(threadIdx.x) * kWave;
    stream_meet();  // (the sums of the tile before have been read)
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int v = 0; v < V; v++) acc[u][v] = v4f{0.f, 0.f, 0.f, 0.f};
    // (steps behind the wave's last add zeros: a load or step that a branch skips
    // would have the compiler wait for more than the oldest loads)
    for (int s = 0; s < n; s += kDepth) {
#pragma unroll
      for (int p = 0; p < kDepth; p++) {
        // (one wave's LDS operations complete in order)
        asm volatile("" ::: "memory");
#pragma unroll
        for (int v = 0; v < V; v++) tile_put(mine + v * kTileBytes, lane, st[p].j[v][0], st[p].j[v][1]);
#pragma unroll
        for (int u = 0; u < U; u++) tile_put(mine + (V + u) * kTileBytes, lane, st[p].m[u][0], st[p].m[u][1]);
        asm volatile("" ::: "memory");
        Operand j[V], m[U];
#pragma unroll
        for (int v = 0; v < V; v++) j[v].both = tile_get(mine + v * kTileBytes, lane);
#pragma unroll
        for (int u = 0; u < U; u++) m[u].both = tile_get(mine + (V + u) * kTileBytes, lane);
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int v = 0; v < V; v++)
#pragma unroll
            for (int u = 0; u < U; u++) acc[u][v] = mfma_bf16(j[v].half(h), m[u].half(h), acc[u][v]);
        __builtin_amdgcn_sched_barrier(0);
        load(st[p], s + p + kDepth);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int v = 0; v < V; v++) pin4(acc[u][v]);
  }
  // Calls done(u, v, sums) for tile u of m and v of j in one of the waves, whose
  // lanes hold j = 4 (lane / 16) + 0..3 of m = lane % 16.
  template <typename Done>
  __device__ __forceinline__ void add(uint8_t* space, Done done) {
    const int lane = threadIdx.x & 63, wv = tile_wave(threadIdx.x);
    float* lds = reinterpret_cast<float*>(space);
    stream_meet();  // (all waves' operands have been read)
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int v = 0; v < V; v++) *reinterpret_cast<v4f*>(lds + ((wv * U + u) * V + v) * 256 + lane * 4) = acc[u][v];
    stream_meet();
#pragma unroll
    for (int i = 0; i < U * V / 4; i++) {
      const int f = i * 4 + wv, u = f / V, v = f % V;
      v4f s = *reinterpret_cast<const v4f*>(lds + f * 256 + lane * 4);
#pragma unroll
      for (int w = 1; w < 4; w++) s += *reinterpret_cast<const v4f*>(lds + (w * U * V + f) * 256 + lane * 4);
      done(u, v, s);
    }
  }
  // The waves meet, their LDS operations done; loads stay under way.
  static __device__ __forceinline__ void stream_meet() { tile_meet<63>(); }
#else
  __device__ void start(const TileOperand&, const TileOperand&) {}
  __device__ void run(uint8_t*) {}
  template <typename Done>
  __device__ void add(uint8_t*, Done) {}
#endif
};

}  // namespace moe
