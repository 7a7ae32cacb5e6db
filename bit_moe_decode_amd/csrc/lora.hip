// lora.hip -- low-rank adapters of many requests at once, beside a projection
// they share: row r with adapter i = ids[r] gets
//   y[r] = bf16( base[r] + scale_i * B_i (A_i x[r]) )
// with A_i [rank, K], B_i [N, rank].  Rows without an adapter keep base.  The
// inner product A x is kept in fp32, never rounded.
#include "lora.h"

namespace moe {

// A x of one row over one part of K: lanes take 8 inputs each, kept in
// registers for every rank; a wave takes the ranks wv, wv + 4, ...
constexpr int kShrinkPart = 2048;  // inputs a part at most: 4 x 8 a lane

__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs l, const uint16_t* __restrict__ x) {
  const int r = blockIdx.x, part = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int id = l.ids[r];
  if ((uint32_t)id >= (uint32_t)l.adapters) return;
  const int rank = lora_rank(l, id);
  const int chunks = l.k / 8;  // of 8 inputs
  const int c0 = (int)((int64_t)chunks * part / l.k_parts), c1 = (int)((int64_t)chunks * (part + 1) / l.k_parts);
  u32x4 xv[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int c = c0 + i * 64 + lane;
    xv[i] = c < c1 ? ld16(x + (size_t)r * l.k + 8 * c) : u32x4{0u, 0u, 0u, 0u};
  }
  for (int j = wv; j < rank; j += 4) {
    const uint16_t* row = l.a + ((size_t)id * l.max_rank + j) * l.k;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int c = c0 + i * 64 + lane;
      if (c >= c1) continue;
      const u32x4 av = ld16(row + 8 * c);
#pragma unroll
      for (int q = 0; q < 4; q++) {
        s = fmaf(__uint_as_float(av[q] << 16), __uint_as_float(xv[i][q] << 16), s);
        s = fmaf(__uint_as_float(av[q] & 0xFFFF0000u), __uint_as_float(xv[i][q] & 0xFFFF0000u), s);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
    if (lane == 0) l.v[((size_t)part * l.rows + r) * l.max_rank + j] = s;
  }
}

// base + B v of one row, an output a thread.
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs l, const uint16_t* base,
                                                          uint16_t* y) {
  __shared__ float sv[kLoraMaxRank];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int n = blockIdx.y * 256 + tid;
  LoraArgs one = l;
  one.ids = l.ids + r;
  one.v = l.v + (size_t)r * l.max_rank;
  lora_load_v(one, 1, sv, tid, 256);
  __syncthreads();
  if (n >= l.n) return;
  const size_t at = (size_t)r * l.n + n;
  y[at] = f32_to_bf16(bf16_to_f32(base[at]) + lora_term(one, 0, n, sv));
}

int lora_k_parts(int rows, int k) {
  const int least = (k + kShrinkPart - 1) / kShrinkPart;
  int parts = (1024 + rows - 1) / rows;  // about four blocks a CU
  const int most = (k + 511) / 512;
  parts = parts < most ? parts : most;
  return parts > least ? parts : least;
}

size_t lora_workspace(int adapters, int max_rank, int n, int k, int rows) {
  return (size_t)lora_k_parts(rows, k) * rows * max_rank * sizeof(float);
}

hipError_t launch_lora_shrink(const LoraArgs& l, const uint16_t* x, hipStream_t stream) {
  hipLaunchKernelGGL(lora_shrink_kernel, dim3(l.rows, l.k_parts), dim3(256), 0, stream, l, x);
  return hipGetLastError();
}

hipError_t launch_lora(LoraArgs l, const uint16_t* x, const uint16_t* base, uint16_t* y,
                       hipStream_t stream) {
  hipError_t e = launch_lora_shrink(l, x, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_expand_kernel, dim3(l.rows, (l.n + 255) / 256), dim3(256), 0, stream, l,
                     base, y);
  return hipGetLastError();
}

}  // namespace moe
