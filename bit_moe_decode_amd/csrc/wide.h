// wide.h -- host interface of wide.hip: the experts' step for any number of
// token rows whose routing is given.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "token_rows.h"

namespace moe {

// One step's shapes and workspace.  Sorted rows: the picks by expert in rows
// [0, picks), then one row a token for the shared expert.
struct WideArgs {
  int H, I, E, shared;
  int tokens;
  int64_t picks;       // 8 * tokens
  float eps;
  uint8_t* act_q;      // [tokens][H] FP8 codes of u
  float* act_s;        // [tokens][H/128] their scales times the row's rstd
  int32_t* order;      // [picks] flat pick of each sorted row
  uint8_t* mid_q;      // [picks + tokens][I]
  float* mid_s;        // [picks + tokens][I/128]
  float* y;            // [picks + tokens][H]
  int32_t* pos;        // [picks]
  int32_t* offsets;    // [E + 1]
  int32_t* counts;     // the sort's workspace
  RowTile* tiles;
  int32_t* n_tiles;
  int tile_rows, max_tiles;
};

struct WideWeights {
  const uint16_t* gamma;
  const uint8_t *gate_c, *up_c, *down_c;  // routed codes
  const float *gate_s, *up_s, *down_s;
  const uint8_t *sg_c, *su_c, *sd_c;      // shared codes
  const float *sg_s, *su_s, *sd_s;
};

int wide_tile_rows(int64_t picks, int experts);
int wide_max_tiles(int64_t picks, int experts, int shared_rows, int tile_rows);
hipError_t launch_wide(const WideArgs& a, const WideWeights& w, const uint16_t* x,
                       const int32_t* ids, const float* gates, uint16_t* out, hipStream_t stream);

}  // namespace moe
