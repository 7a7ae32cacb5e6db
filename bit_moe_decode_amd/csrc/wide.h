// wide.h -- host interface of wide.hip: the experts' step for any number of
// token rows whose routing is given.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "token_rows.h"

namespace moe {

// sorted rows of a tile of the products, at most: by the FP8 MFMA, and summed in
// fp32 (and the shared expert's)
constexpr int kWideTile = 128, kWideExactTile = 80;

// One step's shapes and workspace.  Sorted rows: the picks by expert in rows
// [0, picks), then one row a token for the shared expert.
struct WideArgs {
  int H, I, E, shared;
  int tokens;
  int64_t picks;       // 8 * tokens
  int64_t rows;        // picks, and the tokens once more with a shared expert
  float eps;
  uint8_t* act_q;      // [tokens][H] FP8 codes of u
  float* act_s;        // [tokens][H/128] their scales times the row's rstd
  float* act_t;        // [H/128][rows] the same by sorted row
  int32_t* order;      // [picks] flat pick of each sorted row
  uint8_t* mid_q;      // [rows][I]
  float* mid_s;        // [I/128][rows]
  float* y;            // [rows][H]
  int32_t* pos;        // [picks]
  int32_t* offsets;    // [E + 1]
  int32_t* counts;     // the sort's workspace
  RowTile* tiles;
  int32_t* n_tiles;
  int max_tiles;
};

struct WideWeights {
  const uint16_t* gamma;
  const uint8_t *gate_c, *up_c, *down_c;  // routed codes
  const float *gate_s, *up_s, *down_s;
  const uint8_t *sg_c, *su_c, *sd_c;      // shared codes
  const float *sg_s, *su_s, *sd_s;
};

int wide_max_tiles(int64_t picks, int experts, int shared_rows);
hipError_t launch_wide(const WideArgs& a, const WideWeights& w, const uint16_t* x,
                       const int32_t* ids, const float* gates, uint16_t* out, hipStream_t stream);

}  // namespace moe
