// token_rows.h -- host interface of token_rows.hip: the sort of a batch's
// picks by group and the movement of rows into sorted order and back.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kSortThreads = 1024;
constexpr int kSortSteps = 8;          // picks a thread ranks at most
constexpr int kSortChunk = kSortSteps * kSortThreads;  // picks a block ranks at most
constexpr int kSortMaxGroups = 1024;   // one thread a group
constexpr int64_t kSortMaxPicks = (int64_t)1 << 24;

// Rows [row, end) of the sorted order, all of group `group`, of which one tile
// takes at most the sort's tile_rows (extra_rows for the rows behind the picks).
struct RowTile {
  int32_t group, row, end;
};

struct SortArgs {
  const int32_t* ids;  // [picks]
  int64_t picks;
  int groups;
  int32_t* offsets;  // [groups + 1]
  int32_t* order;    // [picks]
  int32_t* pos;      // [picks]
  int32_t* counts;   // [chunks][groups], workspace of more than one chunk
  // Optional: the tiles of tile_rows rows covering every group's rows, then
  // those of extra_rows covering `extra` more rows behind the picks as group
  // `groups`.
  RowTile* tiles;
  int32_t* n_tiles;
  int tile_rows, extra, extra_rows;
  int spill;  // 1: picks in no group go to the last one
  int chunks, bits, steps;  // set by launch_sort: blocks, bits of a group, picks a thread
};

size_t sort_workspace(int64_t picks, int groups);
// The most tiles of `tile_rows` rows that cover `picks` picks of `groups`
// groups: every group has at most one tile that is not full.
inline int64_t sort_max_tiles(int64_t picks, int groups, int tile_rows) {
  return picks / tile_rows + (picks < groups ? picks : groups);
}
hipError_t launch_sort(SortArgs a, hipStream_t stream);

struct RowArgs {
  const int32_t* pos;  // [tokens, top_k]
  int64_t tokens;
  int top_k, hidden;
  int rows;  // rows of the sorted buffer
  // set by the launches: blocks a row, and the first token of one of several
  uint32_t parts;
  int64_t first;
};

hipError_t launch_gather(const RowArgs& a, bool f32, const void* x, void* xs, hipStream_t stream);
// gates null: every weight 1; add null: nothing added
hipError_t launch_combine_rows(const RowArgs& a, bool f32, const void* y, const float* gates,
                               const void* add, void* out, hipStream_t stream);
hipError_t launch_combine_bwd(const RowArgs& a, bool f32, const void* dout, const void* y,
                              const float* gates, void* dy, float* dgates, hipStream_t stream);

}  // namespace moe
