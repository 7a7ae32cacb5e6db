// embed.h -- host interface of embed.hip: the embedding lookup and its gradient.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct EmbedArgs {
  const int32_t* ids;  // [rows]
  int rows, vocab, hidden;
  float scale;
  bool f32;            // rows (out or dout) are fp32, else bf16
};

struct EmbedGradArgs {
  EmbedArgs e;
  const void* dout;    // [rows][hidden]
  void* dtable;        // [vocab][hidden]
  bool f32, add;       // of dtable
};

hipError_t launch_embed(const EmbedArgs& a, const void* table, void* out, hipStream_t stream);
size_t embed_backward_workspace(int rows, int vocab, int hidden);
hipError_t launch_embed_backward(const EmbedGradArgs& a, void* workspace, hipStream_t stream);

// The rows with an id in [0, vocab), by (id, row): their numbers in *order, how
// many in *kept, both in the workspace.  `clear` (or null) is filled with zeros
// beside it.
size_t id_sort_workspace(int rows, int vocab);
hipError_t launch_id_sort(const int32_t* ids, int rows, int vocab, void* workspace, void* clear, size_t clear_bytes,
                          int32_t** order, const int32_t** kept, hipStream_t stream);

}  // namespace moe
