// lm_loss.h -- host interface of lm_loss.hip: the LM head's softmax cross
// entropy and its gradients.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kLossMaxHidden = 32768;

struct LossArgs {
  const uint16_t* h;       // [rows][hidden]
  const uint16_t* w;       // [vocab][hidden]
  const int32_t* targets;  // [rows]
  int rows, vocab, hidden;
  float* loss;             // [rows]
  float* lse;              // [rows]
};

struct LossGradArgs {
  const uint16_t* h;
  const uint16_t* w;
  const int32_t* targets;
  const float* lse;
  const float* dloss;      // [rows]
  int rows, vocab, hidden;
  uint16_t* dh;            // [rows][hidden], or null
  void* dw;                // [vocab][hidden], or null
  bool f32, add;           // of dw
};

size_t loss_workspace(int rows, int vocab, int hidden);
size_t loss_backward_workspace(int rows, int vocab, int hidden);
hipError_t launch_loss(const LossArgs& a, void* workspace, hipStream_t stream);
hipError_t launch_loss_backward(const LossGradArgs& a, void* workspace, hipStream_t stream);

}  // namespace moe
