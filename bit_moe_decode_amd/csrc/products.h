// products.h -- host interface of products.hip: matrix products of rows
// grouped by expert, and their gradients.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kProductMaxExperts = 1024;
constexpr int64_t kProductMaxRows = (int64_t)1 << 24;

struct ProductArgs {
  const int32_t* offsets;  // [experts + 1] first row of each expert
  int experts, n, k;
  int64_t rows;            // rows of the buffers
  const uint16_t *x, *w, *dy;
  void* y;                 // [rows][n]
  uint16_t* dx;            // [rows][k]
  void* dw;                // [experts][n][k]
  bool f32;                // y or dw is fp32, else bf16
  bool add;                // dw is added to
  float* space;            // the workspace: sums of parts, where there are several
  int parts, part;         // set by the launches: parts of the contraction, entries of one
};

size_t product_workspace(const ProductArgs& a);           // of y
size_t product_backward_workspace(const ProductArgs& a);  // of dx and of dw

hipError_t launch_product(const ProductArgs& a, hipStream_t stream);
hipError_t launch_product_dx(const ProductArgs& a, hipStream_t stream);
hipError_t launch_product_dw(const ProductArgs& a, hipStream_t stream);

}  // namespace moe
