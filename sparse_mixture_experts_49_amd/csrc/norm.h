// Launchers of the layer norm and its gradients (norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kNormMaxWidth = 32768;

struct NormShape {
  int64_t rows;
  int d;
  bool bf16, w_bf16, add_bf16;   // x and what goes with it; weight and bias; add
  float eps;
};

// A matrix by rows: `stride` elements from one to the next.
template <typename P>
struct Rows {
  P* p;
  int64_t stride;
};

struct NormArgs {
  NormShape sh;
  Rows<const void> x, add;       // add.p or null
  const void *weight, *bias;     // or null
  Rows<void> x_out, y;           // x_out.p or null
  float *mean, *rstd;            // or null
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  NormShape sh;
  Rows<const void> dy, x, d_x_out;   // d_x_out.p or null
  const void* weight;                // or null
  const float *mean, *rstd;
  Rows<void> d_x;                    // .p or null, as the next two
  float *d_weight, *d_bias;
  float* part;                       // workspace of norm_grad_part_bytes
};
size_t norm_grad_part_bytes(const NormShape& s);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

}  // namespace moe
