// nm_norm.h -- parameter block and launchers of the layer norm kernels (internal).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace nmk {

struct NormParams {
  const void* X;
  int64_t ldx;
  const void* dY;  // backward
  void* Y;         // forward: Y; backward: dX (row stride ldo)
  int64_t ldy;     // row stride of Y (forward) or dY (backward)
  int64_t ldo;
  int64_t K, T;
  const float *gamma, *beta;
  float eps;
  float *mean, *rstd;  // forward: outputs (may be null); backward: inputs
  float* part;         // backward: tiles x 2 x K row sums (dgamma, dbeta), or null
  int x_f32, y_f32;    // type of X (and dX), type of Y (forward) or dY (backward)
  // set by the launcher
  int lpr, cluster;
  int64_t tiles;
};

cudaError_t launch_norm(NormParams& p, cudaStream_t s);
// Fills p.lpr, p.cluster and p.tiles (the rows of p.part) and the rows per thread.
void norm_grad_shape(NormParams& p, int* rpt);
cudaError_t launch_norm_grad(NormParams& p, int rpt, cudaStream_t s);
cudaError_t launch_norm_grad_reduce(const float* part, int64_t tiles, int64_t K, float* dgamma, float* dbeta,
                                    cudaStream_t s);

}  // namespace nmk
