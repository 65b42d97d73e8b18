// nm_norm.h -- parameter block and launchers of the layer norm kernels (internal).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nmk {

struct NormParams {
  CUtensorMap tm_x, tm_d;  // cached: X and dY in boxes of one strip
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
  uint32_t* status;
  int x_f32, y_f32;    // type of X (and dX), type of Y (forward) or dY (backward)
  // set by norm_shape
  int lpr, cluster, cached;
  int box_rows;         // of a TMA box
  int64_t tiles, rows;  // strips; rows of a CTA's slab
  uint32_t slab, smem;  // bytes
};

void norm_shape(NormParams& p, int64_t bytes);
cudaError_t launch_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_grad(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_grad_reduce(const float* part, int64_t tiles, int64_t K, float* dgamma, float* dbeta,
                                    cudaStream_t s);

}  // namespace nmk
