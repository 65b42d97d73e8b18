// nm_experts.h -- parameter blocks and shared checks of the products grouped by expert (internal).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "nm_host.h"

namespace nmk {

constexpr int kMaxExperts = 1024;

// Y[:, s] = W'_e X[:, s], or its transpose's: M rows of Y.
struct ExpertsParams {
  CUtensorMap tm_vals;  // compressed values {K / 2, R, E}, box {64, 64, 1}, 128B swizzle
  CUtensorMap tm_meta;  // tiled metadata {64 words, column blocks, E x row blocks}, box {64, 1, 8} (transposed: 4)
  CUtensorMap tm_x;     // X K x S (transposed: dY R x S), box {64, 64}, 128B swizzle
  CUtensorMap tm_y;     // Y M x S, box {64 bf16 | 32 fp32, 32 rows}, 128B swizzle
  const int32_t* offsets;
  void* Y;
  int64_t ldy;
  int32_t M, S, E;
  int32_t k_tiles, tiles_m, meta_rblocks;  // stages of a tile, row tiles, row blocks of one expert's metadata
  int out_f32;
  float* parts;  // two slots of partial sums a pair
  struct ExpertsCut* cuts;  // one a pair
  uint32_t* status;
};
// A tile whose stages several pairs have: the first of them notes it, for the kernel that joins their sums.
struct ExpertsCut {
  int32_t pairs;             // 0: this pair is not the first of one
  int32_t slot;              // of the first pair's sums; the others' are their first
  int32_t row0, x0, n;       // the tile
  int32_t c0, c1;            // the columns of it that are the expert's
  int32_t pad;
};
constexpr int kSlotCols = 128;
constexpr int64_t kSlotFloats = 256 * kSlotCols;

// Gradient of the survivors: dV_e[r][j] = sum over expert e's columns s of dY[r][s] X[k_j][s].
struct ExpertsGradParams {
  CUtensorMap tm_a, tm_b;  // dY R x S and X K x S, box {64, 64}, 128B swizzle
  CUtensorMap tm_dv;       // dV {K / 2, R, E} in 16-bit units (fp32: K), box {64, 32, 1}, 128B swizzle
  const int32_t* offsets;
  const uint32_t* meta;
  void* dV;
  int64_t R, K;
  int32_t S, E;
  int32_t tiles_m, tiles_n, meta_cblocks;
  int64_t meta_words;  // of one expert
  int out_f32;
  uint32_t* status;
};

// What the grouped products check alike.
nm_status check_experts(int n, int m, int64_t E, int64_t R, int64_t K, int64_t S, const int32_t* offsets);
// Few columns an expert: two forms.  Whole tiles of the general kernel, one launch, take wide_us a stage, and as long as the
// pairs with the most tiles; equal shares of all stages, the columns laid out with the reduction axis K contiguous first and
// the tiles that several pairs have parts of joined behind (three launches, 9 us more), take few_us.  Measured with one to
// 32 columns an expert, forward / input gradient: 8 x 11008 x 4096 (tiles 4.6 / 1.7 to a pair) whole 84 to 107 / 147 to 149
// us, shares 77 to 81 / 135 to 138; 2 x 4096 x 11008 (0.4 / 1.2) 41 / 61 to 63 and 29 to 30 / 47 to 48; 8 x 4096 x 4096
// (1.7) 38 to 50 / 62 to 65 and 39 to 40 / 62 to 64; 16 x 1024 x 1024 (0.9) 9 to 13 / 15 and 16 to 17 / 22 to 23.
// Two bounds come first, because the model knows nothing that grows with the columns (laying them out, partial sums, the
// join): at most 32 columns an expert, and a 16th of the output's rows.  With many tiles they are right (8 x 4096 x 4096,
// 64 columns each: whole 37 / 61, shares 45 / 68); with few tiles of long reductions they leave time behind (one expert of
// 11008 x 4096, input gradient of 48, 128 columns: whole 77, 76 and shares 34, 41; 8000 x 144, of 16: 55 and 17).
bool few_columns(const ExpertsParams& p, double few_us, double wide_us);
nm_status stage_few(ExpertsParams& p, const uint16_t* X, int64_t ldx, int64_t K, Staged& staged, cudaStream_t stream);
nm_status join_few(const ExpertsParams& p, cudaStream_t stream);
// SM pairs for as many tiles as there can be.
int experts_pairs(const ExpertsParams& p, int max_n);
nm_status make_experts_store_map(ExpertsParams& p, void* Y, int64_t M, int64_t S, int64_t ldy);

}  // namespace nmk
