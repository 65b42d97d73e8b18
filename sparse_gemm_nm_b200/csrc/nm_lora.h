// nm_lora.h -- parameter blocks and launchers of the low-rank adapter kernels (internal).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace nmk {

namespace lora {
constexpr int kTok = 64;       // tokens of a tile
constexpr int kMaxRank = 128;
inline int64_t tiles_of(int64_t T) { return (T + kTok - 1) / kTok; }
inline int rank_stride(int r) { return (r + 15) / 16 * 16; }
}  // namespace lora

// S[t][j] = sum_d M_a[j][d] Z[d][t], a the adapter of token t (rows of tokens without one are not written).
// M is n x rank x D (trans = false) or n x D x rank (trans = true).
struct LoraShrink {
  const uint16_t* M;
  const uint16_t* Z;
  int64_t ldz;
  const int32_t* adapter;
  int64_t n, D, T;
  int rank;
  int vec;      // every row of M starts on 16 bytes
  float* S;     // T x rank_stride(rank)
  int cluster;  // CTAs that share a tile's reduction
};
cudaError_t launch_lora_shrink(LoraShrink& p, bool trans, cudaStream_t s);

// Y[row][t] = base[row][t] + scale_a sum_j M_a[row][j] S[t][j].  M is n x rows x rank (trans = false) or
// n x rank x rows (trans = true).  base is the sum over `splits` fp32 matrices (row stride ldb); with base_row, row
// `row` of the base is its row base_row[row] (none when negative).
struct LoraExpand {
  const uint16_t* M;
  const float* S;
  const int32_t* adapter;
  const float* scale;
  int64_t n, rows, T;
  int rank;
  int vec;
  const float* base;
  int splits;
  int64_t split_stride, ldb;
  const int32_t* base_row;
  void* Y;
  int64_t ldy;
  int out_f32;
};
cudaError_t launch_lora_expand(const LoraExpand& p, bool trans, cudaStream_t s);

// out_a = scale_a sum over the tokens t of adapter a of Z[m][t] V[t][j], stored rows x rank (by_rank = false) or
// rank x rows (by_rank = true) for every a; zeros for an adapter without tokens.
struct LoraOuter {
  const uint16_t* Z;
  int64_t ldz;
  const float* V;  // T x rank_stride(rank)
  const int32_t* adapter;
  const float* scale;
  int64_t n, rows, T;
  int rank;
  const int32_t* tiles;   // n x tiles_of(T): the tiles that hold tokens of the adapter, ascending
  const int32_t* counts;  // n: how many
  void* out;
  int out_f32;
  int cluster;
};
cudaError_t launch_lora_plan(const int32_t* adapter, int64_t T, int64_t n, int32_t* tiles, int32_t* counts,
                             cudaStream_t s);
cudaError_t launch_lora_outer(LoraOuter& p, bool by_rank, cudaStream_t s);

// inv[j] = the k with idx[k] == j (the largest such k), -1 where there is none.
cudaError_t launch_invert_map(const int32_t* idx, int64_t K, int32_t* inv, cudaStream_t s);

}  // namespace nmk
