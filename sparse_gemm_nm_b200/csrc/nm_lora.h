// nm_lora.h -- parameter blocks and launchers of the low-rank adapter kernels (internal).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nmk {

namespace lora {
constexpr int kTok = 64;       // tokens of a tile
constexpr int kMaxRank = 128;
constexpr int kMaxCat = 512;   // rank rows of all adapters together, in the projection's own reduction
inline int64_t tiles_of(int64_t T) { return (T + kTok - 1) / kTok; }
inline int rank_stride(int r) { return (r + 15) / 16 * 16; }
}  // namespace lora

// S[t][j] = sum_d M_a[j][d] Z[d][t], a the adapter of token t.  M is n x rank x D (trans = false) or n x D x rank
// (trans = true).  Results leave in one of three forms:
enum ShrinkOut : int {
  SHRINK_F32 = 0,     // S: T x rank_stride(rank) fp32 (rows of tokens without an adapter are not written)
  SHRINK_TERMS = 1,   // planes x T x rank_stride(rank): the bf16 terms of S (same rows)
  SHRINK_BLOCKS = 2   // planes x cat x ldp: the bf16 terms of s_a S, row a * rank + j, column t; 0 in the columns of
                      // other adapters' tokens and in rows past n * rank.  masks[tile]: the blocks of 64 rows that
                      // hold an adapter of the 64-token tile
};
struct LoraShrink {
  CUtensorMap tm_z;  // Z, box {64 tokens, 128 rows}, 128-byte swizzle
  CUtensorMap tm_m;  // M, when its rows start on 16 bytes: boxes of 32 ranks
  const uint16_t* M;
  const int32_t* adapter;
  const float* scale;  // SHRINK_BLOCKS
  int64_t n, D, T;
  int rank;
  int vec;             // M by tm_m
  int out, planes;
  float* S;
  uint16_t* terms;
  int64_t cat, ldp;    // SHRINK_BLOCKS: rows of a plane (a multiple of 64), row stride
  uint32_t* masks;
  const int32_t* idx;  // with inv: inv[idx[k]] = max k, over entries preset to -1
  int64_t idx_n;
  int32_t* inv;
  uint32_t* status;
  int cluster;         // CTAs that share a tile's reduction
  int stages;          // of its ring
  int early;           // runs beside its predecessor (pdl_enter)
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
  int batch;          // adapters' tiles in flight (set by the launcher, like base_off)
  uint32_t base_off;  // splits > 1: the summed base in shared memory
};
cudaError_t launch_lora_expand(LoraExpand& p, bool trans, cudaStream_t s);

// The adapters' second factors as one matrix, for the projection's own reduction: cat[row][a * rank + j] = B_a[row][j]
// (rows x cat, zero past n * rank; by_rank = false) or cat[a * rank + j][k] = A_a[j][idx[k]] (n * rank x ldc;
// by_rank = true, 0 for an entry of idx outside).  An Inf or NaN is replaced by 0 and its block's flag set, since it
// would meet the zeros of other requests; lora_mend adds its products afterwards.  Also presets inv to -1.
struct LoraCat {
  const uint16_t* M;
  int64_t n, rows;
  int rank;
  int64_t cat, ldc;
  const int32_t* idx;
  uint16_t* out;
  uint32_t* flags;  // one word per block, every one written
  int32_t* inv;     // rows entries, or null
  int blocks;
};
cudaError_t launch_lora_cat(LoraCat& p, bool by_rank, cudaStream_t s);
int lora_cat_blocks();

// What the projection with the adapters in its reduction leaves out: products of non-finite weights (flagged by
// launch_lora_cat), added to Y, and whole rows of Y that no entry of the index map names (inv < 0), written.  Returns at
// once where there is neither.
struct LoraMend {
  const uint16_t* M;  // as in LoraExpand
  const int32_t* adapter;
  int64_t n, rows, T;
  int rank;
  const uint16_t* blocks;  // SHRINK_BLOCKS planes
  int planes;
  int64_t cat, ldp;
  const uint32_t* flags;
  int nflags;
  const int32_t* inv;
  void* Y;
  int64_t ldy;
  int out_f32;
};
cudaError_t launch_lora_mend(const LoraMend& p, bool trans, cudaStream_t s);

// out_a = scale_a sum over the tokens t of adapter a of Z[m][t] V[t][j], stored rows x rank (by_rank = false) or
// rank x rows (by_rank = true) for every a; zeros for an adapter without tokens.
struct LoraOuter {
  CUtensorMap tm_z;  // Z, box {64 tokens, 128 rows}, 128-byte swizzle
  CUtensorMap tm_v;  // SHRINK_TERMS as {rank_stride, T, planes}, box {up to 64, 64, 1}, 128-byte swizzle
  const int32_t* adapter;
  const float* scale;
  int64_t n, rows, T;
  int rank;
  const int32_t* tiles;   // n x tiles_of(T): the tiles that hold tokens of the adapter, ascending
  const int32_t* counts;  // n: how many
  void* out;
  int out_f32;
  uint32_t* status;
  int cluster;
  int early;  // runs beside its predecessor (pdl_enter)
};
cudaError_t launch_lora_plan(const int32_t* adapter, int64_t T, int64_t n, int32_t* tiles, int32_t* counts,
                             cudaStream_t s);
cudaError_t launch_lora_outer(LoraOuter& p, bool by_rank, cudaStream_t s);

// inv[j] = the k with idx[k] == j (the largest such k), -1 where there is none.
cudaError_t launch_invert_map(const int32_t* idx, int64_t K, int32_t* inv, cudaStream_t s);

}  // namespace nmk
