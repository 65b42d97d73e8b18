// nm_xent.cu -- softmax cross entropy of a pruned output head, forward and
// backward, without the logits of the whole vocabulary in memory.
//
// With the logits z = (W' Pi) X (R x T, R the vocabulary):
//   lse[t] = log sum_v exp z[v][t],  loss[t] = lse[t] - z[target[t]][t],
//   G[v][t] = dloss[t] (exp(z[v][t] - lse[t]) - [v == target[t]]),
//   dX = (W' Pi)^T G,  dV = the survivors' entries of G Xp^T.
// Forward: every group of rows leaves a pair (max, sum of exp(z - max)) per
// token, and the token's target row its logit; one last pass joins the pairs in
// order.  The maxima are logits as they are, and differences are taken before
// anything is scaled: the largest term of a sum is then exactly 1, and
// loss = (max - z[target]) + log(sum) has no rounding of the size of the logits
// and is never negative (lse - z[target] of scaled sums was off by 1.5e-5, and
// below 0, for logits of 200).  On shapes of the SM-pair GEMM its epilogue makes
// the pairs of 32 rows from the accumulator in TMEM, and no logit is written
// (32000 x 4096 x 2048 logits would be 262 MB written and read); elsewhere the
// vocabulary is taken in pieces of rows whose logits xent_pairs_kernel reads, 256
// rows to a pair.
// Backward: the logits of a piece are computed again and become G (bf16, rounded
// once: it is an operand of the tensor cores like the dY of nm_spmm_t; two terms
// for up to 256 tokens, see run_xent_grad), again in
// the SM-pair GEMM's epilogue where that serves; G meets the decompressed piece
// of W' in a product that adds to a K x T fp32 accumulator, and Xp in the
// survivor-sampled product for dV.  The accumulator takes one addition per
// piece, in the order of the pieces; with few tiles of dX there are several, for
// ranges of a piece's rows side by side.  Their sum is rounded to dX at the end.
// Launches that need nothing of the one before them start beside it.
//
// Measured: 32000 x 4096 x 2048 forward 264 us (floor 160 us of sparse products;
// the GEMM itself sets the time: its MMA issue and, in a loop, the power cap, 305
// us), backward 1135 us (two dense products of 0.54 TFLOP beside the sparse one;
// 1265 us in a loop); 37 tokens 47 us (floor 23 us of weights; 250 row tiles on
// 148 SMs, and every tile reads X again); 1000 x 768 x 256 backward 33 us,
// launches and their latency.
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_ptx.cuh"
#include "nm_spmm.h"

namespace nmk {

namespace xent {
constexpr int kPairRows = 256;  // logits rows joined into one (max, sum) pair by xent_pairs_kernel
constexpr float kLog2e = 1.4426950408889634f;
}  // namespace xent

// part[pair][t] = (max, sum exp(z - max)) over one pair's kPairRows rows of the logits piece; the rows of targets write
// their logit.  Z is the sum of `splits` matrices.  One block: 32 tokens, one pair.
__global__ void __launch_bounds__(256) xent_pairs_kernel(const float* Z, int splits, int64_t split_stride, int64_t ldz,
                                                         int64_t rows, int64_t T, int64_t v0, const int32_t* target,
                                                         float2* part, float* z_target) {
  using namespace xent;
  __shared__ float s_max[8][32], s_sum[8][32];
  pdl_gate();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 32 + lane;
  const int64_t r0 = (int64_t)blockIdx.y * kPairRows + warp;
  constexpr int kEach = kPairRows / 8;  // rows of a warp, all loaded before the first exponential
  float z[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = r0 + 8 * i;
    z[i] = t < T && r < rows ? __ldcg(Z + r * ldz + t) : -INFINITY;
  }
  for (int q = 1; q < splits; ++q) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (t < T && r0 + 8 * i < rows) z[i] += __ldcg(Z + q * split_stride + (r0 + 8 * i) * ldz + t);
  }
  const int64_t want = t < T ? (int64_t)__ldg(target + t) - v0 - r0 : -1;
  float top = -3.0e38f, sum = 0.f;  // finite: (-inf) - (-inf) must not arise
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    top = fmaxf(top, z[i]);
    if (want == 8 * i) z_target[t] = z[i];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += exp2_fast((z[i] - top) * kLog2e);
  s_max[warp][lane] = top;
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && t < T) {
    float m = s_max[0][lane];
    for (int w = 1; w < 8; ++w) m = fmaxf(m, s_max[w][lane]);
    float s = 0.f;
    for (int w = 0; w < 8; ++w) s += s_sum[w][lane] * exp2_fast((s_max[w][lane] - m) * kLog2e);
    part[(v0 / kPairRows + blockIdx.y) * T + t] = make_float2(m, s);
  }
}

// Joins a token's pairs: with M the largest max and S = sum_p s_p exp(m_p - M), lse = M + log S and
// loss = (M - z[target]) + log S.
__global__ void __launch_bounds__(1024) xent_join_kernel(const float2* part, int64_t pairs, int64_t R, int64_t T,
                                                         const int32_t* target, const float* z_target, float* loss,
                                                         float* lse) {
  using namespace xent;
  __shared__ float s_max[32][33], s_sum[32][33];
  pdl_gate();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 32 + lane;
  float m = -3.0e38f, s = 0.f;
  if (t < T) {
    for (int64_t p0 = warp; p0 < pairs; p0 += 32 * 8) {  // eight pairs in flight
      float2 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = p0 + 32 * i < pairs ? __ldcg(part + (p0 + 32 * i) * T + t) : make_float2(-3.0e38f, 0.f);
      float top = m;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, q[i].x);
      s *= exp2_fast((m - top) * kLog2e);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += q[i].y * exp2_fast((q[i].x - top) * kLog2e);
      m = top;
    }
  }
  s_max[warp][lane] = m;
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && t < T) {
    float top = s_max[0][lane];
#pragma unroll
    for (int w = 1; w < 32; ++w) top = fmaxf(top, s_max[w][lane]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) sum += s_sum[w][lane] * exp2_fast((s_max[w][lane] - top) * kLog2e);
    const float l = logf(sum);
    const int32_t want = __ldg(target + t);
    lse[t] = top + l;
    loss[t] = want >= 0 && (int64_t)want < R ? (top - __ldcg(z_target + t)) + l : 0.f;
  }
}

// The SM-pair epilogues' per-token data, on 16 bytes and padded to `padded` tokens (no target, factor 0).
__global__ void __launch_bounds__(256) xent_columns_kernel(const int32_t* target, const float* lse, const float* dloss,
                                                           int64_t R, int64_t T, int64_t padded, int32_t* tgt,
                                                           float* lse_out, float* d) {
  pdl_gate();
  const int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (t >= padded) return;
  const int32_t w = t < T ? __ldg(target + t) : -1;
  const bool has = w >= 0 && (int64_t)w < R;
  tgt[t] = has ? w : -1;
  if (lse) {
    lse_out[t] = has ? __ldcg(lse + t) : 0.f;
    d[t] = has ? __ldg(dloss + t) : 0.f;
  }
}

// G = dloss (exp(z - lse) - [row == target]) of a logits piece, bf16; 0 where the target is outside [0, R) or dloss is 0,
// whatever the logits are.
// Columns T .. width - 1 (padding to whole 16-byte pieces) are written as 0.  TWO: what the rounding left over follows, as
// a second bf16 term, in columns width .. 2 width - 1.
template <bool TWO>
__global__ void __launch_bounds__(256) xent_g_kernel(const float* Z, int64_t ldz, int64_t rows, int64_t T, int64_t R,
                                                     int64_t v0, const int32_t* target, const float* lse,
                                                     const float* dloss, uint16_t* G, int64_t ldg, int64_t width) {
  using namespace xent;
  pdl_gate();
  const int64_t t = ((int64_t)blockIdx.x * 32 + (threadIdx.x & 31)) * 2;
  if (t >= width) return;
  float l[2], d[2];
  int64_t want[2];
  bool live[2];
  for (int j = 0; j < 2; ++j) {
    const int64_t tj = t + j;
    const int32_t w = tj < T ? __ldg(target + tj) : -1;
    const bool has = w >= 0 && (int64_t)w < R;
    want[j] = (int64_t)w - v0;
    l[j] = has ? __ldcg(lse + tj) : 0.f;
    d[j] = has ? __ldg(dloss + tj) : 0.f;
    live[j] = d[j] != 0.f;  // a NaN is
  }
  for (int64_t r = (int64_t)blockIdx.y * 64 + (threadIdx.x >> 5); r < rows && r < ((int64_t)blockIdx.y + 1) * 64; r += 8) {
    float g[2] = {0.f, 0.f};
    if (live[0]) g[0] = d[0] * (exp2f((__ldcg(Z + r * ldz + t) - l[0]) * kLog2e) - (r == want[0] ? 1.f : 0.f));
    if (live[1]) g[1] = d[1] * (exp2f((__ldcg(Z + r * ldz + t + 1) - l[1]) * kLog2e) - (r == want[1] ? 1.f : 0.f));
    const uint32_t hi = pack_bf16x2(g[0], g[1]);
    *reinterpret_cast<uint32_t*>(G + r * ldg + t) = hi;
    if (TWO) *reinterpret_cast<uint32_t*>(G + r * ldg + width + t) = bf16x2_rest(g[0], g[1], hi);
  }
}

// dX[idx[k]] (dX[k] without idx) = the accumulators' rows k, rounded to bf16; rows mapped outside [0, K) are dropped.
// `parts` sums are added in order: `terms` column blocks of `width` columns in each of the ranges' accumulators.
__global__ void __launch_bounds__(256) xent_round_kernel(const float* acc, int parts, int terms, int64_t width,
                                                         int64_t lda, int64_t K, int64_t T, const int32_t* idx,
                                                         uint16_t* dX, int64_t lddx) {
  pdl_gate();
  const int64_t pieces = (T + 7) / 8, total = K * pieces;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t k = i / pieces, t = (i - k * pieces) * 8;
    const int64_t row = idx ? (int64_t)__ldg(idx + k) : k;
    if (row < 0 || row >= K) continue;
    const float* a = acc + k * lda + t;
    uint16_t* d = dX + row * lddx + t;
    auto part = [&](int q) { return a + q / terms * K * lda + q % terms * width; };
    if (t + 8 <= T) {
      float4 x = __ldcg(reinterpret_cast<const float4*>(a)), y = __ldcg(reinterpret_cast<const float4*>(a) + 1);
      for (int q = 1; q < parts; ++q) {
        const float4* b = reinterpret_cast<const float4*>(part(q));
        const float4 u = __ldcg(b), v = __ldcg(b + 1);
        x.x += u.x;
        x.y += u.y;
        x.z += u.z;
        x.w += u.w;
        y.x += v.x;
        y.y += v.y;
        y.z += v.z;
        y.w += v.w;
      }
      *reinterpret_cast<uint4*>(d) = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                                                pack_bf16x2(y.z, y.w));
    } else {
      for (int j = 0; t + j < T; ++j) {
        float x = __ldcg(a + j);
        for (int q = 1; q < parts; ++q) x += __ldcg(part(q) + j);
        d[j] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xFFFFu);
      }
    }
  }
}

namespace {

struct Head {  // the compressed head and its input (permuted rows already gathered)
  const uint16_t* values;
  const uint32_t* meta;
  int n, m;
  int64_t R, K, T;
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* row_values(int64_t v) const { return values + v * value_cols(K, n, m); }
  const uint32_t* row_meta(int64_t v) const {  // v a multiple of 16 for the tiled metadata
    return meta + (tiled_meta(n, m) ? v / 16 * meta_col_blocks(K) * 64 : v * meta_cols(K, n, m));
  }
};

nm_status check_head(int n, int m, int64_t R, int64_t K, int64_t T) {
  if (R < 0 || K < 0 || T < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (!pattern_ok(n, m)) return fail(NM_ERR_INVALID_ARG, "pattern %d:%d not supported (M in 2,4,8,16; 1<=N<M)", n, m);
  if (K % m != 0) return fail(NM_ERR_INVALID_ARG, "K=%lld is not a multiple of M=%d", (long long)K, m);
  if (R == 0 || K == 0) return fail(NM_ERR_INVALID_ARG, "an output head needs at least one row and one column");
  if (R >= kMaxDim || K >= kMaxDim || T >= kMaxDim) return fail(NM_ERR_UNSUPPORTED, "dimensions must stay below 2^31");
  return NM_OK;
}

// Rows of one piece: a multiple of 256 that takes about 64 MB (fp32 logits, or bf16 gradients where no logits are
// written), so that it stays in L2.
int64_t piece_rows(int64_t R, int64_t K, int64_t T, int64_t bytes = 4) {
  int64_t rows = (64ll << 20) / bytes / (T > 0 ? T : 1) / 256 * 256;
  const int64_t weights = (256ll << 20) / (2 * K) / 256 * 256;  // of a piece, where they are decompressed
  if (rows > weights) rows = weights;
  if (rows < 256) rows = 256;
  if (rows > (1 << 21)) rows = 1 << 21;  // the element-wise kernels' grids: 64 rows a block, 65535 blocks
  return rows < R ? rows : R;
}

// Where only the one-SM GEMM serves a shape, a piece's logits are the dense product of its decompressed weights, except
// for whole 128-deep stages and few tokens, whose weights that GEMM streams by TMA (forward of 15 x 3592 x 876 175 us with
// the one-SM GEMM and 30 dense, 8980 x 216 x 8192 474 and 221, 20482 x 128 x 5443 344 and 308; 32000 x 4096 x 100 100 and
// 161; gradients of 149 x 3224 x 28 245 and 80).
bool dense_logits(int64_t K, int64_t T) { return K % 128 != 0 || T >= 192; }

// Xp[k] = X[idx[k]] when there is an index map.
nm_status gather_input(Head& h, const int32_t* idx, Staged& staged, cudaStream_t s) {
  if (!idx) return NM_OK;
  const int64_t ldp = (h.T + 7) / 8 * 8;
  cudaError_t e = staged.get((size_t)(h.K * ldp * 2));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the permuted input");
  e = launch_gather_rows(h.X, h.ldx, idx, h.K, h.T, staged.as<uint16_t>(), ldp, s);
  if (e != cudaSuccess) return cuda_fail(e, "gather launch");
  h.X = staged.as<uint16_t>();
  h.ldx = ldp;
  return NM_OK;
}

// Per-token data of the SM-pair epilogues: [target | lse | d], each padded to whole tiles (256 and 224 columns).
int64_t padded_tokens(int64_t T) { return (T + 255) / 256 * 256 + 256; }
nm_status column_data(const Head& h, const int32_t* target, const float* lse, const float* dloss, PairEpiData& epi,
                      Staged& staged, cudaStream_t s) {
  const int64_t n = padded_tokens(h.T);
  cudaError_t e = staged.get((size_t)(n * 4 * (lse ? 3 : 1)));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the token data");
  int32_t* tgt = staged.as<int32_t>();
  float* lse_to = staged.as<float>() + n;
  e = launch_pdl(xent_columns_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, target, lse, dloss, h.R, h.T, n,
                 tgt, lse_to, lse_to + n);
  count_launch();
  epi.target = tgt;
  epi.lse = lse_to;
  epi.d = lse_to + n;
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "token data launch");
}

nm_status run_xent(Head h, const int32_t* idx, const int32_t* target, float* loss, float* lse, cudaStream_t s) {
  Staged xp(s), work(s), buf(s), ws(s), cols(s);
  nm_status st = gather_input(h, idx, xp, s);
  if (st != NM_OK) return st;
  const bool fused = spmm_pair_serves(h.values, h.meta, h.n, h.m, h.K, h.T);
  const int64_t per = fused ? 32 : xent::kPairRows;
  const int64_t pairs = (h.R + per - 1) / per;
  cudaError_t e = work.get((size_t)(pairs * h.T * 8 + h.T * 4));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the sums");
  float2* part = work.as<float2>();
  float* z_target = reinterpret_cast<float*>(part + pairs * h.T);
  const unsigned tb = (unsigned)((h.T + 31) / 32);
  if (fused) {  // the GEMM's epilogue leaves the pairs: no logits are written at all
    PairEpiData epi = {};
    epi.mode = PAIR_EPI_LSE;
    epi.part = part;
    epi.z_target = z_target;
    st = column_data(h, target, nullptr, nullptr, epi, cols, s);
    if (st == NM_OK)
      st = run_spmm_epilogue(h.values, h.meta, h.n, h.m, h.R, h.K, h.X, h.ldx, h.T, nullptr, 0, epi, s);
    if (st != NM_OK) return st;
  } else {
    const bool dense = dense_logits(h.K, h.T);
    const int64_t rows = piece_rows(h.R, h.K, h.T), ldz = (h.T + 3) / 4 * 4, ldk = (h.K + 7) / 8 * 8;
    Parts parts;
    const int64_t at_z = parts.take(rows * ldz * 4), at_wd = parts.take(dense ? rows * ldk * 2 : 0);
    e = buf.get(parts.size());
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the logits piece");
    float* z = buf.as<float>(at_z);
    uint16_t* wd = buf.as<uint16_t>(at_wd);
    for (int64_t v0 = 0; v0 < h.R; v0 += rows) {
      const int64_t n = h.R - v0 < rows ? h.R - v0 : rows;
      ws.release();
      GemmPartials raw{&ws, false, 1, 0, 0};
      if (dense) {
        e = launch_decompress(h.row_values(v0), h.row_meta(v0), n, h.K, h.n, h.m, wd, ldk, s);
        if (e != cudaSuccess) return cuda_fail(e, "decompress launch");
        st = dense_product(wd, ldk, n, h.K, h.X, h.ldx, h.T, z, ldz, s);
      } else {
        st = run_spmm(h.row_values(v0), h.row_meta(v0), h.n, h.m, n, h.K, nullptr, h.X, h.ldx, h.T, z, ldz, NM_OUT_F32,
                      &raw, s);
      }
      if (st != NM_OK) return st;
      const bool split = raw.splits > 1;
      e = launch_pdl(xent_pairs_kernel, dim3(tb, (unsigned)((n + per - 1) / per)), dim3(256), 0, s,
                     (const float*)(split ? ws.as<float>() : z), raw.splits, raw.split_stride,
                     split ? raw.ld : ldz, n, h.T, v0, target, part, z_target);
      count_launch();
      if (e != cudaSuccess) return cuda_fail(e, "cross-entropy launch");
    }
  }
  e = launch_pdl(xent_join_kernel, dim3(tb), dim3(1024), 0, s, (const float2*)part, pairs, h.R, h.T, target,
                 (const float*)z_target, loss, lse);
  count_launch();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "cross-entropy launch");
}

nm_status run_xent_grad(Head h, const int32_t* idx, const int32_t* target, const float* lse, const float* dloss,
                        uint16_t* dX, int64_t lddx, uint16_t* dV, cudaStream_t s) {
  Staged xp(s), buf(s), cols(s);
  nm_status st = gather_input(h, idx, xp, s);
  if (st != NM_OK) return st;
  const bool fused = spmm_pair_serves(h.values, h.meta, h.n, h.m, h.K, h.T);
  const bool dense = !fused && dense_logits(h.K, h.T);
  const int64_t ldz = (h.T + 3) / 4 * 4, ldk = (h.K + 7) / 8 * 8;
  // With few tokens a sum has few terms, and the rounding of G to bf16 can be half again the rounding of the result
  // (149 x 3224 x 28: 2.5e-3 of the gradients instead of 1.7e-3).  Up to 128 tokens G's two terms fit the one column tile
  // of dX, up to 256 two, and the steps of dV hide behind its epilogue, so they cost little; above, the products do, and
  // G is rounded once.  The rule is by tokens alone, whichever GEMM serves the shape: adding one does not change it (on
  // the SM-pair GEMM 32000 x 4096 x 256 takes 412 us with two terms and 361 with one, 1000 x 768 x 256 38 and 34).
  const bool two = h.T <= 256;
  const int terms = two ? 2 : 1;
  // The value gradient's product takes X once for each term.  Up to 32 tokens both terms fit one 64-column box and meet a
  // copy of X twice side by side (32000 x 512 x 8 97 us, in two boxes 107); above, a term has whole boxes of its own and
  // the product reads X again (1000 x 768 x 256 38 us, with the copies 44).
  const bool twice = two && h.T <= 32;
  const int64_t per = two && !twice ? 64 : 8, width = (h.T + per - 1) / per * per;  // columns of one term
  const int64_t rows = piece_rows(h.R, h.K, two ? width : h.T, fused && !two ? 2 : 4);  // by G's or the logits' bytes
  const int64_t ldg = terms * width, lda = two ? ldg : ldz, tokens = two ? ldg : h.T;  // of the products
  const int ranges = dense_t_ranges(rows, h.K, tokens);
  PairEpiData epi = {};
  epi.mode = two ? PAIR_EPI_XGRAD2 : PAIR_EPI_XGRAD;
  if (fused) st = column_data(h, target, lse, dloss, epi, cols, s);
  if (st != NM_OK) return st;
  Parts parts;
  const int64_t at_g = parts.take(rows * ldg * 2), at_z = parts.take(fused ? 0 : rows * ldz * 4);
  const int64_t at_wd = parts.take(dX || dense ? rows * ldk * 2 : 0), at_acc = parts.take(dX ? ranges * h.K * lda * 4 : 0);
  const int64_t at_x2 = parts.take(twice && dV ? h.K * ldg * 2 : 0);
  cudaError_t e = buf.get(parts.size());
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the gradient piece");
  uint16_t* g = buf.as<uint16_t>(at_g);
  uint16_t* wd = buf.as<uint16_t>(at_wd);
  float* z = buf.as<float>(at_z);
  float* acc = buf.as<float>(at_acc);
  const uint16_t* x = h.X;  // of the value gradient
  int64_t ldx = h.ldx, x_tokens = h.T;
  if (twice && dV) {
    uint16_t* x2 = buf.as<uint16_t>(at_x2);
    for (int q = 0; q < 2; ++q) {
      e = launch_gather_rows(h.X, h.ldx, nullptr, h.K, h.T, x2 + q * width, ldg, s, nullptr, q > 0);
      if (e != cudaSuccess) return cuda_fail(e, "input copy launch");
    }
    x = x2;
    ldx = x_tokens = ldg;
  }
  for (int64_t v0 = 0; v0 < h.R; v0 += rows) {
    const int64_t n = h.R - v0 < rows ? h.R - v0 : rows;
    if (fused) {  // the GEMM's epilogue turns the logits into G
      epi.row0 = v0;
      st = run_spmm_epilogue(h.row_values(v0), h.row_meta(v0), h.n, h.m, n, h.K, h.X, h.ldx, h.T, g, ldg,
                             epi, s);
      if (st != NM_OK) return st;
    } else {
      if (dense) {
        e = launch_decompress(h.row_values(v0), h.row_meta(v0), n, h.K, h.n, h.m, wd, ldk, s);
        if (e != cudaSuccess) return cuda_fail(e, "decompress launch");
        st = dense_product(wd, ldk, n, h.K, h.X, h.ldx, h.T, z, ldz, s);
      } else {
        st = spmm_rows(h.row_values(v0), h.row_meta(v0), h.n, h.m, n, h.K, h.X, h.ldx, h.T, z, ldz, NM_OUT_F32, s);
      }
      if (st != NM_OK) return st;
      const dim3 grid((unsigned)((width / 2 + 31) / 32), (unsigned)((n + 63) / 64));
      e = launch_pdl(two ? xent_g_kernel<true> : xent_g_kernel<false>, grid, dim3(256), 0, s, (const float*)z, ldz, n, h.T,
                     h.R, v0, target, lse, dloss, g, ldg, width);
      count_launch();
      if (e != cudaSuccess) return cuda_fail(e, "cross-entropy gradient launch");
    }
    if (dX) {
      if (!dense) e = launch_decompress(h.row_values(v0), h.row_meta(v0), n, h.K, h.n, h.m, wd, ldk, s, true);  // beside G's launch
      if (e != cudaSuccess) return cuda_fail(e, "decompress launch");
      st = dense_t_accumulate(wd, ldk, n, h.K, g, ldg, tokens, acc, lda, ranges, v0 > 0, s);
      if (st != NM_OK) return st;
    }
    if (dV) {
      st = run_sddmm(h.row_meta(v0), h.n, h.m, n, h.K, nullptr, g, ldg, x, ldx, tokens,
                     dV + v0 * value_cols(h.K, h.n, h.m), NM_OUT_BF16, s, dX != nullptr, x_tokens);
      if (st != NM_OK) return st;
    }
  }
  if (dX) {
    const int64_t want = (h.K * ((h.T + 7) / 8) + 255) / 256, cap = (int64_t)sm_count_current() * 16;
    e = launch_pdl(xent_round_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, s,
                   (const float*)acc, ranges * terms, terms, width, lda, h.K, h.T, idx, dX, lddx);
    count_launch();
    if (e != cudaSuccess) return cuda_fail(e, "gradient rounding launch");
  }
  return NM_OK;
}

}  // namespace
}  // namespace nmk

using namespace nmk;

extern "C" {

nm_status nm_spmm_xent(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                       const int32_t* idx, const uint16_t* X, int64_t ldx, int64_t T, const int32_t* target,
                       float* loss, float* lse, void* stream) {
  set_last_error("");
  nm_status st = check_head(n, m, R, K, T);
  if (st != NM_OK || T == 0) return st;
  if (!values || !meta || !target || !loss || !lse) return fail(NM_ERR_INVALID_ARG, "null operand");
  if (!aligned_to(values, 2)) return fail(NM_ERR_MISALIGNED, "values misaligned");
  st = check_words({meta, idx, target, loss, lse}, "meta, idx, target, loss and lse");
  if (st == NM_OK) st = check_matrix(X, ldx, T, 2, "X");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  return run_xent(Head{values, meta, n, m, R, K, T, X, ldx}, idx, target, loss, lse,
                  static_cast<cudaStream_t>(stream));
}

nm_status nm_spmm_xent_grad(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                            const int32_t* idx, const uint16_t* X, int64_t ldx, int64_t T, const int32_t* target,
                            const float* lse, const float* dloss, uint16_t* dX, int64_t lddx, uint16_t* dV,
                            void* stream) {
  set_last_error("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  nm_status st = check_head(n, m, R, K, T);
  if (st != NM_OK) return st;
  if (!dX && !dV && T > 0) return fail(NM_ERR_INVALID_ARG, "dX and dV are both null");
  if (dV && !aligned_to(dV, 2)) return fail(NM_ERR_MISALIGNED, "dV misaligned");
  if (T == 0) {  // no tokens: dX has no elements, dV is an empty sum
    if (!dV) return NM_OK;
    st = require_device();
    if (st != NM_OK) return st;
    const int64_t vcols = value_cols(K, n, m);
    cudaError_t e = launch_fill_zero(dV, R, vcols, vcols, 2, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "zero fill");
  }
  if (!values || !meta || !target || !lse || !dloss) return fail(NM_ERR_INVALID_ARG, "null operand");
  if (!aligned_to(values, 2)) return fail(NM_ERR_MISALIGNED, "values misaligned");
  st = check_words({meta, idx, target, lse, dloss}, "meta, idx, target, lse and dloss");
  if (st == NM_OK) st = check_matrix(X, ldx, T, 2, "X");
  if (st == NM_OK && dX) st = check_matrix(dX, lddx, T, 2, "dX");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  return run_xent_grad(Head{values, meta, n, m, R, K, T, X, ldx}, idx, target, lse, dloss, dX, lddx, dV, s);
}

}  // extern "C"
