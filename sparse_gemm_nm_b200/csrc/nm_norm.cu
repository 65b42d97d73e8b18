// nm_norm.cu -- layer norm over the features of each token, forward and
// backward, in the K x T layout of the GEMMs (tokens contiguous).
//
// Forward, per token t:  mean = sum_k x / K, var = sum_k (x - mean)^2 / K,
//   rstd = 1 / sqrt(var + eps), y[k] = (x[k] - mean) rstd gamma[k] + beta[k].
// Backward, with xh = (x - mean) rstd and g = gamma dY:
//   dX = rstd (g - (sum_k g + xh sum_k g xh) / K),
//   dgamma[k] = sum_t dY xh,  dbeta[k] = sum_t dY.
//
// The reduction runs down the columns, so a tile is a strip of 8 * lpr tokens
// (lpr lanes of eight tokens each) by all K features, shared by the CTAs of
// one cluster: CTA c of a cluster of C takes a slab of K / C rows.  With few
// operations per byte the kernels are bound by memory, so the strip is read
// from HBM once: a CTA's slab comes into shared memory by TMA boxes, issued
// before anything else (past T and K they fill zeros, so ragged edges need no
// element loads), and the passes over it read shared memory.  The slab is kept
// to a quarter of the SM's shared memory where a cluster of eight allows it:
// the four CTAs of an SM are then in different phases, and loads, sums and
// stores overlap.  (Holding the rows in registers instead left one CTA per SM,
// 160 registers a thread: 105 us against the floor of 24 us on 768 x 50432.)
// Column sums go lanes -> warps -> CTA, and across the cluster through
// distributed shared memory, every addition in a fixed order.  The forward
// pass takes each CTA's own mean first and the squares about that, and joins
// the CTAs' (mean, squares) pairs: one cluster exchange, and no cancellation
// in the variance.  The backward pass writes each strip's row sums for dgamma
// and dbeta as partials, which norm_grad_reduce_kernel adds in strip order.
// A K too large for a cluster's shared memory reads the strip from global
// memory in every pass (CACHED = false).
#include <cstdint>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_norm.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace norm {
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCols = 64;  // tokens of a strip: eight lanes of eight
constexpr int kMaxCluster = 8;
constexpr int kBoxRows = 32;                     // rows of a TMA box (slabs are whole boxes)
constexpr int64_t kSlabBytes = 52 * 1024;        // four CTAs of an SM
constexpr int64_t kMaxSlabBytes = 216 * 1024;    // one CTA
constexpr uint64_t kWaitNs = 2000000000ull;

// Eight consecutive tokens of one row as held in registers.
template <bool F32>
struct Piece {
  uint4 v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Piece<F32> load_piece(const void* base, int64_t off, int valid) {
  Piece<F32> p;
  if (F32) {
    const float* s = static_cast<const float*>(base) + off;
    if (valid >= 8) {
      p.v[0] = __ldg(reinterpret_cast<const uint4*>(s));
      p.v[F32 ? 1 : 0] = __ldg(reinterpret_cast<const uint4*>(s) + 1);
    } else {  // the row's last tokens one by one, zeros after them
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < valid ? __float_as_uint(__ldg(s + j)) : 0u;
      p.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
      p.v[F32 ? 1 : 0] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(base) + off;
    if (valid >= 8) {
      p.v[0] = __ldg(reinterpret_cast<const uint4*>(s));
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) w[j >> 1] |= (uint32_t)__ldg(s + j) << (16 * (j & 1));
      p.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return p;
}

template <bool F32>
__device__ __forceinline__ void unpack(const Piece<F32>& p, float (&f)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p.v);
  if (F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[F32 ? j : 0]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// The same from shared memory (off in elements; whole pieces only).
template <bool F32>
__device__ __forceinline__ Piece<F32> shared_piece(const uint8_t* base, int64_t off) {
  Piece<F32> p;
  const uint4* s = reinterpret_cast<const uint4*>(base + off * (F32 ? 4 : 2));
  p.v[0] = s[0];
  if (F32) p.v[F32 ? 1 : 0] = s[1];
  return p;
}

__device__ __forceinline__ void store_piece(void* base, int64_t off, bool f32, int valid, const float (&f)[8]) {
  if (f32) {
    float* d = static_cast<float*>(base) + off;
    if (valid >= 8) {
      reinterpret_cast<float4*>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) d[j] = f[j];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(base) + off;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    if (valid >= 8) {
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// Sums of f over the threads of the CTA that hold the same eight tokens, left in out[token] (lpr * 8 values).
// All threads call it; out and scratch are shared memory, scratch kWarps x kMaxCols floats.
__device__ __forceinline__ void column_sums(float (&f)[8], int lpr, float* scratch, float* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int o = lpr; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += __shfl_xor_sync(0xFFFFFFFFu, f[j], o);
  }
  __syncthreads();  // earlier readers of scratch and out are done
  if (lane < lpr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) scratch[warp * kMaxCols + lane * 8 + j] = f[j];
  }
  __syncthreads();
  if ((int)threadIdx.x < lpr * 8) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += scratch[w * kMaxCols + threadIdx.x];
    out[threadIdx.x] = s;
  }
  __syncthreads();
}

__device__ __forceinline__ float ld_cluster(const float* local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(smem_u32(local), rank)) : "memory");
  return v;
}
// Brings `rows` rows from row r0 of a K x T tensor, columns t .. t + 8 lpr, into shared memory as rows of
// 8 lpr elements (boxes of kBoxRows rows; the last box may reach into rows of the next slab or past K).  The first
// lane of every warp calls it and issues its share of the boxes.
__device__ __forceinline__ void load_slab(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int64_t t, int64_t r0,
                                          int64_t boxes, uint32_t box_bytes) {
  for (int64_t b = threadIdx.x >> 5; b < boxes; b += kWarps)
    tma_load_2d(dst + b * box_bytes, tm, bar, (int32_t)t, (int32_t)(r0 + b * kBoxRows));
}
}  // namespace norm

template <bool XF32, bool CACHED>
__global__ void __launch_bounds__(norm::kThreads) norm_kernel(const __grid_constant__ NormParams p) {
  using namespace norm;
  extern __shared__ __align__(128) uint8_t slab[];
  __shared__ float scratch[kWarps * kMaxCols];
  __shared__ float s_mean[kMaxCols], s_m2[kMaxCols], s_rstd[kMaxCols], t_mean[kMaxCols];
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t tile = blockIdx.x / C;
  const int64_t r0 = rank * p.rows, r1 = r0 + p.rows < p.K ? r0 + p.rows : p.K;
  const int64_t mine = r1 > r0 ? r1 - r0 : 0;
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int64_t first = r0 + threadIdx.x / lpr;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);
  if (CACHED && threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (CACHED) __syncthreads();
  pdl_gate();
  bool ok = true;
  if (CACHED) {
    const int64_t boxes = (mine + kBoxRows - 1) / kBoxRows;
    const uint32_t box_bytes = (uint32_t)(kBoxRows * 8 * lpr) * (XF32 ? 4u : 2u);
    if (threadIdx.x % 32 == 0 && boxes > 0) {
      if (threadIdx.x == 0) mbar_arrive_expect_tx(&bar, (uint32_t)boxes * box_bytes);
      load_slab(slab, &p.tm_x, &bar, tile * (8 * lpr), r0, boxes, box_bytes);
    }
    if (boxes > 0) ok = mbar_wait(&bar, 0, &abort_flag, p.status, kWaitNs);
  }
  // Row k's piece of this thread's eight tokens (zeros past T).
  auto row = [&](int64_t k) {
    if (CACHED) return shared_piece<XF32>(slab, (k - r0) * (8 * lpr) + 8 * col8);
    return load_piece<XF32>(p.X, k * p.ldx + t0, valid);
  };

  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int64_t k = first; k < r1; k += step) {
    float f[8];
    unpack<XF32>(row(k), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += f[j];
  }
  column_sums(sum, lpr, scratch, s_mean);
  if ((int)threadIdx.x < lpr * 8) s_mean[threadIdx.x] = mine > 0 ? s_mean[threadIdx.x] / (float)mine : 0.f;
  __syncthreads();
  float m[8], sq[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = s_mean[8 * col8 + j];
#pragma unroll 4
  for (int64_t k = first; k < r1; k += step) {
    float f[8];
    unpack<XF32>(row(k), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[j] += (f[j] - m[j]) * (f[j] - m[j]);
  }
  column_sums(sq, lpr, scratch, s_m2);
  if (C > 1) cluster_sync();  // every CTA's s_mean and s_m2 are written
  if ((int)threadIdx.x < lpr * 8) {
    float mean = 0.f, m2 = 0.f;
    if (C > 1) {
      for (int c = 0; c < C; ++c) {
        const int64_t a = c * p.rows, n = a + p.rows < p.K ? p.rows : (p.K > a ? p.K - a : 0);
        mean += ld_cluster(s_mean + threadIdx.x, c) * ((float)n / (float)p.K);
      }
      for (int c = 0; c < C; ++c) {
        const int64_t a = c * p.rows, n = a + p.rows < p.K ? p.rows : (p.K > a ? p.K - a : 0);
        const float d = ld_cluster(s_mean + threadIdx.x, c) - mean;
        m2 += ld_cluster(s_m2 + threadIdx.x, c) + (float)n * d * d;
      }
    } else {
      mean = s_mean[threadIdx.x];
      m2 = s_m2[threadIdx.x];
    }
    const float rstd = 1.0f / sqrtf(m2 / (float)p.K + p.eps);
    t_mean[threadIdx.x] = mean;
    s_rstd[threadIdx.x] = rstd;
    const int64_t t = tile * (8 * lpr) + threadIdx.x;
    if (ok && rank == 0 && t < p.T) {
      if (p.mean) p.mean[t] = mean;
      if (p.rstd) p.rstd[t] = rstd;
    }
  }
  __syncthreads();
  float rs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = t_mean[8 * col8 + j];
    rs[j] = s_rstd[8 * col8 + j];
  }
  if (ok && valid > 0) {
#pragma unroll 4
    for (int64_t k = first; k < r1; k += step) {
      float f[8];
      unpack<XF32>(row(k), f);
      const float g = p.gamma ? __ldg(p.gamma + k) : 1.f, b = p.beta ? __ldg(p.beta + k) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (f[j] - m[j]) * rs[j] * g + b;
      store_piece(p.Y, k * p.ldy + t0, p.y_f32 != 0, valid, f);
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another still reads its shared memory
}

template <bool XF32, bool DF32, bool CACHED>
__global__ void __launch_bounds__(norm::kThreads) norm_grad_kernel(const __grid_constant__ NormParams p) {
  using namespace norm;
  extern __shared__ __align__(128) uint8_t slab[];  // X's rows, then dY's
  __shared__ float scratch[kWarps * kMaxCols];
  __shared__ float s_c1[kMaxCols], s_c2[kMaxCols], t_c1[kMaxCols], t_c2[kMaxCols];
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t tile = blockIdx.x / C;
  const int64_t r0 = rank * p.rows, r1 = r0 + p.rows < p.K ? r0 + p.rows : p.K;
  const int64_t mine = r1 > r0 ? r1 - r0 : 0;
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int64_t first = r0 + threadIdx.x / lpr;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);
  if (CACHED && threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (CACHED) __syncthreads();
  pdl_gate();
  const int64_t boxes = (mine + kBoxRows - 1) / kBoxRows;
  const uint32_t x_box = (uint32_t)(kBoxRows * 8 * lpr) * (XF32 ? 4u : 2u);
  const uint32_t d_box = (uint32_t)(kBoxRows * 8 * lpr) * (DF32 ? 4u : 2u);
  const uint8_t* d_slab = slab + boxes * x_box;
  bool ok = true;
  if (CACHED && threadIdx.x % 32 == 0 && boxes > 0) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&bar, (uint32_t)boxes * (x_box + d_box));
    load_slab(slab, &p.tm_x, &bar, tile * (8 * lpr), r0, boxes, x_box);
    load_slab(slab + boxes * x_box, &p.tm_d, &bar, tile * (8 * lpr), r0, boxes, d_box);
  }
  float mean[8], rs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mean[j] = j < valid ? __ldg(p.mean + t0 + j) : 0.f;
    rs[j] = j < valid ? __ldg(p.rstd + t0 + j) : 0.f;
  }
  if (CACHED && boxes > 0) ok = mbar_wait(&bar, 0, &abort_flag, p.status, kWaitNs);
  auto x_row = [&](int64_t k) {
    if (CACHED) return shared_piece<XF32>(slab, (k - r0) * (8 * lpr) + 8 * col8);
    return load_piece<XF32>(p.X, k * p.ldx + t0, valid);
  };
  auto d_row = [&](int64_t k) {
    if (CACHED) return shared_piece<DF32>(d_slab, (k - r0) * (8 * lpr) + 8 * col8);
    return load_piece<DF32>(p.dY, k * p.ldy + t0, valid);
  };

  float c1[8] = {0, 0, 0, 0, 0, 0, 0, 0}, c2[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int64_t trips = (mine + step - 1) / step;  // the same for every thread: the row sums shuffle
#pragma unroll 2
  for (int64_t i = 0; i < trips; ++i) {
    const int64_t k = first + i * step;
    float dg = 0.f, db = 0.f;
    if (k < r1) {
      float f[8], e[8];
      unpack<XF32>(x_row(k), f);
      unpack<DF32>(d_row(k), e);
      const float g = p.gamma ? __ldg(p.gamma + k) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = (f[j] - mean[j]) * rs[j];  // 0 past T: rs is 0 there
        c1[j] += g * e[j];
        c2[j] += g * e[j] * h;
        dg += e[j] * h;
        db += e[j];
      }
    }
    if (p.part) {
      for (int o = lpr >> 1; o > 0; o >>= 1) {
        dg += __shfl_xor_sync(0xFFFFFFFFu, dg, o);
        db += __shfl_xor_sync(0xFFFFFFFFu, db, o);
      }
      if (ok && col8 == 0 && k < r1) {
        p.part[tile * 2 * p.K + k] = dg;
        p.part[tile * 2 * p.K + p.K + k] = db;
      }
    }
  }
  column_sums(c1, lpr, scratch, s_c1);
  column_sums(c2, lpr, scratch, s_c2);
  if (C > 1) cluster_sync();
  if ((int)threadIdx.x < lpr * 8) {
    float a = 0.f, b = 0.f;
    if (C > 1) {
      for (int c = 0; c < C; ++c) {
        a += ld_cluster(s_c1 + threadIdx.x, c);
        b += ld_cluster(s_c2 + threadIdx.x, c);
      }
    } else {
      a = s_c1[threadIdx.x];
      b = s_c2[threadIdx.x];
    }
    t_c1[threadIdx.x] = a / (float)p.K;
    t_c2[threadIdx.x] = b / (float)p.K;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c1[j] = t_c1[8 * col8 + j];
    c2[j] = t_c2[8 * col8 + j];
  }
  if (ok && valid > 0) {
#pragma unroll 2
    for (int64_t k = first; k < r1; k += step) {
      float f[8], e[8];
      unpack<XF32>(x_row(k), f);
      unpack<DF32>(d_row(k), e);
      const float g = p.gamma ? __ldg(p.gamma + k) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = (f[j] - mean[j]) * rs[j];
        f[j] = rs[j] * (g * e[j] - (c1[j] + h * c2[j]));
      }
      store_piece(p.Y, k * p.ldo + t0, XF32, valid, f);
    }
  }
  if (C > 1) cluster_sync();
}

// dgamma[k] and dbeta[k]: the strips' partials added in strip order (a fixed
// split of the strips over 32 warps, then the warps in order).  One block per
// 32 features of one of the two outputs.
__global__ void __launch_bounds__(1024) norm_grad_reduce_kernel(const float* part, int64_t tiles, int64_t K,
                                                                float* dgamma, float* dbeta) {
  __shared__ float s[32][33];
  pdl_gate();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = (int64_t)blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float a = 0.f;
  if (k < K) {
    const float* src = part + (blockIdx.y ? K : 0) + k;
#pragma unroll 8
    for (int64_t t = warp; t < tiles; t += 32) a += __ldcg(src + t * 2 * K);
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && k < K) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += s[w][lane];
    out[k] = v;
  }
}

// Strip width, cluster size and rows per CTA, from the bytes of one row element (X, and dY in the backward
// pass).  The widest strip (64 tokens: whole 128-byte lines of bf16) whose slab fits a quarter of an SM in a cluster of
// eight; for larger K strips of 16 tokens (whole 32-byte sectors) that fit at all, then of 8; past that nothing is cached.  Then
// the smallest cluster that keeps the slab there, enlarged while the grid leaves SMs idle.
void norm_shape(NormParams& p, int64_t bytes) {
  using namespace norm;
  auto slab = [&](int l, int c) {
    const int64_t rows = (p.K + c - 1) / c;
    return (rows + kBoxRows - 1) / kBoxRows * kBoxRows * 8 * l * bytes;
  };
  int widest = 8;
  while (widest > 1 && (int64_t)(widest / 2) * 8 >= p.T) widest >>= 1;
  int lpr = widest;
  int64_t limit = kSlabBytes;
  while (lpr > 2 && slab(lpr, kMaxCluster) > limit) lpr >>= 1;
  if (slab(lpr, kMaxCluster) > limit) limit = kMaxSlabBytes;
  if (slab(lpr, kMaxCluster) > limit) lpr = 1;
  p.cached = slab(lpr, kMaxCluster) <= limit;
  int c = 1;
  while (c < kMaxCluster && slab(lpr, c) > limit) c <<= 1;
  p.tiles = (p.T + 8 * lpr - 1) / (8 * lpr);
  while (c < kMaxCluster && p.tiles * c < 2 * (int64_t)sm_count_current() && p.K / c > kThreads / lpr) c <<= 1;
  p.lpr = lpr;
  p.cluster = c;
  p.rows = (p.K + c - 1) / c;
  p.smem = p.cached ? (uint32_t)slab(lpr, c) : 0;
}

template <auto Kern>
static cudaError_t launch_norm_grid(const NormParams& p, cudaStream_t s) {
  if (p.tiles * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.raise(Kern, (uint32_t)norm::kMaxSlabBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles * p.cluster));
  cfg.blockDim = dim3(norm::kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, Kern, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.x_f32)
    return p.cached ? launch_norm_grid<&norm_kernel<true, true>>(p, s) : launch_norm_grid<&norm_kernel<true, false>>(p, s);
  return p.cached ? launch_norm_grid<&norm_kernel<false, true>>(p, s) : launch_norm_grid<&norm_kernel<false, false>>(p, s);
}

template <bool XF32, bool DF32>
static cudaError_t launch_norm_grad_types(const NormParams& p, cudaStream_t s) {
  return p.cached ? launch_norm_grid<&norm_grad_kernel<XF32, DF32, true>>(p, s)
                  : launch_norm_grid<&norm_grad_kernel<XF32, DF32, false>>(p, s);
}

cudaError_t launch_norm_grad(const NormParams& p, cudaStream_t s) {
  if (p.x_f32) return p.y_f32 ? launch_norm_grad_types<true, true>(p, s) : launch_norm_grad_types<true, false>(p, s);
  return p.y_f32 ? launch_norm_grad_types<false, true>(p, s) : launch_norm_grad_types<false, false>(p, s);
}

cudaError_t launch_norm_grad_reduce(const float* part, int64_t tiles, int64_t K, float* dgamma, float* dbeta,
                                    cudaStream_t s) {
  cudaError_t e = launch_pdl(norm_grad_reduce_kernel, dim3((unsigned)((K + 31) / 32), 2), dim3(1024), 0, s, part,
                             tiles, K, dgamma, dbeta);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace nmk

using namespace nmk;

// Map of a K x T tensor in boxes of kBoxRows rows of one strip.
static nm_status norm_map(CUtensorMap* tm, const void* base, int64_t K, int64_t T, int64_t ld, nm_out_dtype dtype,
                          int lpr, const char* what) {
  const bool f32 = dtype == NM_OUT_F32;
  return make_tmap(tm, base, (uint64_t)T, (uint64_t)K, (uint64_t)(ld * dtype_bytes(dtype)), 8u * (uint32_t)lpr,
                   (uint32_t)norm::kBoxRows, 0, what,
                   f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

extern "C" {

nm_status nm_layer_norm(const void* X, int64_t ldx, nm_out_dtype x_dtype, int64_t K, int64_t T, const float* gamma,
                        const float* beta, float eps, void* Y, int64_t ldy, nm_out_dtype y_dtype, float* mean,
                        float* rstd, void* stream) {
  set_last_error("");
  if (K < 0 || T < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (K == 0) return fail(NM_ERR_INVALID_ARG, "K is 0: the mean of no features is undefined");
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return fail(NM_ERR_INVALID_ARG, "bad dtype");
  if (!(eps >= 0.f && eps < 3.0e38f)) return fail(NM_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (K >= kMaxDim || T >= kMaxDim) return fail(NM_ERR_UNSUPPORTED, "dimensions must stay below 2^31");
  if (T == 0) return NM_OK;
  nm_status st = check_matrix(X, ldx, T, dtype_bytes(x_dtype), "X");
  if (st == NM_OK) st = check_matrix(Y, ldy, T, dtype_bytes(y_dtype), "Y");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  NormParams p = {};
  p.X = X;
  p.ldx = ldx;
  p.x_f32 = x_dtype == NM_OUT_F32;
  p.Y = Y;
  p.ldy = ldy;
  p.y_f32 = y_dtype == NM_OUT_F32;
  p.K = K;
  p.T = T;
  p.gamma = gamma;
  p.beta = beta;
  p.eps = eps;
  p.mean = mean;
  p.rstd = rstd;
  norm_shape(p, dtype_bytes(x_dtype));
  if (p.cached) st = norm_map(&p.tm_x, X, K, T, ldx, x_dtype, p.lpr, "X");
  if (st != NM_OK) return st;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  cudaError_t e = launch_norm(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "layer norm launch");
}

nm_status nm_layer_norm_grad(const void* dY, int64_t lddy, nm_out_dtype dy_dtype, const void* X, int64_t ldx,
                             nm_out_dtype x_dtype, int64_t K, int64_t T, const float* gamma, const float* mean,
                             const float* rstd, void* dX, int64_t lddx, float* dgamma, float* dbeta, void* stream) {
  set_last_error("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K < 0 || T < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (K == 0) return fail(NM_ERR_INVALID_ARG, "K is 0: the mean of no features is undefined");
  if (!dtype_ok(x_dtype) || !dtype_ok(dy_dtype)) return fail(NM_ERR_INVALID_ARG, "bad dtype");
  if (K >= kMaxDim || T >= kMaxDim) return fail(NM_ERR_UNSUPPORTED, "dimensions must stay below 2^31");
  if (T == 0) {  // empty sums
    if (!dgamma && !dbeta) return NM_OK;
    nm_status st = require_device();
    if (st != NM_OK) return st;
    cudaError_t e = launch_norm_grad_reduce(nullptr, 0, K, dgamma, dbeta, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "layer norm gradient reduction launch");
  }
  nm_status st = check_matrix(dY, lddy, T, dtype_bytes(dy_dtype), "dY");
  if (st == NM_OK) st = check_matrix(X, ldx, T, dtype_bytes(x_dtype), "X");
  if (st == NM_OK) st = check_matrix(dX, lddx, T, dtype_bytes(x_dtype), "dX");
  if (st == NM_OK && (!mean || !rstd)) st = fail(NM_ERR_INVALID_ARG, "mean or rstd is null");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  NormParams p = {};
  p.X = X;
  p.ldx = ldx;
  p.x_f32 = x_dtype == NM_OUT_F32;
  p.dY = dY;
  p.ldy = lddy;
  p.y_f32 = dy_dtype == NM_OUT_F32;
  p.Y = dX;
  p.ldo = lddx;
  p.K = K;
  p.T = T;
  p.gamma = gamma;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  norm_shape(p, dtype_bytes(x_dtype) + dtype_bytes(dy_dtype));
  if (p.cached) st = norm_map(&p.tm_x, X, K, T, ldx, x_dtype, p.lpr, "X");
  if (p.cached && st == NM_OK) st = norm_map(&p.tm_d, dY, K, T, lddy, dy_dtype, p.lpr, "dY");
  if (st != NM_OK) return st;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  Staged part(s);
  if (dgamma || dbeta) {
    cudaError_t e = part.get((size_t)p.tiles * 2 * (size_t)K * 4);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the row sums");
    p.part = part.as<float>();
  }
  cudaError_t e = launch_norm_grad(p, s);
  if (e != cudaSuccess) return cuda_fail(e, "layer norm gradient launch");
  if (p.part) e = launch_norm_grad_reduce(p.part, p.tiles, K, dgamma, dbeta, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "layer norm gradient reduction launch");
}

}  // extern "C"
