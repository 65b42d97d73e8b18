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
// one cluster: CTA c of a cluster of C takes a slab of K / C rows.  Every
// thread keeps its rows' 16-byte pieces in registers (RPT rows), so the strip
// is read from HBM once: with few operations per byte the kernels are bound by
// memory, and all of a CTA's loads are in flight before the first sum.  Column
// sums go lanes -> warps -> CTA, and across the cluster through distributed
// shared memory, every addition in a fixed order.  The forward pass takes each
// CTA's own mean first and the squares about that, and joins the CTAs' (mean,
// squares) pairs: one cluster exchange, and no cancellation in the variance.
// The backward pass writes each strip's row sums for dgamma and dbeta as
// partials, which norm_grad_reduce_kernel adds in strip order.  K too large
// for the registers of a cluster of eight reads the strip again for each pass
// (RPT = 0).
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

// Keeps a bf16 piece in its packed form between passes: without this the compiler holds the unpacked floats of
// every row across the column sums, twice the registers (227 instead of about 120 at 16 rows).
template <bool F32>
__device__ __forceinline__ void keep_packed(Piece<F32>& p) {
  if (!F32) asm volatile("" : "+r"(p.v[0].x), "+r"(p.v[0].y), "+r"(p.v[0].z), "+r"(p.v[0].w));
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
}  // namespace norm

template <bool XF32, int RPT>
__global__ void __launch_bounds__(norm::kThreads) norm_kernel(const NormParams p) {
  using namespace norm;
  __shared__ float scratch[kWarps * kMaxCols];
  __shared__ float s_mean[kMaxCols], s_m2[kMaxCols], s_rstd[kMaxCols], t_mean[kMaxCols];
  pdl_gate();
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t tile = blockIdx.x / C;
  const int64_t rows = (p.K + C - 1) / C;
  const int64_t r0 = rank * rows, r1 = r0 + rows < p.K ? r0 + rows : p.K;
  const int64_t mine = r1 > r0 ? r1 - r0 : 0;
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int64_t first = r0 + threadIdx.x / lpr;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);

  Piece<XF32> x[RPT > 0 ? RPT : 1];
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (RPT > 0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t k = first + (int64_t)i * step;
      x[i] = load_piece<XF32>(p.X, k * p.ldx + t0, k < r1 ? valid : 0);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float f[8];
      unpack<XF32>(x[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      keep_packed<XF32>(x[i]);
    }
  } else {
    for (int64_t k = first; k < r1; k += step) {
      float f[8];
      unpack<XF32>(load_piece<XF32>(p.X, k * p.ldx + t0, valid), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
    }
  }
  column_sums(sum, lpr, scratch, s_mean);
  if ((int)threadIdx.x < lpr * 8) s_mean[threadIdx.x] = mine > 0 ? s_mean[threadIdx.x] / (float)mine : 0.f;
  __syncthreads();
  float m[8], sq[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = s_mean[8 * col8 + j];
  if (RPT > 0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      if (first + (int64_t)i * step >= r1) continue;
      float f[8];
      unpack<XF32>(x[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[j] += (f[j] - m[j]) * (f[j] - m[j]);
      keep_packed<XF32>(x[i]);
    }
  } else {
    for (int64_t k = first; k < r1; k += step) {
      float f[8];
      unpack<XF32>(load_piece<XF32>(p.X, k * p.ldx + t0, valid), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[j] += (f[j] - m[j]) * (f[j] - m[j]);
    }
  }
  column_sums(sq, lpr, scratch, s_m2);
  if (C > 1) cluster_sync();  // every CTA's s_mean and s_m2 are written
  if ((int)threadIdx.x < lpr * 8) {
    float mean = 0.f, m2 = 0.f;
    if (C > 1) {
      for (int c = 0; c < C; ++c) {
        const int64_t a = c * rows, n = a + rows < p.K ? rows : (p.K > a ? p.K - a : 0);
        mean += ld_cluster(s_mean + threadIdx.x, c) * ((float)n / (float)p.K);
      }
      for (int c = 0; c < C; ++c) {
        const int64_t a = c * rows, n = a + rows < p.K ? rows : (p.K > a ? p.K - a : 0);
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
    if (rank == 0 && t < p.T) {
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
  auto write_row = [&](int64_t k, const Piece<XF32>& piece) {
    float f[8];
    unpack<XF32>(piece, f);
    const float g = p.gamma ? __ldg(p.gamma + k) : 1.f, b = p.beta ? __ldg(p.beta + k) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (f[j] - m[j]) * rs[j] * g + b;
    store_piece(p.Y, k * p.ldy + t0, p.y_f32 != 0, valid, f);
  };
  if (RPT > 0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t k = first + (int64_t)i * step;
      if (k < r1 && valid > 0) write_row(k, x[i]);
    }
  } else if (valid > 0) {
    for (int64_t k = first; k < r1; k += step) write_row(k, load_piece<XF32>(p.X, k * p.ldx + t0, valid));
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another still reads its shared memory
}

template <bool XF32, bool DF32, int RPT>
__global__ void __launch_bounds__(norm::kThreads) norm_grad_kernel(const NormParams p) {
  using namespace norm;
  __shared__ float scratch[kWarps * kMaxCols];
  __shared__ float s_c1[kMaxCols], s_c2[kMaxCols], t_c1[kMaxCols], t_c2[kMaxCols];
  pdl_gate();
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t tile = blockIdx.x / C;
  const int64_t rows = (p.K + C - 1) / C;
  const int64_t r0 = rank * rows, r1 = r0 + rows < p.K ? r0 + rows : p.K;
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int64_t first = r0 + threadIdx.x / lpr;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);

  float mean[8], rs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mean[j] = j < valid ? __ldg(p.mean + t0 + j) : 0.f;
    rs[j] = j < valid ? __ldg(p.rstd + t0 + j) : 0.f;
  }
  Piece<XF32> x[RPT > 0 ? RPT : 1];
  Piece<DF32> d[RPT > 0 ? RPT : 1];
  float c1[8] = {0, 0, 0, 0, 0, 0, 0, 0}, c2[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  auto add_row = [&](int64_t k, const Piece<XF32>& xp, const Piece<DF32>& dp) {
    float f[8], e[8];
    unpack<XF32>(xp, f);
    unpack<DF32>(dp, e);
    const float g = p.gamma && k < r1 ? __ldg(p.gamma + k) : 1.f;
    float dg = 0.f, db = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float h = (f[j] - mean[j]) * rs[j];  // 0 past T: rs is 0 there
      c1[j] += g * e[j];
      c2[j] += g * e[j] * h;
      dg += e[j] * h;
      db += e[j];
    }
    if (p.part) {
      for (int o = lpr >> 1; o > 0; o >>= 1) {
        dg += __shfl_xor_sync(0xFFFFFFFFu, dg, o);
        db += __shfl_xor_sync(0xFFFFFFFFu, db, o);
      }
      if (col8 == 0 && k < r1) {
        p.part[tile * 2 * p.K + k] = dg;
        p.part[tile * 2 * p.K + p.K + k] = db;
      }
    }
  };
  if (RPT > 0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t k = first + (int64_t)i * step;
      x[i] = load_piece<XF32>(p.X, k * p.ldx + t0, k < r1 ? valid : 0);
      d[i] = load_piece<DF32>(p.dY, k * p.ldy + t0, k < r1 ? valid : 0);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      add_row(first + (int64_t)i * step, x[i], d[i]);
      keep_packed<XF32>(x[i]);
      keep_packed<DF32>(d[i]);
    }
  } else {
    const int64_t trips = r1 > r0 ? (r1 - r0 + step - 1) / step : 0;  // the same for every lane: add_row shuffles
    for (int64_t i = 0; i < trips; ++i) {
      const int64_t k = first + i * step;
      add_row(k, load_piece<XF32>(p.X, k * p.ldx + t0, k < r1 ? valid : 0),
              load_piece<DF32>(p.dY, k * p.ldy + t0, k < r1 ? valid : 0));
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
  auto write_row = [&](int64_t k, const Piece<XF32>& xp, const Piece<DF32>& dp) {
    float f[8], e[8];
    unpack<XF32>(xp, f);
    unpack<DF32>(dp, e);
    const float g = p.gamma ? __ldg(p.gamma + k) : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float h = (f[j] - mean[j]) * rs[j];
      f[j] = rs[j] * (g * e[j] - (c1[j] + h * c2[j]));
    }
    store_piece(p.Y, k * p.ldo + t0, XF32, valid, f);
  };
  if (RPT > 0) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t k = first + (int64_t)i * step;
      if (k < r1 && valid > 0) write_row(k, x[i], d[i]);
    }
  } else if (valid > 0) {
    for (int64_t k = first; k < r1; k += step)
      write_row(k, load_piece<XF32>(p.X, k * p.ldx + t0, valid), load_piece<DF32>(p.dY, k * p.ldy + t0, valid));
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

// Strip width, cluster size and rows per thread.  Strips of 64 tokens (whole
// 128-byte lines of bf16) while a cluster of eight holds K rows of them in
// registers, narrower ones for larger K or few tokens; then the smallest
// cluster that holds the strip, enlarged while the grid leaves SMs idle.
static void norm_shape(NormParams& p, int max_rpt, int* rpt) {
  int lpr = 8;
  while (lpr > 1 && (int64_t)(lpr / 2) * 8 >= p.T) lpr >>= 1;
  auto need = [&](int l, int c) {
    const int64_t rows = (p.K + c - 1) / c, step = norm::kThreads / l;
    return (rows + step - 1) / step;
  };
  while (lpr > 1 && need(lpr, norm::kMaxCluster) > max_rpt) lpr >>= 1;
  int c = 1;
  while (c < norm::kMaxCluster && need(lpr, c) > max_rpt) c <<= 1;
  const int64_t tiles = (p.T + 8 * lpr - 1) / (8 * lpr);
  while (c < norm::kMaxCluster && tiles * c < 2 * (int64_t)sm_count_current() && need(lpr, c) > 1) c <<= 1;
  const int64_t n = need(lpr, c);
  p.lpr = lpr;
  p.cluster = c;
  p.tiles = tiles;
  *rpt = n > max_rpt ? 0 : (int)n;
}

void norm_grad_shape(NormParams& p, int* rpt) { norm_shape(p, (p.x_f32 || p.y_f32) ? 8 : 16, rpt); }

template <typename Kern>
static cudaError_t launch_norm_grid(Kern kernel, const NormParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles * p.cluster));
  cfg.blockDim = dim3(norm::kThreads);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool XF32>
static cudaError_t norm_rpt(const NormParams& p, int rpt, cudaStream_t s) {
  if (rpt == 0) return launch_norm_grid(norm_kernel<XF32, 0>, p, s);
  if (rpt <= 2) return launch_norm_grid(norm_kernel<XF32, 2>, p, s);
  if (rpt <= 4) return launch_norm_grid(norm_kernel<XF32, 4>, p, s);
  if (rpt <= 8) return launch_norm_grid(norm_kernel<XF32, 8>, p, s);
  return launch_norm_grid(norm_kernel<XF32, 16>, p, s);
}

template <bool XF32, bool DF32>
static cudaError_t norm_grad_rpt(const NormParams& p, int rpt, cudaStream_t s) {
  if (rpt == 0) return launch_norm_grid(norm_grad_kernel<XF32, DF32, 0>, p, s);
  if (rpt <= 2) return launch_norm_grid(norm_grad_kernel<XF32, DF32, 2>, p, s);
  if (rpt <= 4) return launch_norm_grid(norm_grad_kernel<XF32, DF32, 4>, p, s);
  if (rpt <= 8) return launch_norm_grid(norm_grad_kernel<XF32, DF32, 8>, p, s);
  if (!XF32 && !DF32) return launch_norm_grid(norm_grad_kernel<false, false, 16>, p, s);
  return cudaErrorInvalidValue;  // norm_grad_shape keeps four-byte operands at eight rows
}

cudaError_t launch_norm(NormParams& p, cudaStream_t s) {
  int rpt = 0;
  norm_shape(p, 16, &rpt);
  if (p.tiles * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  return p.x_f32 ? norm_rpt<true>(p, rpt, s) : norm_rpt<false>(p, rpt, s);
}

cudaError_t launch_norm_grad(NormParams& p, int rpt, cudaStream_t s) {
  if (p.tiles * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  if (p.x_f32) return p.y_f32 ? norm_grad_rpt<true, true>(p, rpt, s) : norm_grad_rpt<true, false>(p, rpt, s);
  return p.y_f32 ? norm_grad_rpt<false, true>(p, rpt, s) : norm_grad_rpt<false, false>(p, rpt, s);
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
  int rpt = 0;
  norm_grad_shape(p, &rpt);
  Staged part(s);
  if (dgamma || dbeta) {
    cudaError_t e = part.get((size_t)p.tiles * 2 * (size_t)K * 4);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the row sums");
    p.part = part.as<float>();
  }
  cudaError_t e = launch_norm_grad(p, rpt, s);
  if (e != cudaSuccess) return cuda_fail(e, "layer norm gradient launch");
  if (p.part) e = launch_norm_grad_reduce(p.part, p.tiles, K, dgamma, dbeta, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "layer norm gradient reduction launch");
}

}  // extern "C"
