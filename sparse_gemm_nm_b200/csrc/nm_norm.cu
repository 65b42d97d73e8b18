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
// element loads), and the passes over it read shared memory.  A slab takes at
// most half of the SM's shared memory where a cluster of eight allows it, so
// that one CTA loads while the other computes.  Arithmetic is in packed float32
// pairs.  768 x 50432 takes 35 us forward (floor 24 us) and 78 us backward
// (36 us), bound by a CTA's own phases (load, passes between barriers, store),
// which one other CTA of the SM covers: 39 and 45 % of the cycles issue.  Tried
// and slower: persistent clusters that fetch the next strip while they work on
// one (57 and 93 us), 512 threads a CTA (40 and 90 us), rows held in registers
// with one CTA to an SM (105 us forward).
// Column sums go lanes -> warps -> CTA, and across the cluster through
// distributed shared memory, every addition in a fixed order.  The forward
// pass takes each CTA's own mean first and the squares about that, and joins
// the CTAs' (mean, squares) pairs: one cluster exchange, and no cancellation
// in the variance.  The backward pass writes each strip's row sums for dgamma
// and dbeta as partials, which norm_grad_reduce_kernel adds in strip order.
// A K too large for a cluster's shared memory reads the strip from global
// memory in every pass (CACHED = false).
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_norm.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace norm {
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCols = 64;  // tokens of a strip, at most (eight lanes of eight)
constexpr int kMaxCluster = 8;
constexpr int64_t kSlabBytes = 104 * 1024;     // with gamma and beta: two CTAs to an SM
constexpr int64_t kMaxSlabBytes = 216 * 1024;  // one
constexpr uint64_t kWaitNs = 2000000000ull;

// Two float32 values, worked on by the packed float32 instructions (one issue for both).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Eight consecutive tokens of a row, as four pairs.
template <bool F32>
__device__ __forceinline__ void load_global(const void* base, int64_t off, int valid, F2 (&f)[4]) {
  if (F32) {
    const float* s = static_cast<const float*>(base) + off;
    if (valid >= 8) {
      const float4 a = *reinterpret_cast<const float4*>(s), b = *(reinterpret_cast<const float4*>(s) + 1);
      f[0] = f2(a.x, a.y);
      f[1] = f2(a.z, a.w);
      f[2] = f2(b.x, b.y);
      f[3] = f2(b.z, b.w);
    } else {  // the row's last tokens one by one, zeros after them
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = f2(2 * j < valid ? s[2 * j] : 0.f, 2 * j + 1 < valid ? s[2 * j + 1] : 0.f);
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(base) + off;
    uint32_t w[4] = {0, 0, 0, 0};
    if (valid >= 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(s);
      w[0] = a.x;
      w[1] = a.y;
      w[2] = a.z;
      w[3] = a.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) w[j >> 1] |= (uint32_t)s[j] << (16 * (j & 1));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
}

// The same from shared memory (whole pieces; zeros past T and K were filled in).
template <bool F32>
__device__ __forceinline__ void load_shared(const uint8_t* at, F2 (&f)[4]) {
  if (F32) {
    const float4 a = *reinterpret_cast<const float4*>(at), b = *(reinterpret_cast<const float4*>(at) + 1);
    f[0] = f2(a.x, a.y);
    f[1] = f2(a.z, a.w);
    f[2] = f2(b.x, b.y);
    f[3] = f2(b.z, b.w);
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
}

// Eight tokens to global memory: WHOLE, or the first `valid` of them one by one.
template <bool F32, bool WHOLE>
__device__ __forceinline__ void store_piece(uint8_t* at, int valid, const F2 (&p)[4]) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) split(p[j], f[2 * j], f[2 * j + 1]);
  if (F32) {
    float* d = reinterpret_cast<float*>(at);
    if (WHOLE) {
      reinterpret_cast<float4*>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) d[j] = f[j];
    }
  } else {
    uint16_t* d = reinterpret_cast<uint16_t*>(at);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    if (WHOLE) {
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// Sums of N quantities over the threads of the CTA that hold the same eight tokens, left in out[n][token].
// All threads call it; out and scratch are shared memory, scratch N x kWarps x kMaxCols floats.
template <int N>
__device__ __forceinline__ void column_sums(F2 (&q)[N][4], int lpr, float* scratch, float (*out)[kMaxCols]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float f[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) split(q[n][j], f[n][2 * j], f[n][2 * j + 1]);
  for (int o = lpr; o < 32; o <<= 1) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[n][j] += __shfl_xor_sync(0xFFFFFFFFu, f[n][j], o);
  }
  if (lane < lpr) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < 8; ++j) scratch[(n * kWarps + warp) * kMaxCols + lane * 8 + j] = f[n][j];
  }
  __syncthreads();
  const int n = threadIdx.x / kMaxCols, t = threadIdx.x % kMaxCols;
  if (n < N && t < lpr * 8) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += scratch[(n * kWarps + w) * kMaxCols + t];
    out[n][t] = s;
  }
  __syncthreads();
}

__device__ __forceinline__ float ld_cluster(const float* local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(smem_u32(local), rank)) : "memory");
  return v;
}
// The same place of every CTA of the cluster (0 past C): all reads in flight together.
__device__ __forceinline__ void ld_cluster_all(const float* local, int C, float (&v)[kMaxCluster]) {
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) v[c] = c < C ? ld_cluster(local, c) : 0.f;
}

// n rows, U of them at a time with nothing between their loads, then one by one: body(index of the first,
// integral_constant U or 1).
template <int U, typename Body>
__device__ __forceinline__ void each_row(int n, Body body) {
  int i = 0;
  for (; i + U <= n; i += U) body(i, std::integral_constant<int, U>());
  for (; i < n; ++i) body(i, std::integral_constant<int, 1>());
}

// Brings `rows` rows from row r0 of a K x T tensor, columns t .. t + 8 lpr, into shared memory as rows of
// 8 lpr elements (boxes of box_rows rows; the last box may reach into rows of the next slab or past K).  The first
// lane of every warp calls it and issues its share of the boxes.
__device__ __forceinline__ void load_slab(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int64_t t, int64_t r0,
                                          int64_t boxes, int box_rows, uint32_t box_bytes) {
  for (int64_t b = threadIdx.x >> 5; b < boxes; b += kWarps)
    tma_load_2d(dst + b * box_bytes, tm, bar, (int32_t)t, (int32_t)(r0 + b * box_rows));
}
}  // namespace norm

template <bool XF32, bool YF32, bool CACHED>
__global__ void __launch_bounds__(norm::kThreads, 2) norm_kernel(const __grid_constant__ NormParams p) {
  using namespace norm;
  extern __shared__ __align__(128) uint8_t smem[];  // the slab, then (gamma, beta) of every row
  __shared__ float scratch[kWarps * kMaxCols];
  __shared__ float s_mean[1][kMaxCols], s_m2[1][kMaxCols], s_rstd[kMaxCols], t_mean[kMaxCols];
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t r0 = rank * p.rows;
  const int mine = (int)(r0 < p.K ? (p.K - r0 < p.rows ? p.K - r0 : p.rows) : 0);  // rows of this CTA
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int first = threadIdx.x / lpr;
  const int n = first < mine ? (mine - first + step - 1) / step : 0;  // rows of this thread: first, + step, ...
  if (CACHED && threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_gate();
  bool ok = true;
  constexpr int kX = XF32 ? 32 : 16, kY = YF32 ? 32 : 16;  // bytes of eight tokens
  const int boxes = (mine + p.box_rows - 1) / p.box_rows;
  const uint32_t box_bytes = (uint32_t)(p.box_rows * lpr * kX);
  const int64_t tile = blockIdx.x / C;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);
  if (CACHED && threadIdx.x % 32 == 0 && boxes > 0) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&bar, (uint32_t)boxes * box_bytes);
    load_slab(smem, &p.tm_x, &bar, tile * (8 * lpr), r0, boxes, p.box_rows, box_bytes);
  }
  float2* s_affine = reinterpret_cast<float2*>(smem + p.slab);
  auto affine = [&](int k) {
    const float g = p.gamma ? __ldg(p.gamma + r0 + k) : 1.f, b = p.beta ? __ldg(p.beta + r0 + k) : 0.f;
    return make_float2(g, b);
  };
  if (CACHED)
    for (int k = threadIdx.x; k < mine; k += kThreads) s_affine[k] = affine(k);  // read after the first __syncthreads

  if (CACHED && boxes > 0) ok = mbar_wait(&bar, 0, &abort_flag, p.status, kWaitNs);
  const uint8_t* x_at = smem + (first * lpr + col8) * kX;
  constexpr int kXStep = kThreads * kX;  // bytes between this thread's rows
  // The i-th row of this thread: its eight tokens (zeros past T).
  auto row = [&](int i, F2 (&f)[4]) {
    if (CACHED)
      load_shared<XF32>(x_at + i * kXStep, f);
    else
      load_global<XF32>(p.X, (r0 + first + (int64_t)i * step) * p.ldx + t0, valid, f);
  };

  const F2 zero = f2(0.f, 0.f);
  F2 sum[1][4] = {{zero, zero, zero, zero}};
  each_row<4>(n, [&](int i, auto u) {
    constexpr int U = decltype(u)::value;
    F2 f[U][4];
#pragma unroll
    for (int r = 0; r < U; ++r) row(i + r, f[r]);
#pragma unroll
    for (int r = 0; r < U; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[0][j] = add2(sum[0][j], f[r][j]);
  });
  column_sums<1>(sum, lpr, scratch, s_mean);
  // this CTA's own mean, negated: the squares are taken about it
  const float per = mine > 0 ? 1.0f / (float)mine : 0.f;
  F2 m[4], sq[1][4] = {{zero, zero, zero, zero}};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    m[j] = f2(-(s_mean[0][8 * col8 + 2 * j] * per), -(s_mean[0][8 * col8 + 2 * j + 1] * per));
  each_row<4>(n, [&](int i, auto u) {
    constexpr int U = decltype(u)::value;
    F2 f[U][4];
#pragma unroll
    for (int r = 0; r < U; ++r) row(i + r, f[r]);
#pragma unroll
    for (int r = 0; r < U; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 d = add2(f[r][j], m[j]);
        sq[0][j] = fma2(d, d, sq[0][j]);
      }
  });
  column_sums<1>(sq, lpr, scratch, s_m2);
  if (C > 1) cluster_sync();  // every CTA's s_mean (sums) and s_m2 are written
  if ((int)threadIdx.x < lpr * 8) {
    float mean = s_mean[0][threadIdx.x] / (float)p.K, m2 = s_m2[0][threadIdx.x];
    if (C > 1) {
      float a[kMaxCluster], q[kMaxCluster];
      ld_cluster_all(&s_mean[0][threadIdx.x], C, a);
      ld_cluster_all(&s_m2[0][threadIdx.x], C, q);
      float total = 0.f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) total += a[c];
      mean = total / (float)p.K;
      m2 = 0.f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= C) continue;
        const int64_t at = c * p.rows;
        const float rows = (float)(at < p.K ? (p.K - at < p.rows ? p.K - at : p.rows) : 0);
        const float d = rows > 0.f ? a[c] * (1.0f / rows) - mean : 0.f;
        m2 += q[c] + rows * d * d;
      }
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
  if (C > 1) cluster_arrive();  // done with the other CTAs' sums
  __syncthreads();
  F2 rs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = f2(-t_mean[8 * col8 + 2 * j], -t_mean[8 * col8 + 2 * j + 1]);
    rs[j] = f2(s_rstd[8 * col8 + 2 * j], s_rstd[8 * col8 + 2 * j + 1]);
  }
  uint8_t* out = static_cast<uint8_t*>(p.Y) + ((r0 + first) * p.ldy + t0) * (kY / 8);
  const int64_t out_step = step * p.ldy * (kY / 8);
  auto write = [&](auto whole) {
    each_row<2>(n, [&](int i, auto u) {
      constexpr int U = decltype(u)::value;
      F2 f[U][4];
      float2 a[U];
#pragma unroll
      for (int r = 0; r < U; ++r) {
        a[r] = CACHED ? s_affine[first + (i + r) * step] : affine(first + (i + r) * step);
        row(i + r, f[r]);
      }
#pragma unroll
      for (int r = 0; r < U; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[r][j] = fma2(mul2(add2(f[r][j], m[j]), rs[j]), f2(a[r].x, a[r].x), f2(a[r].y, a[r].y));
        store_piece<YF32, decltype(whole)::value>(out, valid, f[r]);
        out += out_step;
      }
    });
  };
  if (ok && valid == 8)
    write(std::true_type());
  else if (ok && valid > 0)
    write(std::false_type());
  if (C > 1) cluster_wait();  // the other CTAs have read this one's sums
}

template <bool XF32, bool DF32, bool CACHED>
__global__ void __launch_bounds__(norm::kThreads, 2) norm_grad_kernel(const __grid_constant__ NormParams p) {
  using namespace norm;
  extern __shared__ __align__(128) uint8_t smem[];  // X's slab, dY's, then gamma of every row
  __shared__ float scratch[2 * kWarps * kMaxCols];
  __shared__ float s_c[2][kMaxCols], t_c[2][kMaxCols];
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster, lpr = p.lpr;
  const int64_t r0 = rank * p.rows;
  const int mine = (int)(r0 < p.K ? (p.K - r0 < p.rows ? p.K - r0 : p.rows) : 0);  // rows of this CTA
  const int col8 = threadIdx.x % lpr;
  const int step = kThreads / lpr;
  const int first = threadIdx.x / lpr;
  const int n = first < mine ? (mine - first + step - 1) / step : 0;  // rows of this thread: first, + step, ...
  const int turns = (mine + step - 1) / step;                         // of any thread, at most
  if (CACHED && threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_gate();
  constexpr int kX = XF32 ? 32 : 16, kD = DF32 ? 32 : 16;  // bytes of eight tokens
  const int boxes = (mine + p.box_rows - 1) / p.box_rows;
  const uint32_t x_box = (uint32_t)(p.box_rows * lpr * kX), d_box = (uint32_t)(p.box_rows * lpr * kD);
  bool ok = true;
  const int64_t tile = blockIdx.x / C;
  const int64_t t0 = tile * (8 * lpr) + 8 * col8;
  const int valid = t0 >= p.T ? 0 : (p.T - t0 < 8 ? (int)(p.T - t0) : 8);
  if (CACHED && threadIdx.x % 32 == 0 && boxes > 0) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&bar, (uint32_t)boxes * (x_box + d_box));
    load_slab(smem, &p.tm_x, &bar, tile * (8 * lpr), r0, boxes, p.box_rows, x_box);
    load_slab(smem + boxes * x_box, &p.tm_d, &bar, tile * (8 * lpr), r0, boxes, p.box_rows, d_box);
  }
  float* s_gamma = reinterpret_cast<float*>(smem + p.slab);
  auto gamma = [&](int k) { return p.gamma ? __ldg(p.gamma + r0 + k) : 1.f; };
  if (CACHED)
    for (int k = threadIdx.x; k < mine; k += kThreads) s_gamma[k] = gamma(k);
  __syncthreads();

  F2 mean[4], rs[4];  // the mean negated
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool a = 2 * j < valid, b = 2 * j + 1 < valid;
    mean[j] = f2(a ? -p.mean[t0 + 2 * j] : 0.f, b ? -p.mean[t0 + 2 * j + 1] : 0.f);
    rs[j] = f2(a ? p.rstd[t0 + 2 * j] : 0.f, b ? p.rstd[t0 + 2 * j + 1] : 0.f);
  }
  if (CACHED && boxes > 0) ok = mbar_wait(&bar, 0, &abort_flag, p.status, kWaitNs);
  const uint8_t* x_at = smem + (first * lpr + col8) * kX;
  const uint8_t* d_at = smem + boxes * x_box + (first * lpr + col8) * kD;
  auto rows = [&](int i, F2 (&f)[4], F2 (&e)[4]) {
    if (CACHED) {
      load_shared<XF32>(x_at + i * (kThreads * kX), f);
      load_shared<DF32>(d_at + i * (kThreads * kD), e);
    } else {
      const int64_t k = r0 + first + (int64_t)i * step;
      load_global<XF32>(p.X, k * p.ldx + t0, valid, f);
      load_global<DF32>(p.dY, k * p.ldy + t0, valid, e);
    }
  };

  const F2 zero = f2(0.f, 0.f);
  F2 c[2][4] = {{zero, zero, zero, zero}, {zero, zero, zero, zero}};
  // One row's terms of the column sums, and its own sums over the eight tokens.
  auto take = [&](const F2 (&f)[4], const F2 (&e)[4], float g, float& dg, float& db) {
    const F2 g2 = f2(g, g);
    F2 a = zero, b = zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const F2 h = mul2(add2(f[j], mean[j]), rs[j]);  // 0 past T: rs is 0 there
      const F2 ge = mul2(g2, e[j]);
      c[0][j] = add2(c[0][j], ge);
      c[1][j] = fma2(ge, h, c[1][j]);
      a = fma2(e[j], h, a);
      b = add2(b, e[j]);
    }
    float lo, hi;
    split(a, lo, hi);
    dg = lo + hi;
    split(b, lo, hi);
    db = lo + hi;
  };
  float* part = p.part + tile * 2 * p.K + r0;
  auto keep = [&](int i, float dg, float db) {  // the sums of row first + i * step; every lane takes part
    for (int o = lpr >> 1; o > 0; o >>= 1) {
      dg += __shfl_xor_sync(0xFFFFFFFFu, dg, o);
      db += __shfl_xor_sync(0xFFFFFFFFu, db, o);
    }
    if (col8 != 0 || i >= n) return;
    const int k = first + i * step;
    part[k] = dg;
    part[p.K + k] = db;
  };
  const bool sums = p.part != nullptr;
  // Turns taken two at a time: those in which every lane of the warp has its rows.
  const int both = CACHED && __all_sync(0xFFFFFFFFu, n == turns) ? turns / 2 * 2 : 0;
  for (int i = 0; i < both; i += 2) {
    F2 f[2][4], e[2][4];
    float dg[2], db[2];
    rows(i, f[0], e[0]);
    rows(i + 1, f[1], e[1]);
    take(f[0], e[0], s_gamma[first + i * step], dg[0], db[0]);
    take(f[1], e[1], s_gamma[first + (i + 1) * step], dg[1], db[1]);
    if (sums) {
      keep(i, dg[0], db[0]);
      keep(i + 1, dg[1], db[1]);
    }
  }
  for (int i = both; i < turns; ++i) {
    float dg = 0.f, db = 0.f;
    if (i < n) {
      F2 f[4], e[4];
      rows(i, f, e);
      take(f, e, gamma(first + i * step), dg, db);
    }
    if (sums) keep(i, dg, db);
  }
  column_sums<2>(c, lpr, scratch, s_c);
  if (C > 1) cluster_sync();
  {
    const int q = threadIdx.x / kMaxCols, t = threadIdx.x % kMaxCols;
    if (q < 2 && t < lpr * 8) {
      float total = s_c[q][t];
      if (C > 1) {
        float a[kMaxCluster];
        ld_cluster_all(&s_c[q][t], C, a);
        total = 0.f;
#pragma unroll
        for (int u = 0; u < kMaxCluster; ++u) total += a[u];
      }
      t_c[q][t] = -total / (float)p.K;
    }
  }
  if (C > 1) cluster_arrive();  // done with the other CTAs' sums
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[q][j] = f2(t_c[q][8 * col8 + 2 * j], t_c[q][8 * col8 + 2 * j + 1]);
  uint8_t* out = static_cast<uint8_t*>(p.Y) + ((r0 + first) * p.ldo + t0) * (kX / 8);
  const int64_t out_step = step * p.ldo * (kX / 8);
  auto write = [&](auto whole) {
    each_row<2>(n, [&](int i, auto u) {
      constexpr int U = decltype(u)::value;
      F2 f[U][4], e[U][4];
      float g[U];
#pragma unroll
      for (int r = 0; r < U; ++r) {
        g[r] = CACHED ? s_gamma[first + (i + r) * step] : gamma(first + (i + r) * step);
        rows(i + r, f[r], e[r]);
      }
#pragma unroll
      for (int r = 0; r < U; ++r) {
        const F2 g2 = f2(g[r], g[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 h = mul2(add2(f[r][j], mean[j]), rs[j]);
          f[r][j] = mul2(rs[j], fma2(g2, e[r][j], fma2(h, c[1][j], c[0][j])));
        }
        store_piece<XF32, decltype(whole)::value>(out, valid, f[r]);
        out += out_step;
      }
    });
  };
  if (ok && valid == 8)
    write(std::true_type());
  else if (ok && valid > 0)
    write(std::false_type());
  if (C > 1) cluster_wait();  // the other CTAs have read this one's sums
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

// Strip width, cluster size and rows per CTA, from the bytes of one element (X's type, and dY's in the backward pass).
// Strips of 64 tokens (128 bytes of bf16 a row; strips of 32 tokens: 40 us instead of 36 forward, 111 instead of 85
// backward, 768 x 50432), narrower for few tokens and for a K whose slab does not leave half an SM in a cluster of
// eight; for larger K strips of 16 tokens that fit at all, then of 8; past that nothing is cached.  Then the smallest
// cluster that keeps the slab there (a cluster's synchronisation cost more than smaller slabs and more CTAs to an SM
// gained: 51 and 106 us with slabs of 52 KB), enlarged while the grid leaves SMs idle.
void norm_shape(NormParams& p, int64_t bytes) {
  using namespace norm;
  auto box_of = [](int64_t rows) { return rows >= 512 ? 128 : 32; };  // whole boxes; few of them to issue
  auto slab = [&](int l, int c) {
    const int64_t rows = (p.K + c - 1) / c;
    const int64_t box = box_of(rows);
    return (rows + box - 1) / box * box * 8 * l * bytes;
  };
  auto total = [&](int l, int c) { return slab(l, c) + (p.K + c - 1) / c * 8; };  // gamma and beta behind it
  int lpr = kMaxCols / 8;
  while (lpr > 1 && (int64_t)(lpr / 2) * 8 >= p.T) lpr >>= 1;
  int64_t limit = kSlabBytes;
  while (lpr > 2 && total(lpr, kMaxCluster) > limit) lpr >>= 1;
  if (total(lpr, kMaxCluster) > limit) limit = kMaxSlabBytes;
  if (total(lpr, kMaxCluster) > limit) lpr = 1;
  p.cached = total(lpr, kMaxCluster) <= limit;
  int c = 1;
  while (c < kMaxCluster && total(lpr, c) > limit) c <<= 1;
  p.tiles = (p.T + 8 * lpr - 1) / (8 * lpr);
  while (c < kMaxCluster && p.tiles * c < 2 * (int64_t)sm_count_current() && p.K / c > kThreads / lpr) c <<= 1;
  p.lpr = lpr;
  p.cluster = c;
  p.rows = (p.K + c - 1) / c;
  p.box_rows = box_of(p.rows);
  p.slab = p.cached ? (uint32_t)slab(lpr, c) : 0;
  p.smem = p.cached ? (uint32_t)total(lpr, c) : 0;
}

template <auto Kern>
static cudaError_t launch_norm_grid(const NormParams& p, cudaStream_t s) {
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

template <bool XF32, bool YF32>
static cudaError_t launch_norm_types(const NormParams& p, cudaStream_t s) {
  return p.cached ? launch_norm_grid<&norm_kernel<XF32, YF32, true>>(p, s)
                  : launch_norm_grid<&norm_kernel<XF32, YF32, false>>(p, s);
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.x_f32) return p.y_f32 ? launch_norm_types<true, true>(p, s) : launch_norm_types<true, false>(p, s);
  return p.y_f32 ? launch_norm_types<false, true>(p, s) : launch_norm_types<false, false>(p, s);
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

// Map of a K x T tensor in boxes of box_rows rows of one strip.
static nm_status norm_map(CUtensorMap* tm, const void* base, int64_t K, int64_t T, int64_t ld, nm_out_dtype dtype,
                          const NormParams& p, const char* what) {
  const bool f32 = dtype == NM_OUT_F32;
  return make_tmap(tm, base, (uint64_t)T, (uint64_t)K, (uint64_t)(ld * dtype_bytes(dtype)), 8u * (uint32_t)p.lpr,
                   (uint32_t)p.box_rows, 0, what,
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
  if (st == NM_OK) st = check_words({gamma, beta, mean, rstd}, "gamma, beta, mean and rstd");
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
  if (p.cached) st = norm_map(&p.tm_x, X, K, T, ldx, x_dtype, p, "X");
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
  nm_status st = check_words({gamma, mean, rstd, dgamma, dbeta}, "gamma, mean, rstd, dgamma and dbeta");
  if (st != NM_OK) return st;
  if (T == 0) {  // empty sums
    if (!dgamma && !dbeta) return NM_OK;
    st = require_device();
    if (st != NM_OK) return st;
    cudaError_t e = launch_norm_grad_reduce(nullptr, 0, K, dgamma, dbeta, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "layer norm gradient reduction launch");
  }
  st = check_matrix(dY, lddy, T, dtype_bytes(dy_dtype), "dY");
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
  if (p.cached) st = norm_map(&p.tm_x, X, K, T, ldx, x_dtype, p, "X");
  if (p.cached && st == NM_OK) st = norm_map(&p.tm_d, dY, K, T, lddy, dy_dtype, p, "dY");
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
