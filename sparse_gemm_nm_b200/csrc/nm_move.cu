// nm_move.cu -- tokens to the columns grouped by expert and back, for activations with the tokens contiguous.
//
//   gather        Xg[r][s] = X[r][source[s] mod T]
//   combine       Y[r][t] = sum_j gate[j][t] Yg[r][slot[j][t]]
//   combine_grad  dYg[r][s] = gate[source[s]] dY[r][source[s] mod T],  dgate[j][t] = sum_r dY[r][t] Yg[r][slot[j][t]]
//
// Moving columns of a row-major matrix means picking 2-byte elements.  From global memory every element is a request of its
// own; so a CTA brings RB rows into shared memory whole, the RB elements of a column side by side (one 2, 4 or 8-byte word a
// column), picks columns there, and rows are stored in 16-byte units again: HBM sees each row read and written once, in
// order.  Four rows make one shared-memory access serve four elements; fewer rows, where four would leave room for only one
// CTA on an SM (loading and picking then take turns).  Short rows: a CTA takes several groups of rows, so that its threads
// have columns enough.  Rows too long for shared memory are picked from global memory.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace mv {
constexpr int kThreads = 512;
constexpr int64_t kTileBytes = 72 * 1024;  // three CTAs to an SM
constexpr int64_t kMaxTile = 200 * 1024;   // one

struct Params {
  const uint16_t* in;  // rows picked from: X, Yg, dY
  int64_t ldin;
  int32_t cols_in;
  void* out;           // rows written: Xg, Y, dYg
  int64_t ldout;
  int32_t cols_out;
  int32_t rows, T, k;
  uint32_t inv_T;          // floor(2^32 / T), at most 2^32 - 1
  const int32_t* index;    // source (S) or slot (k x T)
  const float* gate;       // k x T, or null
  int out_f32;
  int vec;                 // index (and gate) may be read 16 bytes at a time
  int groups;              // row groups of a CTA
  int depth;               // long rows: groups of rows in the ring
  uint32_t* status;
  // combine_grad
  const uint16_t* yg;
  int64_t ldyg;
  float* part;             // [CTA rows][S]
};

// RB elements of a column, as one word.
template <int RB> struct Word;
template <> struct Word<1> { using type = uint16_t; };
template <> struct Word<2> { using type = uint32_t; };
template <> struct Word<4> { using type = uint2; };

__device__ __forceinline__ float bf(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// source mod T (source >= 0): the estimate of the quotient is at most one too small.
__device__ __forceinline__ int32_t token_of(int32_t source, int32_t T, uint32_t inv_T) {
  const uint32_t q = __umulhi((uint32_t)source, inv_T);
  const int32_t r = source - (int32_t)q * T;
  return r >= T ? r - T : r;
}

// Eight consecutive 32-bit values, `fill` behind the first `valid`.  Indices and gates are read by every CTA: ordinary loads,
// which L1 holds (past it, a few lines of L2 that all SMs ask for at once: 4096 rows of 200 columns, combine_grad 25 us).
template <typename V>
__device__ __forceinline__ void load8(const V* p, int valid, bool vec, V fill, V (&v)[8]) {
  if (vec && valid >= 8) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const V*>(&w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? p[i] : fill;
  }
}

// The rows of this CTA's groups into shared memory, tile[group][column], RB rows a word; rows past the last are zeros.
template <int RB>
__device__ __forceinline__ void load_rows(const Params& p, int64_t row0, typename Word<RB>::type* tile) {
  const int32_t pairs = (p.cols_in + 1) >> 1;  // of columns; rows are padded to 16 bytes or end with the matrix
  const int32_t items = p.groups * pairs;  // what they take fits shared memory
#pragma unroll 2
  for (int32_t i = threadIdx.x; i < items; i += blockDim.x) {
    const int32_t g = p.groups == 1 ? 0 : i / pairs, c = (i - g * pairs) * 2;
    uint32_t w[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = row0 + (int64_t)g * RB + r;
      const uint16_t* at = p.in + row * p.ldin + c;
      w[r] = row >= p.rows ? 0u : c + 1 < p.cols_in ? __ldcg(reinterpret_cast<const uint32_t*>(at)) : (uint32_t)__ldcg(at);
    }
    typename Word<RB>::type* to = tile + g * (2 * pairs) + c;
    if constexpr (RB == 1) {
      *reinterpret_cast<uint32_t*>(to) = w[0];
    } else if constexpr (RB == 2) {
      *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
    } else {
      *reinterpret_cast<uint4*>(to) = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                                                 __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
    }
  }
}

// The RB elements of column c (outside [0, cols_in): zeros), bf16 pairs.  Read in any case, from column 0 where there is
// none, and masked: loads behind a condition would be waited for one by one.
template <int RB, bool DIRECT>
__device__ __forceinline__ void pick(const Params& p, const typename Word<RB>::type* tile, int64_t row, int32_t c,
                                     uint32_t (&w)[(RB + 1) / 2]) {
  const bool in = (uint32_t)c < (uint32_t)p.cols_in;
  const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
  const int32_t at = in ? c : 0;
  if constexpr (DIRECT) {
    w[0] = (uint32_t)p.in[row * p.ldin + at] & keep;
  } else if constexpr (RB == 4) {
    const uint2 v = tile[at];
    w[0] = v.x & keep;
    w[1] = v.y & keep;
  } else {
    w[0] = (uint32_t)tile[at] & keep;
  }
}

// Eight columns of a row.
__device__ __forceinline__ void store8(uint16_t* to, int valid, const uint32_t (&w)[4]) {
  if (valid >= 8) {
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) to[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* to, int valid, const float (&f)[8]) {
  if (valid >= 8) {
    reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) to[i] = f[i];
  }
}

// Row r of eight picked columns as four bf16 pairs.
template <int RB>
__device__ __forceinline__ void row_of(const uint32_t (&v)[8][(RB + 1) / 2], int r, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __byte_perm(v[2 * i][r >> 1], v[2 * i + 1][r >> 1], (r & 1) ? 0x7632 : 0x5410);
}

template <int RB, bool DIRECT>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ Params p) {
  using W = typename Word<RB>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  W* tile = reinterpret_cast<W*>(smem);
  const int64_t row0 = (int64_t)blockIdx.x * p.groups * RB;
  const int32_t width = (p.cols_in + 1) & ~1;
  pdl_gate();
  if (!DIRECT) {
    load_rows<RB>(p, row0, tile);
    __syncthreads();
  }
  const int32_t units = (p.cols_out + 7) >> 3;
  const int64_t items = (int64_t)p.groups * units;
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < items; i += (int64_t)gridDim.y * blockDim.x) {
    const int g = p.groups == 1 ? 0 : (int)((uint32_t)i / (uint32_t)units);
    const int32_t s = (int32_t)(i - (int64_t)g * units) * 8;
    const int64_t row = row0 + (int64_t)g * RB;
    if (row >= p.rows) break;
    const int valid = p.cols_out - s;
    int32_t src[8];
    load8<int32_t>(p.index + s, valid, p.vec, -1, src);
    uint32_t v[8][(RB + 1) / 2];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      pick<RB, DIRECT>(p, tile + (int64_t)g * width, row, src[c] < 0 ? -1 : token_of(src[c], p.T, p.inv_T), v[c]);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      if (row + r >= p.rows) break;
      uint32_t w[4];
      row_of<RB>(v, r, w);
      store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + s, valid, w);
    }
  }
}

// Sums in fp32, j ascending, rounded once.  A slot outside the columns adds nothing, whatever its gate is.
template <int RB, bool DIRECT>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ Params p) {
  using W = typename Word<RB>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  W* tile = reinterpret_cast<W*>(smem);
  const int64_t row0 = (int64_t)blockIdx.x * p.groups * RB;
  const int32_t width = (p.cols_in + 1) & ~1;
  pdl_gate();
  if (!DIRECT) {
    load_rows<RB>(p, row0, tile);
    __syncthreads();
  }
  const int32_t units = (p.cols_out + 7) >> 3;
  const int64_t items = (int64_t)p.groups * units;
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < items; i += (int64_t)gridDim.y * blockDim.x) {
    const int g = p.groups == 1 ? 0 : (int)((uint32_t)i / (uint32_t)units);
    const int32_t t = (int32_t)(i - (int64_t)g * units) * 8;
    const int64_t row = row0 + (int64_t)g * RB;
    if (row >= p.rows) break;
    const int valid = p.cols_out - t;
    float acc[RB][8];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[r][c] = 0.f;
#pragma unroll 2
    for (int j = 0; j < p.k; ++j) {
      int32_t slot[8];
      float gate[8];
      load8<int32_t>(p.index + (int64_t)j * p.T + t, valid, p.vec, -1, slot);
      if (p.gate) {
        load8<float>(p.gate + (int64_t)j * p.T + t, valid, p.vec, 0.f, gate);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) gate[c] = 1.f;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t v[(RB + 1) / 2];
        pick<RB, DIRECT>(p, tile + (int64_t)g * width, row, slot[c], v);
        const float f = (uint32_t)slot[c] < (uint32_t)p.cols_in ? gate[c] : 0.f;
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][c] = fmaf(f, r & 1 ? bf_hi(v[r >> 1]) : bf_lo(v[r >> 1]), acc[r][c]);
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      if (row + r >= p.rows) break;
      if (p.out_f32) {
        store8(static_cast<float*>(p.out) + (row + r) * p.ldout + t, valid, acc[r]);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(acc[r][2 * c], acc[r][2 * c + 1]);
        store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + t, valid, w);
      }
    }
  }
}

// A CTA takes `groups` groups of RB rows one after the other and one range of the columns (gridDim.y), whose dot products
// it keeps in shared memory (each by the thread that owns the column) and leaves as one partial sum a column.
template <int RB, bool DIRECT>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const __grid_constant__ Params p) {
  using W = typename Word<RB>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t units = (p.cols_out + 7) >> 3;
  const int32_t per = (units + (int32_t)gridDim.y - 1) / (int32_t)gridDim.y;
  const int32_t u0 = (int32_t)blockIdx.y * per, u1 = min(u0 + per, units);
  float4* dots = reinterpret_cast<float4*>(smem);  // two a unit
  W* tile = reinterpret_cast<W*>(smem + (int64_t)per * 32);
  pdl_gate();
  Params one = p;
  one.groups = 1;
  for (int g = 0; g < p.groups; ++g) {
    const int64_t row = ((int64_t)blockIdx.x * p.groups + g) * RB;
    if (row >= p.rows) break;
    if (!DIRECT) {
      if (g) __syncthreads();  // the last group's columns are picked
      load_rows<RB>(one, row, tile);
      __syncthreads();
    }
    for (int32_t u = u0 + (int32_t)threadIdx.x; u < u1; u += blockDim.x) {
      const int32_t s = u * 8;
      const int valid = p.cols_out - s;
      int32_t src[8];
      load8<int32_t>(p.index + s, valid, p.vec, -1, src);
      uint4 y[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        y[r] = make_uint4(0, 0, 0, 0);
        if (row + r >= p.rows) continue;
        const uint16_t* at = p.yg + (row + r) * p.ldyg + s;
        if (valid >= 8) {
          y[r] = __ldcg(reinterpret_cast<const uint4*>(at));
        } else {
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < valid) w[c >> 1] |= (uint32_t)__ldcg(at + c) << (16 * (c & 1));
          y[r] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      float dot[8];
      if (g) {
        const float4 a = dots[2 * (u - u0)], b = dots[2 * (u - u0) + 1];
        dot[0] = a.x, dot[1] = a.y, dot[2] = a.z, dot[3] = a.w, dot[4] = b.x, dot[5] = b.y, dot[6] = b.z, dot[7] = b.w;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) dot[c] = 0.f;
      }
      float d[RB][8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t v[(RB + 1) / 2];
        const bool live = src[c] >= 0 && src[c] < p.k * p.T;
        pick<RB, DIRECT>(p, tile, row, live ? token_of(src[c], p.T, p.inv_T) : -1, v);
        const float gate = !live ? 0.f : p.gate ? p.gate[src[c]] : 1.f;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float dy = r & 1 ? bf_hi(v[r >> 1]) : bf_lo(v[r >> 1]);
          const uint32_t yw = c < 2 ? y[r].x : c < 4 ? y[r].y : c < 6 ? y[r].z : y[r].w;
          if (live) dot[c] = fmaf(dy, c & 1 ? bf_hi(yw) : bf_lo(yw), dot[c]);
          d[r][c] = live ? gate * dy : 0.f;
        }
      }
      dots[2 * (u - u0)] = make_float4(dot[0], dot[1], dot[2], dot[3]);
      dots[2 * (u - u0) + 1] = make_float4(dot[4], dot[5], dot[6], dot[7]);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        if (row + r >= p.rows) break;
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(d[r][2 * c], d[r][2 * c + 1]);
        store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + s, valid, w);
      }
    }
  }
  // Each thread reads back the columns that it owns.
  for (int32_t u = u0 + (int32_t)threadIdx.x; u < u1; u += blockDim.x) {
    float4* to = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * (units * 8) + u * 8);
    to[0] = dots[2 * (u - u0)];
    to[1] = dots[2 * (u - u0) + 1];
  }
}

// Few tokens: rows of Yg and dY are a few lines, picked from L1; a thread keeps its eight columns and takes row after row, the
// CTA's threads side by side in rows.  gridDim.y ranges of kFewThreads units.
constexpr int kFewThreads = 256;
__global__ void __launch_bounds__(kFewThreads) combine_grad_few_kernel(const __grid_constant__ Params p) {
  __shared__ float4 sums[kFewThreads][2];
  const int32_t all = (p.cols_out + 7) >> 3, u0 = (int32_t)blockIdx.y * kFewThreads, units = min(all - u0, kFewThreads);
  const int lanes = kFewThreads / units, rl = (int)threadIdx.x / units, u = u0 + (int)threadIdx.x - rl * units;
  const int32_t s = 8 * u;
  const int valid = p.cols_out - s;
  pdl_gate();
  float dot[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) dot[c] = 0.f;
  if (rl < lanes) {
    int32_t src[8];
    float gate[8];
    uint32_t live = 0;  // a bit a column
    load8<int32_t>(p.index + s, valid, p.vec, -1, src);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const bool has = src[c] >= 0 && src[c] < p.k * p.T;
      live |= (has ? 1u : 0u) << c;
      src[c] = has ? src[c] : 0;  // (any token: what is read is not used)
      gate[c] = 1.f;
    }
    if (p.gate) {
#pragma unroll
      for (int c = 0; c < 8; ++c) gate[c] = p.gate[src[c]];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      gate[c] = live >> c & 1u ? gate[c] : 0.f;
      src[c] = token_of(src[c], p.T, p.inv_T);
    }
    const int64_t end = min((int64_t)p.rows, ((int64_t)blockIdx.x + 1) * p.groups);
    // A row's elements, the next row's on their way meanwhile (the stores hide from the compiler that they may be).
    auto fetch = [&](int64_t row, uint32_t (&x)[8], uint32_t (&y)[4]) {
      const uint16_t* from = p.in + row * p.ldin;
      const uint16_t* at = p.yg + row * p.ldyg + s;
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = from[src[c]];
      if (valid >= 8) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(at));
        y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
      } else {
        y[0] = y[1] = y[2] = y[3] = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < valid) y[c >> 1] |= (uint32_t)__ldcg(at + c) << (16 * (c & 1));
      }
    };
    uint32_t x[8], y[4];
    int64_t row = (int64_t)blockIdx.x * p.groups + rl;
    if (row < end) fetch(row, x, y);
    for (; row < end; row += lanes) {
      uint32_t nx[8] = {}, ny[4] = {};
      if (row + lanes < end) fetch(row + lanes, nx, ny);
      float d[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // a column of no token may hold anything
        const uint32_t keep = 0u - (live >> c & 1u);
        const float dy = bf(x[c] & keep), yv = __uint_as_float((c & 1 ? y[c >> 1] & 0xFFFF0000u : y[c >> 1] << 16) & keep);
        dot[c] = fmaf(dy, yv, dot[c]);
        d[c] = gate[c] * dy;
      }
      uint32_t w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(d[2 * c], d[2 * c + 1]);
      store8(static_cast<uint16_t*>(p.out) + row * p.ldout + s, valid, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = nx[c];
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = ny[c];
    }
  }
  // The rows' lanes of a unit, two by two.
  sums[threadIdx.x][0] = make_float4(dot[0], dot[1], dot[2], dot[3]);
  sums[threadIdx.x][1] = make_float4(dot[4], dot[5], dot[6], dot[7]);
  int half = 1;
  while (2 * half < lanes) half *= 2;
  for (; lanes > 1 && half > 0; half >>= 1) {
    __syncthreads();
    if (rl < half && rl + half < lanes) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 a = sums[threadIdx.x][i];
        const float4 b = sums[threadIdx.x + half * units][i];
        a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        sums[threadIdx.x][i] = a;
      }
    }
  }
  if (rl == 0) {
    float4* to = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * (all * 8) + s);
    to[0] = sums[threadIdx.x][0];
    to[1] = sums[threadIdx.x][1];
  }
}

// ------------------------------------------------------------ long rows
// The same by persistent CTAs that keep every column's index (and gate) in shared memory, 16 and 32 bits each, and take
// group after group of kRows rows: read again for every group, the indices are as many bytes as the rows themselves.
// Rows arrive by bulk copies in a ring of groups, as they lie in memory, so that loads never stop for the threads (with rows
// brought through registers between two barriers, the loads of a CTA waited for its picks and the other way round: combine
// of 8192 tokens at two experts, 4096 rows, 65 to 82 us).  A column is one 2-byte access a row, of random banks: about half
// the time that HBM takes for the same row.  The word behind a row's columns is zero and stands for no column.
namespace lng {
constexpr int kThreads = 1024;
constexpr int64_t kMaxSmem = 226 * 1024;
constexpr int kMaxDepth = 8;
constexpr int64_t kLeastOut = 4096;  // columns of the result, eight a thread: half the CTA's threads at least
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kBarBytes = 2 * kMaxDepth * 8 + 16;

__host__ __device__ inline int32_t row_bytes(int32_t cols) { return ((cols + 7) & ~7) * 2 + 16; }

// The ring of a CTA's groups of rows: group i has the rows (blockIdx.x + i gridDim.x) ROWS ..
template <int ROWS>
struct Ring {
  uint64_t *full, *empty;
  volatile int* abort;
  uint8_t* slots;
  int32_t pitch, issued;
  uint32_t slot, phase;  // of the group being read
  bool ok;

  // smem: kBarBytes, then depth x ROWS rows.  Every thread; followed by a barrier of the CTA.
  __device__ __forceinline__ void init(const Params& p, uint8_t* smem) {
    full = reinterpret_cast<uint64_t*>(smem);
    empty = full + kMaxDepth;
    abort = reinterpret_cast<volatile int*>(empty + kMaxDepth);
    slots = smem + kBarBytes;
    pitch = row_bytes(p.cols_in);
    issued = 0;
    slot = 0;
    phase = 0;
    ok = true;
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.depth; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], kThreads / 32);
      }
      *abort = 0;
      fence_barrier_init();
      fence_proxy_async_smem();
    }
    for (int i = threadIdx.x; i < p.depth * ROWS; i += kThreads)
      *reinterpret_cast<uint4*>(slots + (int64_t)(i + 1) * pitch - 16) = make_uint4(0, 0, 0, 0);
  }
  // Thread 0: the next group's copies, once its slot has been read.
  __device__ __forceinline__ void issue(const Params& p) {
    const int64_t row0 = ((int64_t)blockIdx.x + (int64_t)issued * gridDim.x) * ROWS;
    if (row0 >= p.rows || !ok) return;
    const int at = issued % p.depth;
    const uint32_t turn = (uint32_t)(issued / p.depth);
    ok = mbar_wait(&empty[at], (turn & 1u) ^ 1u, abort, p.status, kWaitNs);
    if (!ok) return;
    uint8_t* to = slots + (int64_t)at * ROWS * pitch;
    const uint32_t whole = (uint32_t)((p.cols_in + 7) >> 3) * 16u, part = (uint32_t)(p.cols_in >> 3) * 16u;
    uint32_t bytes = 0;
    for (int r = 0; r < ROWS && row0 + r < p.rows; ++r) {
      const bool last = row0 + r == p.rows - 1;  // memory may end with its last column
      bytes += last ? part : whole;
      if (last)
        for (int c = p.cols_in & ~7; c < p.cols_in; ++c)
          reinterpret_cast<uint16_t*>(to + r * pitch)[c] = p.in[(row0 + r) * p.ldin + c];
    }
    mbar_arrive_expect_tx(&full[at], bytes);
    for (int r = 0; r < ROWS && row0 + r < p.rows; ++r) {
      const uint32_t n = row0 + r == p.rows - 1 ? part : whole;
      if (n) bulk_load(to + r * pitch, p.in + (row0 + r) * p.ldin, n, &full[at]);
    }
    ++issued;
  }
  // The rows of the group to be read, for a warp.
  __device__ __forceinline__ const uint8_t* wait(const Params& p) {
    ok = mbar_wait_warp(&full[slot], phase, abort, p.status, kWaitNs);
    return slots + (int64_t)slot * ROWS * pitch;
  }
  __device__ __forceinline__ void done(const Params& p, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == (uint32_t)p.depth) {
      slot = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void leave() {
    __syncthreads();
    if (*abort && threadIdx.x == 0) sleep_about_ns(200000ull);  // copies in flight
  }
};

// Eight 16-bit indices from shared memory.
__device__ __forceinline__ void indices(const uint16_t* at, int32_t (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(at);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (int32_t)(w[i] & 0xFFFFu);
    v[2 * i + 1] = (int32_t)(w[i] >> 16);
  }
}
__device__ __forceinline__ void values(const float* at, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

constexpr int kGradUnits = 2;  // units of eight columns a thread holds the dot products of

// The gather has room for two tiles of RB rows as words, and one access a column then serves RB rows: the next group's rows
// are on their way to registers while this one's columns are picked, and go to the other tile (8192 tokens at two experts,
// 4096 rows: 42 us, from the ring 50).
template <int RB>
struct Next {
  static constexpr int kUnits = 4 / RB;  // units of eight columns a thread brings
  uint4 v[kUnits][RB];

  __device__ __forceinline__ void fetch(const Params& p, int64_t row0) {
    const int32_t units = (p.cols_in + 7) >> 3;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int32_t u = (int32_t)threadIdx.x + i * kThreads;
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        v[i][r] = make_uint4(0, 0, 0, 0);
        if (u >= units || row0 + r >= p.rows) continue;
        const uint16_t* at = p.in + (row0 + r) * p.ldin + 8 * u;
        if (8 * u + 8 <= p.cols_in) {
          v[i][r] = __ldcg(reinterpret_cast<const uint4*>(at));
        } else {  // the row's last columns one by one
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (8 * u + c < p.cols_in) w[c >> 1] |= (uint32_t)__ldcg(at + c) << (16 * (c & 1));
          v[i][r] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  // Into the tile, the RB elements of a column side by side.  Lanes store their 16-byte pieces in different orders, so that
  // eight of them meet every bank once.
  __device__ __forceinline__ void put(const Params& p, typename Word<RB>::type* tile) const {
    const int32_t units = (p.cols_in + 7) >> 3;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int32_t u = (int32_t)threadIdx.x + i * kThreads;
      if (u >= units) continue;
      uint4* to = reinterpret_cast<uint4*>(tile + 8 * u);
      if constexpr (RB == 1) {
        to[0] = v[i][0];
      } else if constexpr (RB == 2) {
        const uint4 a = v[i][0], b = v[i][1];
        const uint4 lo = make_uint4(__byte_perm(a.x, b.x, 0x5410), __byte_perm(a.x, b.x, 0x7632),
                                    __byte_perm(a.y, b.y, 0x5410), __byte_perm(a.y, b.y, 0x7632));
        const uint4 hi = make_uint4(__byte_perm(a.z, b.z, 0x5410), __byte_perm(a.z, b.z, 0x7632),
                                    __byte_perm(a.w, b.w, 0x5410), __byte_perm(a.w, b.w, 0x7632));
        const int second = (u >> 2) & 1;
        to[second] = second ? hi : lo;
        to[second ^ 1] = second ? lo : hi;
      } else {
        const uint4 a = v[i][0], b = v[i][1], c = v[i][2], d = v[i][3];
        uint4 q[4];
        q[0] = make_uint4(__byte_perm(a.x, b.x, 0x5410), __byte_perm(c.x, d.x, 0x5410), __byte_perm(a.x, b.x, 0x7632),
                          __byte_perm(c.x, d.x, 0x7632));
        q[1] = make_uint4(__byte_perm(a.y, b.y, 0x5410), __byte_perm(c.y, d.y, 0x5410), __byte_perm(a.y, b.y, 0x7632),
                          __byte_perm(c.y, d.y, 0x7632));
        q[2] = make_uint4(__byte_perm(a.z, b.z, 0x5410), __byte_perm(c.z, d.z, 0x5410), __byte_perm(a.z, b.z, 0x7632),
                          __byte_perm(c.z, d.z, 0x7632));
        q[3] = make_uint4(__byte_perm(a.w, b.w, 0x5410), __byte_perm(c.w, d.w, 0x5410), __byte_perm(a.w, b.w, 0x7632),
                          __byte_perm(c.w, d.w, 0x7632));
        const int turn = (u >> 1) & 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = j ^ turn;
          to[k] = k & 2 ? (k & 1 ? q[3] : q[2]) : (k & 1 ? q[1] : q[0]);
        }
      }
    }
  }
};

template <int RB>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ Params p) {
  using W = typename Word<RB>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t width = (p.cols_in + 7) & ~7, units = (p.cols_out + 7) >> 3;
  uint16_t* index = reinterpret_cast<uint16_t*>(smem);
  W* const tiles = reinterpret_cast<W*>(smem + (int64_t)units * 16);
  pdl_gate();
  Next<RB> next;
  int64_t row = (int64_t)blockIdx.x * RB;
  next.fetch(p, row);
  for (int32_t s = threadIdx.x; s < units * 8; s += kThreads) {
    const int32_t src = s < p.cols_out ? __ldcg(p.index + s) : -1;
    index[s] = src < 0 ? (uint16_t)0xFFFFu : (uint16_t)token_of(src, p.T, p.inv_T);
  }
  for (int second = 0; row < p.rows; row += (int64_t)gridDim.x * RB, second ^= 1) {
    W* tile = tiles + second * width;
    next.put(p, tile);
    __syncthreads();  // and all are through with the other tile
    next.fetch(p, row + (int64_t)gridDim.x * RB);
    for (int32_t u = threadIdx.x; u < units; u += kThreads) {
      int32_t t[8];
      indices(index + 8 * u, t);
      uint32_t v[8][(RB + 1) / 2];
#pragma unroll
      for (int c = 0; c < 8; ++c) pick<RB, false>(p, tile, row, t[c], v[c]);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        if (row + r >= p.rows) break;
        uint32_t w[4];
        row_of<RB>(v, r, w);
        store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + 8 * u, p.cols_out - 8 * u, w);
      }
    }
  }
}
// Rows of its word (0: it does not fit).
inline int gather_rows(int64_t cols, int64_t cols_out, int64_t rows, int64_t beside) {
  const int64_t units = (cols + 7) / 8;
  if (cols_out < kLeastOut) return 0;
  for (int rb = 4; rb >= 1; rb >>= 1)
    if (cols < 0xFFFF && units <= (int64_t)kThreads * (4 / rb) && 2 * units * 16 * rb + beside <= kMaxSmem &&
        rows >= 3 * (int64_t)rb * sm_count_current())
      return rb;
  return 0;
}
template <int RB>
static cudaError_t launch_gather(const Params& p, unsigned grid, size_t smem, cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(gather_kernel<RB>, (uint32_t)kMaxSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(gather_kernel<RB>, dim3(grid), dim3(kThreads), smem, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// gridDim.y ranges of the tokens.
template <int ROWS>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t all = (p.cols_out + 7) >> 3, none = (p.cols_in + 7) & ~7;
  const int32_t most = (all + (int32_t)gridDim.y - 1) / (int32_t)gridDim.y, per = most * 8;
  const int32_t u0 = (int32_t)blockIdx.y * most, units = min(most, all - u0);
  const int lane = threadIdx.x & 31;
  float* gates = reinterpret_cast<float*>(smem);
  uint16_t* index = reinterpret_cast<uint16_t*>(gates + (p.gate ? (int64_t)p.k * per : 0));
  Ring<ROWS> ring;
  ring.init(p, reinterpret_cast<uint8_t*>(index + (int64_t)p.k * per));
  __syncthreads();
  pdl_gate();
  if (threadIdx.x == 0)
    for (int i = 0; i < p.depth; ++i) ring.issue(p);
  for (int j = 0; j < p.k; ++j)
    for (int32_t i = threadIdx.x; i < units * 8; i += kThreads) {
      const int32_t t = 8 * u0 + i, s = t < p.T ? __ldcg(p.index + (int64_t)j * p.T + t) : -1;
      const bool has = (uint32_t)s < (uint32_t)p.cols_in;
      index[j * per + i] = has ? (uint16_t)s : (uint16_t)none;
      if (p.gate) gates[j * per + i] = has ? __ldcg(p.gate + (int64_t)j * p.T + t) : 0.f;
    }
  __syncthreads();
  for (int64_t row = (int64_t)blockIdx.x * ROWS; row < p.rows; row += (int64_t)gridDim.x * ROWS) {
    const uint8_t* rows = ring.wait(p);
    if (!ring.ok) break;
    for (int32_t u = threadIdx.x; u < units; u += kThreads) {
      float acc[ROWS][8];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = 0.f;
      for (int j = 0; j < p.k; ++j) {
        int32_t s[8];
        float gate[8];
        indices(index + j * per + 8 * u, s);
        if (p.gate) {
          values(gates + j * per + 8 * u, gate);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) gate[c] = 1.f;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const uint16_t* from = reinterpret_cast<const uint16_t*>(rows + r * ring.pitch);
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[r][c] = fmaf(gate[c], bf(from[s[c]]), acc[r][c]);
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (row + r >= p.rows) break;
        if (p.out_f32) {
          store8(static_cast<float*>(p.out) + (row + r) * p.ldout + 8 * (u0 + u), p.cols_out - 8 * (u0 + u), acc[r]);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(acc[r][2 * c], acc[r][2 * c + 1]);
          store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + 8 * (u0 + u), p.cols_out - 8 * (u0 + u), w);
        }
      }
    }
    ring.done(p, lane);
    if (threadIdx.x == 0) ring.issue(p);
  }
  ring.leave();
}

// Eight columns of Yg from column s on, zeros behind the last.
__device__ __forceinline__ uint4 columns8(const Params& p, int64_t row, int32_t s) {
  if (row >= p.rows) return make_uint4(0, 0, 0, 0);
  const uint16_t* at = p.yg + row * p.ldyg + s;
  if (s + 8 <= p.cols_out) return __ldcg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (s + c < p.cols_out) w[c >> 1] |= (uint32_t)__ldcg(at + c) << (16 * (c & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// gridDim.y ranges of kThreads * kGradUnits units of the columns at most; the dot products stay with the threads.
template <int ROWS>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t all = (p.cols_out + 7) >> 3, none = (p.cols_in + 7) & ~7;
  const int32_t per = (all + (int32_t)gridDim.y - 1) / (int32_t)gridDim.y;
  const int32_t u0 = (int32_t)blockIdx.y * per, units = min(per, all - u0);
  const int lane = threadIdx.x & 31;
  float* gates = reinterpret_cast<float*>(smem);
  uint16_t* index = reinterpret_cast<uint16_t*>(gates + per * 8);
  Ring<ROWS> ring;
  ring.init(p, reinterpret_cast<uint8_t*>(index + per * 8));
  __syncthreads();
  pdl_gate();
  if (threadIdx.x == 0)
    for (int i = 0; i < p.depth; ++i) ring.issue(p);
  uint4 y[kGradUnits][ROWS];  // the next group's columns of Yg
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int32_t u = (int32_t)threadIdx.x + i * kThreads;
        if (u < units) y[i][r] = columns8(p, row + r, 8 * (u0 + u));
      }
  };
  int64_t row = (int64_t)blockIdx.x * ROWS;
  fetch(row);
  for (int32_t i = threadIdx.x; i < units * 8; i += kThreads) {
    const int32_t s = 8 * u0 + i, src = s < p.cols_out ? __ldcg(p.index + s) : -1;
    const bool has = src >= 0 && src < p.k * p.T;
    index[i] = has ? (uint16_t)token_of(src, p.T, p.inv_T) : (uint16_t)none;
    gates[i] = !has ? 0.f : p.gate ? __ldcg(p.gate + src) : 1.f;
  }
  __syncthreads();
  float dot[kGradUnits][8];
#pragma unroll
  for (int i = 0; i < kGradUnits; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) dot[i][c] = 0.f;
  for (; row < p.rows; row += (int64_t)gridDim.x * ROWS) {
    const uint8_t* rows = ring.wait(p);
    if (!ring.ok) break;
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) {
      const int32_t u = (int32_t)threadIdx.x + i * kThreads;
      if (u >= units) break;
      const int32_t s = 8 * (u0 + u);
      const uint4 packed = *reinterpret_cast<const uint4*>(index + 8 * u);
      uint32_t w[ROWS][4];
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const uint32_t pair = c < 2 ? packed.x : c < 4 ? packed.y : c < 6 ? packed.z : packed.w;
        const int32_t t0 = (int32_t)(pair & 0xFFFFu), t1 = (int32_t)(pair >> 16);
        const float2 gate = *reinterpret_cast<const float2*>(gates + 8 * u + c);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const uint16_t* from = reinterpret_cast<const uint16_t*>(rows + r * ring.pitch);
          const uint32_t yw = c < 2 ? y[i][r].x : c < 4 ? y[i][r].y : c < 6 ? y[i][r].z : y[i][r].w;
          const float d0 = bf(from[t0]), d1 = bf(from[t1]);
          // a column of no token may hold anything, and so may the rows behind the last
          if (t0 != none && row + r < p.rows) dot[i][c] = fmaf(d0, bf_lo(yw), dot[i][c]);
          if (t1 != none && row + r < p.rows) dot[i][c + 1] = fmaf(d1, bf_hi(yw), dot[i][c + 1]);
          w[r][c >> 1] = pack_bf16x2(gate.x * d0, gate.y * d1);
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (row + r < p.rows)
          store8(static_cast<uint16_t*>(p.out) + (row + r) * p.ldout + s, p.cols_out - s, w[r]);
        y[i][r] = columns8(p, row + (int64_t)gridDim.x * ROWS + r, s);  // while the other units are at work
      }
    }
    ring.done(p, lane);
    if (threadIdx.x == 0) ring.issue(p);
  }
#pragma unroll
  for (int i = 0; i < kGradUnits; ++i) {
    const int32_t u = (int32_t)threadIdx.x + i * kThreads;
    if (u >= units) break;
    float4* to = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * (all * 8) + 8 * (u0 + u));
    to[0] = make_float4(dot[i][0], dot[i][1], dot[i][2], dot[i][3]);
    to[1] = make_float4(dot[i][4], dot[i][5], dot[i][6], dot[i][7]);
  }
  ring.leave();
}

// How a ring form takes a call: groups of `rows` rows, `depth` of them in the ring, the columns of the result in `ranges`.
struct Plan {
  int rows, depth;
  int64_t ranges, per;  // units a range
};
// For rows of `cols` elements and `units` units of the result, at most `most` a range, `beside` bytes of indices and gates
// a unit.  rows = 0 where no form fits (16-bit indices, two groups in shared memory) or each CTA would have too little to be
// worth its start.
inline Plan plan_of(int64_t cols, int64_t units, int64_t most, int64_t rows, int64_t beside) {
  if (cols > 65000) return Plan{0, 0, 0, 0};
  for (int64_t ranges = (units + most - 1) / most; ranges <= 16; ++ranges) {
    const int64_t per = (units + ranges - 1) / ranges;
    if (per < (ranges == 1 ? kThreads / 2 : 128)) break;
    for (int group = 2; group >= 1; --group) {
      if (rows * ranges < 3 * (int64_t)group * sm_count_current()) continue;
      const int64_t depth = (kMaxSmem - beside * per - kBarBytes) / ((int64_t)row_bytes((int32_t)cols) * group);
      if (depth >= 2) return Plan{group, depth < kMaxDepth ? (int)depth : kMaxDepth, ranges, per};
    }
  }
  return Plan{0, 0, 0, 0};
}
inline size_t smem_of(const Params& p, const Plan& l, int64_t beside) {
  return (size_t)(beside * l.per + kBarBytes + (int64_t)l.depth * l.rows * row_bytes(p.cols_in));
}
// CTAs for each range: one to an SM in all.
inline unsigned ctas_of(int64_t rows, const Plan& l) {
  const int64_t groups = (rows + l.rows - 1) / l.rows, ctas = sm_count_current() / l.ranges;
  return (unsigned)(groups < ctas ? groups : ctas < 1 ? 1 : ctas);
}
inline unsigned grid_of(int64_t rows, int group) {
  const int64_t groups = (rows + group - 1) / group, sms = sm_count_current();
  return (unsigned)(groups < sms ? groups : sms);
}
}  // namespace lng

// dgate[source[s]] = the partial sums of column s, in order; 0 for a pair without a column.  32 columns a CTA, whose warps
// take the partial sums in eight ranges.
__global__ void __launch_bounds__(256) dgate_kernel(const float* part, int32_t parts, int64_t pitch, const int32_t* source,
                                                    const int32_t* slot, int64_t n, int32_t S, float* dgate) {
  __shared__ float sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t s = (int64_t)blockIdx.x * 32 + lane;
  const int32_t b0 = parts * warp / 8, b1 = parts * (warp + 1) / 8;
  pdl_gate();
  float sum = 0.f;
  if (s < S) {
    int32_t b = b0;
    for (; b + 8 <= b1; b += 8) {
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = __ldcg(part + (b + q) * pitch + s);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum += f[q];
    }
    for (; b < b1; ++b) sum += __ldcg(part + b * pitch + s);
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  if (s < S) {
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += sums[w][lane];
    const int32_t src = __ldcg(source + s);
    if (src >= 0 && src < n) dgate[src] = sum;
  }
  if (s < n && (uint32_t)__ldcg(slot + s) >= (uint32_t)S) dgate[s] = 0.f;
}

static uint32_t inverse(int64_t T) {
  const uint64_t q = (1ull << 32) / (uint64_t)T;
  return q > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)q;
}

// Rows a word holds for rows of `cols` elements, beside `beside` bytes.  0: picked from global memory, where the row does not
// fit, or where it is two lines of L1 and not worth a barrier, or gives a group of rows to few threads (13824 rows, one
// token at two experts: combine 61 -> 8 us).
static int rows_of_word(int64_t cols, int64_t cols_out, int64_t rows, int64_t beside) {
  const int64_t one = (cols + 1) / 2 * 4;  // bytes of a row
  if (cols <= 128 || cols_out <= 256) return 0;
  for (int rb = 4; rb > 1; rb >>= 1)
    if (one * rb + beside <= kTileBytes && rows >= rb) return rb;
  for (int rb = 2; rb >= 1; rb >>= 1)
    if (one * rb + beside <= kMaxTile && (rows >= rb || rb == 1)) return rb;
  return 0;
}

template <template <int, bool> class Launch, typename... A>
static cudaError_t dispatch(int rb, A&&... a) {
  switch (rb) {
    case 4: return Launch<4, false>::go(a...);
    case 2: return Launch<2, false>::go(a...);
    case 1: return Launch<1, false>::go(a...);
    default: return Launch<1, true>::go(a...);
  }
}
template <typename Kernel>
static cudaError_t start(Kernel kernel, SmemLimit& limit, dim3 grid, size_t smem, const Params& p, cudaStream_t s,
                         int threads = kThreads) {
  cudaError_t e = limit.raise(kernel, (uint32_t)lng::kMaxSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, grid, dim3((unsigned)threads), smem, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int RB, bool DIRECT>
struct Gather {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s, int threads = kThreads) {
    static SmemLimit limit;
    return start(gather_kernel<RB, DIRECT>, limit, grid, smem, p, s, threads);
  }
};
template <int RB, bool DIRECT>
struct Combine {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s, int threads = kThreads) {
    static SmemLimit limit;
    return start(combine_kernel<RB, DIRECT>, limit, grid, smem, p, s, threads);
  }
};
template <int RB, bool DIRECT>
struct CombineGrad {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s, int threads = kThreads) {
    static SmemLimit limit;
    return start(combine_grad_kernel<RB, DIRECT>, limit, grid, smem, p, s, threads);
  }
};

// Threads for the units of a CTA's groups.
static int threads_of(int64_t cols_out, int groups) {
  const int64_t t = (((cols_out + 7) / 8 * groups) + 63) / 64 * 64;
  return t < 128 ? 128 : t < kThreads ? (int)t : kThreads;
}
// Few rows: CTAs that share a group of rows (each brings it), until every SM has one.
static unsigned shares_of(int64_t ctas, int64_t cols_out, int groups, int threads) {
  const int64_t most = ((cols_out + 7) / 8 * groups + threads - 1) / threads, want = sm_count_current() / ctas;
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}
// Row groups of a CTA: enough for its threads to have a unit of columns each, within the tile's bytes and the rows.
static int groups_of(int rb, int64_t rows, int64_t cols_in, int64_t cols_out) {
  const int64_t units = (cols_out + 7) / 8, one = rb ? (cols_in + 1) / 2 * 4 * rb : 1;
  int64_t g = kThreads / units;
  if (g * one > kTileBytes) g = kTileBytes / one;
  const int64_t need = (rows + (rb ? rb : 1) - 1) / (rb ? rb : 1);
  const int64_t spread = need / (4 * sm_count_current());  // CTAs for all SMs first
  if (g > spread) g = spread;
  return g < 1 ? 1 : (int)g;
}

static nm_status check(int64_t rows, int64_t T, int64_t k, int64_t S) {
  if (rows < 0 || T < 0 || S < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (k < 1) return fail(NM_ERR_INVALID_ARG, "k must be positive");
  const int64_t lim = kMaxDim - 4096;
  if (rows >= lim || T >= lim || S >= lim || (T > 0 && k >= lim / T))
    return fail(NM_ERR_UNSUPPORTED, "dimensions (and k * T) must stay below 2^31");
  return NM_OK;
}
}  // namespace mv

}  // namespace nmk

using namespace nmk;

extern "C" nm_status nm_experts_gather(const uint16_t* X, int64_t ldx, int64_t K, int64_t T, const int32_t* source, int64_t S,
                                       uint16_t* Xg, int64_t ldg, void* stream) {
  set_last_error("");
  nm_status st = mv::check(K, T, 1, S);
  if (st != NM_OK) return st;
  if (K == 0 || S == 0) return NM_OK;
  if (!source) return fail(NM_ERR_INVALID_ARG, "source is null");
  if (T == 0) return fail(NM_ERR_INVALID_ARG, "columns of no tokens");
  st = check_matrix(X, ldx, T, 2, "X");
  if (st == NM_OK) st = check_matrix(Xg, ldg, S, 2, "Xg");
  if (st == NM_OK) st = check_words({source}, "source");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  mv::Params p{};
  p.in = X, p.ldin = ldx, p.cols_in = (int32_t)T;
  p.out = Xg, p.ldout = ldg, p.cols_out = (int32_t)S;
  p.rows = (int32_t)K, p.T = (int32_t)T, p.k = 1, p.inv_T = mv::inverse(T);
  p.index = source;
  p.vec = al16(source);
  const int64_t beside = (S + 7) / 8 * 16;
  const int lrb = mv::lng::gather_rows(T, S, K, beside);
  if (lrb) {
    const size_t smem = (size_t)(2 * ((T + 7) / 8 * 16 * lrb) + beside);
    const unsigned grid = mv::lng::grid_of(K, lrb);
    const cudaError_t e = lrb == 4   ? mv::lng::launch_gather<4>(p, grid, smem, (cudaStream_t)stream)
                          : lrb == 2 ? mv::lng::launch_gather<2>(p, grid, smem, (cudaStream_t)stream)
                                     : mv::lng::launch_gather<1>(p, grid, smem, (cudaStream_t)stream);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "gather launch");
  }
  const int rb = mv::rows_of_word(T, S, K, 0), step = rb ? rb : 1;
  p.groups = mv::groups_of(rb, K, T, S);
  const int64_t ctas = (K + (int64_t)p.groups * step - 1) / ((int64_t)p.groups * step);
  const int threads = mv::threads_of(S, p.groups);
  const cudaError_t e = mv::dispatch<mv::Gather>(rb, p, dim3((unsigned)ctas, mv::shares_of(ctas, S, p.groups, threads)),
                                                 (size_t)((T + 1) / 2 * 4 * rb * p.groups), (cudaStream_t)stream, threads);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "gather launch");
}

extern "C" nm_status nm_experts_combine(const uint16_t* Yg, int64_t ldg, int64_t S, int64_t R, int64_t T, int k,
                                        const int32_t* slot, const float* gate, void* Y, int64_t ldy, nm_out_dtype y_dtype,
                                        void* stream) {
  set_last_error("");
  nm_status st = mv::check(R, T, k, S);
  if (st != NM_OK) return st;
  if (!dtype_ok(y_dtype)) return fail(NM_ERR_INVALID_ARG, "bad output dtype");
  if (R == 0 || T == 0) return NM_OK;
  if (!slot) return fail(NM_ERR_INVALID_ARG, "slot is null");
  st = S > 0 ? check_matrix(Yg, ldg, S, 2, "Yg") : NM_OK;
  if (st == NM_OK) st = check_matrix(Y, ldy, T, dtype_bytes(y_dtype), "Y");
  if (st == NM_OK) st = check_words({slot, gate}, "slot and gate");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  if (S == 0) {  // no columns: zeros
    const int64_t size = dtype_bytes(y_dtype);
    const cudaError_t e = cudaMemset2DAsync(Y, (size_t)(ldy * size), 0, (size_t)(T * size), (size_t)R, (cudaStream_t)stream);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "zero result");
  }
  mv::Params p{};
  p.in = Yg, p.ldin = ldg, p.cols_in = (int32_t)S;
  p.out = Y, p.ldout = ldy, p.cols_out = (int32_t)T;
  p.rows = (int32_t)R, p.T = (int32_t)T, p.k = k, p.inv_T = mv::inverse(T);
  p.index = slot, p.gate = gate;
  p.out_f32 = y_dtype == NM_OUT_F32;
  p.vec = al16(slot) && al16(gate) && (T % 4 == 0 || k == 1);
  const int64_t beside = 8 * (gate ? 6 : 2) * (int64_t)k;  // bytes a unit
  const mv::lng::Plan plan = mv::lng::plan_of(S, (T + 7) / 8, INT32_MAX, R, beside);
  if (plan.rows) {
    p.status = status_word_ptr();
    if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
    p.depth = plan.depth;
    const dim3 grid(mv::lng::ctas_of(R, plan), (unsigned)plan.ranges);
    const size_t smem = mv::lng::smem_of(p, plan, beside);
    static SmemLimit one, two;
    const cudaError_t e =
        plan.rows == 2
            ? mv::start(mv::lng::combine_kernel<2>, two, grid, smem, p, (cudaStream_t)stream, mv::lng::kThreads)
            : mv::start(mv::lng::combine_kernel<1>, one, grid, smem, p, (cudaStream_t)stream, mv::lng::kThreads);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "combine launch");
  }
  const int rb = mv::rows_of_word(S, T, R, 0), step = rb ? rb : 1;
  p.groups = mv::groups_of(rb, R, S, T);
  const int64_t ctas = (R + (int64_t)p.groups * step - 1) / ((int64_t)p.groups * step);
  const int threads = mv::threads_of(T, p.groups);
  const cudaError_t e = mv::dispatch<mv::Combine>(rb, p, dim3((unsigned)ctas, mv::shares_of(ctas, T, p.groups, threads)),
                                                  (size_t)((S + 1) / 2 * 4 * rb * p.groups), (cudaStream_t)stream, threads);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "combine launch");
}

extern "C" nm_status nm_experts_combine_grad(const uint16_t* dY, int64_t lddy, int64_t R, int64_t T, int k,
                                             const uint16_t* Yg, int64_t ldg, int64_t S, const int32_t* slot,
                                             const int32_t* source, const float* gate, uint16_t* dYg, int64_t lddg,
                                             float* dgate, void* stream) {
  set_last_error("");
  nm_status st = mv::check(R, T, k, S);
  if (st != NM_OK) return st;
  if (T > 0 && (!slot || !dgate)) return fail(NM_ERR_INVALID_ARG, "slot or dgate is null");
  if (S > 0 && !source) return fail(NM_ERR_INVALID_ARG, "source is null");
  if (S > 0 && R > 0) {
    if (T == 0) return fail(NM_ERR_INVALID_ARG, "columns of no tokens");
    st = check_matrix(dY, lddy, T, 2, "dY");
    if (st == NM_OK) st = check_matrix(Yg, ldg, S, 2, "Yg");
    if (st == NM_OK) st = check_matrix(dYg, lddg, S, 2, "dYg");
  }
  if (st == NM_OK) st = check_words({slot, source, gate, dgate}, "slot, source, gate and dgate");
  if (st != NM_OK || T == 0) return st;
  st = require_device();
  if (st != NM_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (S == 0 || R == 0) {
    const cudaError_t e = cudaMemsetAsync(dgate, 0, (size_t)k * T * 4, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "zero gradient");
  }
  mv::Params p{};
  p.in = dY, p.ldin = lddy, p.cols_in = (int32_t)T;
  p.out = dYg, p.ldout = lddg, p.cols_out = (int32_t)S;
  p.rows = (int32_t)R, p.T = (int32_t)T, p.k = k, p.inv_T = mv::inverse(T);
  p.index = source, p.gate = gate;
  p.vec = al16(source);
  p.yg = Yg, p.ldyg = ldg;
  const int64_t units = (S + 7) / 8;
  // Long rows: ranges of the columns that a CTA's threads hold.
  Staged part(s);
  cudaError_t e;
  int64_t ctas, ranges, per;
  const mv::lng::Plan plan = mv::lng::plan_of(T, units, (int64_t)mv::lng::kThreads * mv::lng::kGradUnits, R, 48);
  if (plan.rows) {
    p.status = status_word_ptr();
    if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
    p.depth = plan.depth;
    ctas = mv::lng::ctas_of(R, plan);
    e = part.get((size_t)ctas * units * 32);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the gates' sums");
    p.part = part.as<float>();
    const dim3 grid((unsigned)ctas, (unsigned)plan.ranges);
    const size_t smem = mv::lng::smem_of(p, plan, 48);
    static SmemLimit one, two;
    e = plan.rows == 2 ? mv::start(mv::lng::combine_grad_kernel<2>, two, grid, smem, p, s, mv::lng::kThreads)
                       : mv::start(mv::lng::combine_grad_kernel<1>, one, grid, smem, p, s, mv::lng::kThreads);
  } else if (T <= 128 && units <= 65535ll * mv::kFewThreads) {
    ranges = (units + mv::kFewThreads - 1) / mv::kFewThreads;
    const int64_t lanes = mv::kFewThreads / (units < mv::kFewThreads ? units : mv::kFewThreads);
    ctas = 2 * (int64_t)sm_count_current() / ranges;
    if (ctas > (R + 2 * lanes - 1) / (2 * lanes)) ctas = (R + 2 * lanes - 1) / (2 * lanes);  // two rows a thread at least
    if (ctas < 1) ctas = 1;
    p.groups = (int)((R + ctas - 1) / ctas);
    ctas = (R + p.groups - 1) / p.groups;
    e = part.get((size_t)ctas * units * 32);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the gates' sums");
    p.part = part.as<float>();
    e = launch_pdl(mv::combine_grad_few_kernel, dim3((unsigned)ctas, (unsigned)ranges), dim3(mv::kFewThreads), 0, s, p);
    count_launch();
  } else {
    ranges = (units + 2047) / 2048;  // whose sums take at most 64 KB; up to 128 where the grid's axis ends
    if (ranges > 65535) ranges = 65535;
    per = (units + ranges - 1) / ranges;
    const int rb = mv::rows_of_word(T, kMaxDim, R, 32 * per), step = rb ? rb : 1;
    const int64_t row_groups = (R + step - 1) / step;
    // A few CTAs to an SM (two with the largest tiles), each with as many row groups as that leaves; more of them only write
    // more partial sums.
    ctas = (units <= 256 ? 8 : units <= 512 ? 4 : 2) * (int64_t)sm_count_current() / ranges;
    if (ctas < 1) ctas = 1;
    if (ctas > row_groups) ctas = row_groups;
    p.groups = (int)((row_groups + ctas - 1) / ctas);
    ctas = (row_groups + p.groups - 1) / p.groups;
    e = part.get((size_t)ctas * units * 32);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the gates' sums");
    p.part = part.as<float>();
    e = mv::dispatch<mv::CombineGrad>(rb, p, dim3((unsigned)ctas, (unsigned)ranges),
                                      (size_t)(32 * per + (T + 1) / 2 * 4 * rb), s, units <= 256 ? 256 : mv::kThreads);
  }
  if (e == cudaSuccess) {
    const int64_t n = (int64_t)k * T, most_of = n > S ? n : S;
    e = launch_pdl(mv::dgate_kernel, dim3((unsigned)((most_of + 31) / 32)), dim3(256), 0, s, (const float*)p.part,
                   (int32_t)ctas, units * 8, source, slot, n, (int32_t)S, dgate);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "combine gradient launch");
}
