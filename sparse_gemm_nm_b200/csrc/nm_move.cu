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

// Eight consecutive 32-bit values, `fill` behind the first `valid`.
template <typename V>
__device__ __forceinline__ void load8(const V* p, int valid, bool vec, V fill, V (&v)[8]) {
  if (vec && valid >= 8) {
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p)), b = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const V*>(&w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? __ldcg(p + i) : fill;
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

// The RB elements of column c (outside [0, cols_in): zeros), bf16 pairs.
template <int RB, bool DIRECT>
__device__ __forceinline__ void pick(const Params& p, const typename Word<RB>::type* tile, int64_t row, int32_t c,
                                     uint32_t (&w)[(RB + 1) / 2]) {
  const bool in = (uint32_t)c < (uint32_t)p.cols_in;
  if constexpr (DIRECT) {
    w[0] = in ? (uint32_t)p.in[row * p.ldin + c] : 0u;
  } else if constexpr (RB == 4) {
    const uint2 v = in ? tile[c] : make_uint2(0u, 0u);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = in ? (uint32_t)tile[c] : 0u;
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
  for (int64_t i = threadIdx.x; i < items; i += blockDim.x) {
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
  for (int64_t i = threadIdx.x; i < items; i += blockDim.x) {
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
        const float gate = !live ? 0.f : p.gate ? __ldg(p.gate + src[c]) : 1.f;
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

// dgate[j][t] = the partial sums of column slot[j][t], in order; 0 without a column.
__global__ void __launch_bounds__(256) dgate_kernel(const float* part, int32_t parts, int64_t pitch, const int32_t* slot,
                                                    int64_t n, int32_t S, float* dgate) {
  pdl_gate();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int32_t s = __ldcg(slot + i);
  float sum = 0.f;
  if ((uint32_t)s < (uint32_t)S) {
    int32_t b = 0;
    for (; b + 8 <= parts; b += 8) {
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = __ldcg(part + (b + q) * pitch + s);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum += f[q];
    }
    for (; b < parts; ++b) sum += __ldcg(part + b * pitch + s);
  }
  dgate[i] = sum;
}

static uint32_t inverse(int64_t T) {
  const uint64_t q = (1ull << 32) / (uint64_t)T;
  return q > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)q;
}

// Rows a word holds for rows of `cols` elements (0: picked from global memory), beside `beside` bytes.
static int rows_of_word(int64_t cols, int64_t rows, int64_t beside) {
  const int64_t one = (cols + 1) / 2 * 4;  // bytes of a row
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
static cudaError_t start(Kernel kernel, SmemLimit& limit, dim3 grid, size_t smem, const Params& p, cudaStream_t s) {
  cudaError_t e = limit.raise(kernel, (uint32_t)(208 * 1024));
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, grid, dim3(kThreads), smem, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int RB, bool DIRECT>
struct Gather {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s) {
    static SmemLimit limit;
    return start(gather_kernel<RB, DIRECT>, limit, grid, smem, p, s);
  }
};
template <int RB, bool DIRECT>
struct Combine {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s) {
    static SmemLimit limit;
    return start(combine_kernel<RB, DIRECT>, limit, grid, smem, p, s);
  }
};
template <int RB, bool DIRECT>
struct CombineGrad {
  static cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s) {
    static SmemLimit limit;
    return start(combine_grad_kernel<RB, DIRECT>, limit, grid, smem, p, s);
  }
};

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
  const int rb = mv::rows_of_word(T, K, 0), step = rb ? rb : 1;
  p.groups = mv::groups_of(rb, K, T, S);
  const int64_t ctas = (K + (int64_t)p.groups * step - 1) / ((int64_t)p.groups * step);
  const cudaError_t e = mv::dispatch<mv::Gather>(rb, p, dim3((unsigned)ctas), (size_t)((T + 1) / 2 * 4 * rb * p.groups),
                                                 (cudaStream_t)stream);
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
  mv::Params p{};
  p.in = Yg, p.ldin = ldg, p.cols_in = (int32_t)S;
  p.out = Y, p.ldout = ldy, p.cols_out = (int32_t)T;
  p.rows = (int32_t)R, p.T = (int32_t)T, p.k = k, p.inv_T = mv::inverse(T);
  p.index = slot, p.gate = gate;
  p.out_f32 = y_dtype == NM_OUT_F32;
  p.vec = al16(slot) && al16(gate) && (T % 4 == 0 || k == 1);
  const int rb = mv::rows_of_word(S, R, 0), step = rb ? rb : 1;
  p.groups = mv::groups_of(rb, R, S, T);
  const int64_t ctas = (R + (int64_t)p.groups * step - 1) / ((int64_t)p.groups * step);
  const cudaError_t e = mv::dispatch<mv::Combine>(rb, p, dim3((unsigned)ctas), (size_t)((S + 1) / 2 * 4 * rb * p.groups),
                                                  (cudaStream_t)stream);
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
  if (st == NM_OK) st = require_device();
  if (st != NM_OK || T == 0) return st;
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
  // Columns in ranges whose sums take at most 64 KB.
  const int64_t units = (S + 7) / 8, ranges = (units + 2047) / 2048, per = (units + ranges - 1) / ranges;
  const int rb = mv::rows_of_word(T, R, 32 * per), step = rb ? rb : 1;
  const int64_t row_groups = (R + step - 1) / step;
  // Two CTAs to an SM, each with as many row groups as that leaves; more CTAs only write more partial sums.
  int64_t ctas = 2 * (int64_t)sm_count_current() / ranges;
  if (ctas < 1) ctas = 1;
  if (ctas > row_groups) ctas = row_groups;
  p.groups = (int)((row_groups + ctas - 1) / ctas);
  ctas = (row_groups + p.groups - 1) / p.groups;
  Staged part(s);
  cudaError_t e = part.get((size_t)ctas * units * 32);
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the gates' sums");
  p.part = part.as<float>();
  e = mv::dispatch<mv::CombineGrad>(rb, p, dim3((unsigned)ctas, (unsigned)ranges),
                                    (size_t)(32 * per + (T + 1) / 2 * 4 * rb), s);
  if (e == cudaSuccess) {
    const int64_t n = (int64_t)k * T;
    e = launch_pdl(mv::dgate_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, (const float*)p.part, (int32_t)ctas,
                   units * 8, slot, n, (int32_t)S, dgate);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "combine gradient launch");
}
