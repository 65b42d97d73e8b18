// nm_clip.cu -- the norm over many gradients at once, and their scaling to a largest norm:
//   norm = sqrt(sum over tensors of sum g^2),   out = g max_norm / norm where norm > max_norm, else g.
//
// Bound by memory: every gradient is read twice and written once (the factor needs all of them).  The tensors' addresses and
// sizes travel as kernel parameters, so a captured call holds no host memory and tables need no copy; both passes walk one
// list of pieces of 16384 elements over a persistent grid, the second from its end, where the first has left what L2 holds.
// Squares are added in fp32 over the 32 elements that a thread loads at a time and in 64 bits from there on.  Where the 32
// add up to less than 1e-25 or more than 1e30 they are squared again in 64 bits: above 1e-25, squares below 2^-126 (1.2e-38),
// which fp32 has in fewer bits or not at all, are 4e-12 of the sum together, and below 1e30 none has overflown.
// Every CTA leaves one sum, and each CTA of the second pass adds them up in the same order, so results repeat bit for bit.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <memory>
#include <new>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace clip {
constexpr int kThreads = 256;
constexpr int kCtasPerSm = 6;
constexpr int64_t kPiece = 16384;  // elements

struct Tensor {
  const void* in;
  void* out;
  int64_t n;
  int32_t piece;  // its first piece
  int32_t f32;
};
template <int N>
struct Params {
  Tensor t[N];
  int32_t count, pieces;
  double* sums;       // this launch's, one a CTA
  const double* all;  // second pass: of every launch, or (behind the pass's first launch) what that has made of them
  int32_t num_all;
  float max_norm;
  float* norm;        // set in the launch that writes it,
  double* total;      // ... with the sum of all
};

template <int N>
__device__ __forceinline__ int tensor_of(const Params<N>& p, int32_t piece) {
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].piece <= piece)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Sum of the squares of the elements in NV 16-byte units.
template <bool F32, int NV>
__device__ __forceinline__ double squares(const uint4 (&u)[NV]) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        s[j] = fmaf(__uint_as_float(w[j]), __uint_as_float(w[j]), s[j]);
      } else {
        const float2 f = pair_of(w[j]);
        s[j] = fmaf(f.x, f.x, fmaf(f.y, f.y, s[j]));
      }
    }
  }
  const float c = (s[0] + s[1]) + (s[2] + s[3]);
  if (c > 1e-25f && c < 1e30f) return (double)c;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) any |= u[i].x | u[i].y | u[i].z | u[i].w;
  if (any == 0u) return 0.;
  double d = 0.;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        const double x = (double)__uint_as_float(w[j]);
        d = fma(x, x, d);
      } else {
        const float2 f = pair_of(w[j]);
        d = fma((double)f.x, (double)f.x, fma((double)f.y, (double)f.y, d));
      }
    }
  }
  return d;
}

template <bool F32>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

template <bool F32>
__device__ __forceinline__ void store_element(void* p, int64_t i, float x) {
  if (F32)
    static_cast<float*>(p)[i] = x;
  else
    static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <bool F32>
__device__ double piece_squares(const Tensor& t, int64_t a, int64_t b) {
  constexpr int kPer = F32 ? 4 : 8;
  double d = 0.;
  int64_t i = a;
  if ((reinterpret_cast<uintptr_t>(t.in) & 15) == 0) {
    const uint4* v = reinterpret_cast<const uint4*>(t.in);
    const int64_t end = b / kPer;  // whole units
    int64_t k = a / kPer + threadIdx.x;
    for (; k + 3 * kThreads < end; k += 4 * kThreads) {
      const uint4 u[4] = {v[k], v[k + kThreads], v[k + 2 * kThreads], v[k + 3 * kThreads]};
      d += squares<F32, 4>(u);
    }
    for (; k < end; k += kThreads) {
      const uint4 u[1] = {v[k]};
      d += squares<F32, 1>(u);
    }
    i = end * kPer;
  }
  for (i += threadIdx.x; i < b; i += kThreads) {
    const double x = (double)element<F32>(t.in, i);
    d = fma(x, x, d);
  }
  return d;
}

// Sum over the CTA, in every thread.
__device__ __forceinline__ double cta_sum(double d, double* scratch) {
#pragma unroll
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) d += scratch[w];
  return d;
}

template <int N>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ Params<N> p) {
  __shared__ double scratch[kThreads / 32];
  pdl_gate();
  double d = 0.;
  for (int32_t c = blockIdx.x; c < p.pieces; c += gridDim.x) {
    const Tensor& t = p.t[tensor_of(p, c)];
    const int64_t a = (int64_t)(c - t.piece) * kPiece, b = a + kPiece < t.n ? a + kPiece : t.n;
    d += t.f32 ? piece_squares<true>(t, a, b) : piece_squares<false>(t, a, b);
  }
  d = cta_sum(d, scratch);
  if (threadIdx.x == 0) p.sums[blockIdx.x] = d;
}

template <bool F32>
__device__ __forceinline__ uint4 scaled(uint4 u, float f) {
  if (F32)
    return make_uint4(__float_as_uint(__uint_as_float(u.x) * f), __float_as_uint(__uint_as_float(u.y) * f),
                      __float_as_uint(__uint_as_float(u.z) * f), __float_as_uint(__uint_as_float(u.w) * f));
  const float2 a = pair_of(u.x), b = pair_of(u.y), c = pair_of(u.z), d = pair_of(u.w);
  return make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(b.x * f, b.y * f), pack_bf16x2(c.x * f, c.y * f),
                    pack_bf16x2(d.x * f, d.y * f));
}

template <bool F32>
__device__ void piece_scale(const Tensor& t, int64_t a, int64_t b, float f) {
  constexpr int kPer = F32 ? 4 : 8;
  int64_t i = a;
  if (((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) & 15) == 0) {
    const uint4* v = reinterpret_cast<const uint4*>(t.in);
    uint4* o = reinterpret_cast<uint4*>(t.out);
    const int64_t end = b / kPer;
    int64_t k = a / kPer + threadIdx.x;
    for (; k + 3 * kThreads < end; k += 4 * kThreads) {
      const uint4 u[4] = {v[k], v[k + kThreads], v[k + 2 * kThreads], v[k + 3 * kThreads]};
#pragma unroll
      for (int q = 0; q < 4; ++q) o[k + q * kThreads] = scaled<F32>(u[q], f);
    }
    for (; k < end; k += kThreads) o[k] = scaled<F32>(v[k], f);
    i = end * kPer;
  }
  for (i += threadIdx.x; i < b; i += kThreads) store_element<F32>(t.out, i, element<F32>(t.in, i) * f);
}

// A factor below the smallest normal float, which fp32 holds in fewer bits or as zero: the product in 64 bits.
template <bool F32>
__device__ void piece_scale_tiny(const Tensor& t, int64_t a, int64_t b, double f) {
  for (int64_t i = a + threadIdx.x; i < b; i += kThreads)
    store_element<F32>(t.out, i, (float)((double)element<F32>(t.in, i) * f));
}

template <int N>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Params<N> p) {
  __shared__ double scratch[kThreads / 32];
  pdl_gate();
  double d = 0.;
  for (int i = threadIdx.x; i < p.num_all; i += kThreads) d += __ldcg(p.all + i);
  d = cta_sum(d, scratch);
  const double norm = sqrt(d);
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) {
    *p.norm = (float)norm;
    *p.total = d;
  }
  // A norm that is no number or infinite, as the caller sees it in fp32, scales nothing.
  const bool scales = norm > (double)p.max_norm && (float)norm <= FLT_MAX;
  const double factor = scales ? (double)p.max_norm / norm : 1.;
  const float f = (float)factor;
  const bool tiny = f < FLT_MIN && factor > 0.;
  for (int32_t c = p.pieces - 1 - (int32_t)blockIdx.x; c >= 0; c -= gridDim.x) {
    const Tensor& t = p.t[tensor_of(p, c)];
    if (t.out == nullptr || (f == 1.f && t.out == t.in)) continue;
    const int64_t a = (int64_t)(c - t.piece) * kPiece, b = a + kPiece < t.n ? a + kPiece : t.n;
    if (tiny)
      t.f32 ? piece_scale_tiny<true>(t, a, b, factor) : piece_scale_tiny<false>(t, a, b, factor);
    else if (t.f32)
      piece_scale<true>(t, a, b, f);
    else
      piece_scale<false>(t, a, b, f);
  }
}

template <int N>
static nm_status run(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes, int64_t count,
                     float max_norm, float* norm, cudaStream_t s) {
  const int grid = kCtasPerSm * sm_count_current();
  const int64_t launches = count > 0 ? (count + N - 1) / N : 1;
  Staged sums(s);
  const int64_t num_all = launches * grid;
  cudaError_t e = sums.get((size_t)(num_all + 1) * 8);
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the sums of squares");
  for (int pass = 0; pass < 2; ++pass) {
    // The second pass takes the launches' tensors from the last to the first, as it does their pieces.
    for (int64_t k = 0; k < launches; ++k) {
      const int64_t l = pass ? launches - 1 - k : k;
      Params<N> p;
      p.count = 0;
      int64_t pieces = 0;
      for (int64_t i = l * N; i < count && i < (l + 1) * N; ++i) {
        if (sizes[i] == 0) continue;
        p.t[p.count++] = Tensor{grads[i], outs ? outs[i] : nullptr, sizes[i], (int32_t)pieces, dtypes[i] == NM_OUT_F32};
        pieces += (sizes[i] + kPiece - 1) / kPiece;
        if (pieces >= kMaxDim - grid) return fail(NM_ERR_UNSUPPORTED, "too many elements");
      }
      p.pieces = pass && !outs ? 0 : (int32_t)pieces;  // the norm alone: nothing to walk through
      p.sums = sums.as<double>(l * grid * 8);
      // Only the pass's first launch adds all sums up: every launch's CTAs reading those of every launch would be reads
      // with the square of the gradients (204800 of one element: 58 ms, now the 31 that the host takes).
      p.all = sums.as<double>(k == 0 ? 0 : num_all * 8);
      p.num_all = k == 0 ? (int32_t)num_all : 1;
      p.total = sums.as<double>(num_all * 8);
      p.max_norm = max_norm;
      p.norm = k == 0 ? norm : nullptr;
      if (pass && !outs && k > 0) break;  // the norm alone
      if (!pass) {
        e = launch_pdl(square_kernel<N>, dim3((unsigned)grid), dim3(kThreads), 0, s, p);
      } else {
        const int64_t ctas = !outs || pieces < 1 ? 1 : pieces < grid ? pieces : grid;
        e = launch_pdl(scale_kernel<N>, dim3((unsigned)ctas), dim3(kThreads), 0, s, p);
      }
      count_launch();
      if (e == cudaSuccess) e = cudaGetLastError();
      if (e != cudaSuccess) return cuda_fail(e, "gradient norm launch");
    }
  }
  return NM_OK;
}

// An output that is also another gradient or its output would be scaled twice, or by two CTAs at once.
static nm_status check_outs(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes,
                            int64_t count) {
  struct Range {
    uintptr_t from, to;
    bool out;
  };
  const std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)count + 1]);
  if (!r) return fail(NM_ERR_CUDA, "no host memory for %lld ranges", (long long)count);
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    const uintptr_t g = (uintptr_t)grads[i], o = (uintptr_t)outs[i], bytes = (uintptr_t)(sizes[i] * dtype_bytes(dtypes[i]));
    if (bytes == 0) continue;
    r[n++] = Range{o, o + bytes, true};
    if (g != o) r[n++] = Range{g, g + bytes, false};
  }
  const auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
  if (!std::is_sorted(r.get(), r.get() + n, before)) std::sort(r.get(), r.get() + n, before);
  uintptr_t any = 0, out = 0;  // ends of the ranges so far
  for (int64_t i = 0; i < n; ++i) {
    if (r[i].from < (r[i].out ? any : out)) return fail(NM_ERR_INVALID_ARG, "an output overlaps another gradient or output");
    any = std::max(any, r[i].to);
    if (r[i].out) out = std::max(out, r[i].to);
  }
  return NM_OK;
}
}  // namespace clip

}  // namespace nmk

using namespace nmk;

extern "C" nm_status nm_clip_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes,
                                   int64_t count, float max_norm, float* norm, void* stream) {
  set_last_error("");
  if (count < 0) return fail(NM_ERR_INVALID_ARG, "negative count");
  if (!(max_norm >= 0.f)) return fail(NM_ERR_INVALID_ARG, "max_norm must not be negative");
  if (!norm) return fail(NM_ERR_INVALID_ARG, "norm is null");
  if (count > 0 && (!grads || !sizes || !dtypes)) return fail(NM_ERR_INVALID_ARG, "grads, sizes or dtypes is null");
  nm_status st = check_words({norm}, "norm");
  if (st != NM_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    if (!dtype_ok(dtypes[i])) return fail(NM_ERR_INVALID_ARG, "bad dtype of gradient %lld", (long long)i);
    if (sizes[i] < 0) return fail(NM_ERR_INVALID_ARG, "negative size of gradient %lld", (long long)i);
    if (sizes[i] > 0 && (!grads[i] || (outs && !outs[i])))
      return fail(NM_ERR_INVALID_ARG, "gradient %lld or its output is null", (long long)i);
    const uintptr_t a = (uintptr_t)dtype_bytes(dtypes[i]);
    if (!aligned_to(grads[i], a) || (outs && !aligned_to(outs[i], a)))
      return fail(NM_ERR_MISALIGNED, "gradient %lld is not aligned to its elements", (long long)i);
  }
  if (count >= kMaxDim / 64) return fail(NM_ERR_UNSUPPORTED, "too many gradients");
  if (outs) st = clip::check_outs(grads, outs, sizes, dtypes, count);
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  return count <= 64 ? clip::run<64>(grads, outs, sizes, dtypes, count, max_norm, norm, (cudaStream_t)stream)
                     : clip::run<640>(grads, outs, sizes, dtypes, count, max_norm, norm, (cudaStream_t)stream);
}
