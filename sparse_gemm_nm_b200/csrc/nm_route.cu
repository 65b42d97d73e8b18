// nm_route.cu -- the router of a layer of experts: every token's k experts, their gates, and the tokens as columns grouped by
// expert; and the gradient of the gates.
//
// Logits l are E x T (experts x tokens, tokens contiguous).  Per token the k largest in descending order, ties to the lower
// expert, a NaN above every number; -inf is never chosen.  gate[j] = exp(l[e_j]) / sum of exp(l) over the chosen (renorm) or
// over all experts.  Grouped columns: expert by expert, tokens ascending; slot[j][t] is a token's column, source[s] = j T + t
// what column s holds.
//
// route_kernel takes 32 tokens a CTA, a lane each, and splits the experts over its warps, so that 16 tokens are not a chain
// of E loads: every warp keeps its slice's k best in registers (sorted, as order-preserving integers), and a tree of
// two-list merges in shared memory joins the slices.  A word per expert, a bit per token, then gives every chosen pair's
// rank among the 32 tokens by one population count: no atomics whose order matters, no sort.  Each CTA leaves its counts
// (a byte per expert); place_kernel adds up those of the CTAs before, which gives the columns.  With 32 tokens or fewer the
// first kernel does that itself.  Few bytes (16384 tokens of 64 experts: 2 MB): bound by the launches and by latency.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"

namespace nmk {

namespace route {
constexpr int kMaxK = 16;
constexpr int kMaxE = 1024;
constexpr int kWarps = 8;        // slices of the experts, at most
constexpr int kPlaceThreads = 512;
constexpr int kMaxChunk = 16;    // groups of 32 tokens a CTA of place_kernel takes at a time, at most

struct Params {
  const void* logits;
  int64_t ld;
  int32_t E, T, k;
  int renorm;
  int32_t* expert;  // k x T
  float* gate;      // k x T
  int32_t* slot;    // k x T
  int32_t* source;  // k T
  int32_t* offsets; // E + 1
  uint8_t* counts;  // E x pitch: chosen pairs of every expert in every group of 32 tokens
  int32_t groups, pitch;
  int32_t chunk;    // groups a CTA of place_kernel takes at a time, a power of two
  int32_t turns;    // ... and how often
};

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return __ldcg(p); }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)__ldcg(p) << 16); }

// An integer that grows with x: equal for -0 and +0, above all numbers for a NaN, 0x007FFFFF for -inf.
constexpr uint32_t kNegInf = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x != x ? 0xFFFFFFFFu : (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t key) {
  return key == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}

// Exclusive sums of n values in shared memory by the CTA's first warp, the total behind them.
__device__ __forceinline__ void scan_exclusive(int32_t* v, int n, int lane) {
  int32_t base = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int32_t own = i0 + lane < n ? v[i0 + lane] : 0;
    int32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += up;
    }
    if (i0 + lane < n) v[i0 + lane] = base + sum - own;
    base += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  if (lane == 0) v[n] = base;
}

// KT: places of a list (k rounded up to a power of two).
template <typename L, int KT>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const __grid_constant__ Params p) {
  __shared__ uint32_t keys[kWarps][KT][32];
  __shared__ uint16_t ids[kWarps][KT][32];
  __shared__ float sums[kWarps][2][32];
  __shared__ uint32_t mask[kMaxE];
  __shared__ int32_t start[kMaxE + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int32_t t = (int32_t)blockIdx.x * 32 + lane;
  const bool live = t < p.T;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0u;
  pdl_gate();

  // ------------------------------------------- the best of this warp's slice
  uint32_t key[KT];
  uint32_t id[KT];
#pragma unroll
  for (int i = 0; i < KT; ++i) key[i] = kNegInf, id[i] = 0xFFFFu;
  const int e0 = (int)((int64_t)p.E * warp / warps), e1 = (int)((int64_t)p.E * (warp + 1) / warps);
  const L* col = static_cast<const L*>(p.logits) + t;
  // Of the slice: the largest number (not below -FLT_MAX, so that no difference is inf - inf), sum of exp(l - it).
  float top = __uint_as_float(0xFF7FFFFFu), sum = 0.f;
  for (int eb = e0; eb < e1; eb += 8) {
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      l[i] = live && eb + i < e1 ? load_logit<L>(col + (int64_t)(eb + i) * p.ld) : __uint_as_float(0xFF800000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t o = order_key(l[i]);
      if (o > key[KT - 1]) {  // a later expert goes behind an equal one
        uint32_t in = o, in_id = (uint32_t)(eb + i);
        bool up = false;  // once it has its place, the rest moves down one, equals in their order
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          up = up || in > key[j];
          const uint32_t ok = key[j], oi = id[j];
          key[j] = up ? in : ok;
          id[j] = up ? in_id : oi;
          in = up ? ok : in;
          in_id = up ? oi : in_id;
        }
      }
    }
    if (!p.renorm) {
      float m = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, l[i]);
      sum *= expf(top - m);
      top = m;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += expf(l[i] - m);
    }
  }
#pragma unroll
  for (int i = 0; i < KT; ++i) keys[warp][i][lane] = key[i], ids[warp][i][lane] = (uint16_t)id[i];
  sums[warp][0][lane] = top;
  sums[warp][1][lane] = sum;
  __syncthreads();

  // ------------------------------------------------- lists joined two by two
  for (int step = 1; step < warps; step <<= 1) {
    const int other = warp + step;
    const bool joins = (warp & (2 * step - 1)) == 0 && other < warps;
    if (joins) {
      int a = 0, b = 0;
      uint32_t ka = keys[warp][0][lane], kb = keys[other][0][lane];
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const bool second = kb > ka;  // of equals the lower slice's expert
        key[i] = second ? kb : ka;
        id[i] = second ? ids[other][b][lane] : ids[warp][a][lane];
        if (second)
          kb = ++b < KT ? keys[other][b][lane] : 0u;
        else
          ka = ++a < KT ? keys[warp][a][lane] : 0u;
      }
      if (!p.renorm) {
        const float t1 = sums[other][0][lane], s1 = sums[other][1][lane], m = fmaxf(top, t1);
        sum = sum * expf(top - m) + s1 * expf(t1 - m);
        top = m;
      }
    }
    __syncthreads();
    if (joins) {
#pragma unroll
      for (int i = 0; i < KT; ++i) keys[warp][i][lane] = key[i], ids[warp][i][lane] = (uint16_t)id[i];
      sums[warp][0][lane] = top;
      sums[warp][1][lane] = sum;
    }
    __syncthreads();
  }

  // ----------------------------------------------- gates and ranks (warp 0)
  if (warp == 0 && live) {
    const float best = of_key(key[0]);
    float ex[KT], total = 0.f;
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      ex[j] = j < p.k && key[j] > kNegInf ? expf(of_key(key[j]) - best) : 0.f;
      total += ex[j];
    }
    // All experts: the sum was taken against the largest number, which is the best logit unless that is a NaN.
    if (!p.renorm) total = sum;
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      if (j >= p.k) break;
      const bool has = key[j] > kNegInf;
      const int64_t at = (int64_t)j * p.T + t;
      p.expert[at] = has ? (int32_t)id[j] : -1;
      p.gate[at] = ex[j] == 0.f ? 0.f : ex[j] / total;  // beside a logit of +inf the finite ones have 0, not 0 / NaN
      if (has) atomicOr(&mask[id[j]], 1u << lane);
    }
  }
  __syncthreads();
  if (p.groups > 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.counts[(int64_t)e * p.pitch + blockIdx.x] = (uint8_t)__popc(mask[e]);
    if ((int)blockIdx.x == p.groups - 1 && p.pitch > p.groups)  // place_kernel reads whole pieces of 16 groups
      for (int e = threadIdx.x; e < p.E; e += blockDim.x)
        for (int g = p.groups; g < p.pitch; ++g) p.counts[(int64_t)e * p.pitch + g] = 0;
    if (warp == 0 && live) {
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (j < p.k && key[j] > kNegInf)
          p.slot[(int64_t)j * p.T + t] = __popc(mask[id[j]] & ((1u << lane) - 1u));  // place_kernel adds the rest
    }
    return;
  }
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) start[e] = __popc(mask[e]);
  __syncthreads();
  if (warp == 0) scan_exclusive(start, p.E, lane);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = start[e];
  for (int s = start[p.E] + threadIdx.x; s < p.k * p.T; s += blockDim.x) p.source[s] = -1;
  if (warp == 0 && live) {
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      if (j >= p.k) break;
      int32_t s = -1;
      if (key[j] > kNegInf) {
        s = start[id[j]] + __popc(mask[id[j]] & ((1u << lane) - 1u));
        p.source[s] = j * p.T + t;
      }
      p.slot[(int64_t)j * p.T + t] = s;
    }
  }
}

// Columns of the pairs of p.chunk groups of 32 tokens at a time: every expert's pairs in the groups before, its first column,
// and the chunk's own groups, each from the byte counts.  A CTA reads all counts once, so there are no more of them than run
// together, four to an SM: beyond 16 groups for each (303104 tokens) a CTA takes p.turns chunks, one behind the other.  With
// a CTA for every 16 groups the counts read grew with the square of the tokens: 2^26 tokens of two experts 138 ms.
__global__ void __launch_bounds__(kPlaceThreads, 4) place_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t smem[];
  int32_t* start = smem;                   // E + 1: total, then first column of the expert
  int32_t* base = start + p.E + 1;         // E x chunk: pairs of the expert before the group
  int32_t* so_far = base + p.E * p.chunk;  // E: before the next chunk
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = (int)blockIdx.x * p.turns * p.chunk;
  pdl_gate();
  // The pairs of the groups from g0 on, `before` of them before.  A warp an expert.
  auto spread = [&](int e, int g0, int32_t before) {
    const uint8_t* row = p.counts + (int64_t)e * p.pitch;
    const int32_t own = lane < p.chunk && g0 + lane < p.groups ? (int32_t)__ldcg(row + g0 + lane) : 0;
    int32_t sum = own;  // of the chunk's groups up to the lane's
#pragma unroll
    for (int o = 1; o < kMaxChunk; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane < p.chunk) base[e * p.chunk + lane] = before + sum - own;
    if (lane == p.chunk - 1) so_far[e] = before + sum;
  };
  const uint32_t part = (uint32_t)(first & 15);  // groups of the piece of 16 that the chunk starts in
  uint32_t keep[4];                              // their bytes
#pragma unroll
  for (int i = 0; i < 4; ++i)
    keep[i] = part >= 4u * i + 4u ? 0xFFFFFFFFu : part <= 4u * i ? 0u : (1u << (8u * (part - 4u * i))) - 1u;
  for (int e = warp; e < p.E; e += kPlaceThreads / 32) {
    const uint8_t* row = p.counts + (int64_t)e * p.pitch;
    uint32_t all = 0, before = 0;
    for (int i = lane; i < p.pitch / 16; i += 32) {  // bytes behind the last group are zero
      const uint4 u = __ldcg(reinterpret_cast<const uint4*>(row) + i);
      const uint32_t n = __dp4a(u.x, 0x01010101u, __dp4a(u.y, 0x01010101u,
                                __dp4a(u.z, 0x01010101u, __dp4a(u.w, 0x01010101u, 0u))));
      all += n;
      if (i < first / 16)
        before += n;
      else if (i == first / 16)
        before = __dp4a(u.x & keep[0], 0x01010101u, __dp4a(u.y & keep[1], 0x01010101u,
                        __dp4a(u.z & keep[2], 0x01010101u, __dp4a(u.w & keep[3], 0x01010101u, before))));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    }
    spread(e, first, (int32_t)before);
    if (lane == 0) start[e] = (int32_t)all;
  }
  __syncthreads();
  if (warp == 0) scan_exclusive(start, p.E, lane);
  __syncthreads();
  const int shift = 5 + (31 - __clz(p.chunk));  // a row of chunk x 32 tokens for every j
  for (int turn = 0;;) {
    const int g0 = first + turn * p.chunk;
    const int32_t t0 = g0 * 32, tokens = min(p.T - t0, p.chunk * 32);
    for (int i = threadIdx.x; i < p.k << shift; i += kPlaceThreads) {
      const int j = i >> shift, t = i & ((1 << shift) - 1);
      if (t >= tokens) continue;
      const int64_t at = (int64_t)j * p.T + t0 + t;
      const int32_t e = __ldcg(p.expert + at);
      int32_t s = -1;
      if (e >= 0) {
        s = start[e] + base[e * p.chunk + (t >> 5)] + __ldcg(p.slot + at);
        p.source[s] = j * p.T + t0 + t;
      }
      p.slot[at] = s;
    }
    if (++turn == p.turns || g0 + p.chunk >= p.groups) break;
    __syncthreads();  // all are through with this chunk's counts
    for (int e = warp; e < p.E; e += kPlaceThreads / 32) {
      const int32_t before = so_far[e];
      __syncwarp();
      spread(e, g0 + p.chunk, before);
    }
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.E; e += kPlaceThreads) p.offsets[e] = start[e];
  for (int64_t s = start[p.E] + (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x; s < (int64_t)p.k * p.T;
       s += (int64_t)gridDim.x * kPlaceThreads)
    p.source[s] = -1;
}

// ------------------------------------------------------------------ gradient
struct GradParams {
  const void* logits;
  int64_t ld;
  int32_t E, T, k;
  int renorm;
  const int32_t* expert;
  const float *gate, *dgate;
  void* dlogits;
  int64_t ldd;
};

template <typename L>
__device__ __forceinline__ L round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t round_to<uint16_t>(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// dl[e] = p_e ([e chosen] dgate - sum_j gate_j dgate_j), p_e = gate_0 exp(l_e - l_{e_0}) (full softmax) or the gate of a
// chosen e and 0 of the others (renorm).  32 tokens a CTA, a lane each; the warps take the experts' rows.
template <typename L>
__global__ void __launch_bounds__(256) route_grad_kernel(const __grid_constant__ GradParams p) {
  __shared__ uint32_t mask[kMaxE];
  __shared__ int32_t who[kMaxK][32];
  __shared__ float gates[kMaxK][32], part[kMaxK][32];  // gate, gate dgate
  __shared__ float best_of[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int32_t t = (int32_t)blockIdx.x * 32 + lane;
  const bool live = t < p.T;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0u;
  pdl_gate();
  __syncthreads();
  if (live) {
    for (int j = warp; j < p.k; j += warps) {
      const int64_t at = (int64_t)j * p.T + t;
      const int32_t e = __ldcg(p.expert + at);
      const float gate = __ldcg(p.gate + at), d = __ldcg(p.dgate + at);
      const bool has = e >= 0 && e < p.E;  // (another number is no expert's)
      who[j][lane] = has ? e : -1;
      gates[j][lane] = has ? gate : 0.f;
      part[j][lane] = has ? gate * d : 0.f;
      if (has) atomicOr(&mask[e], 1u << lane);
      if (j == 0) best_of[lane] = has ? load_logit<L>(static_cast<const L*>(p.logits) + (int64_t)e * p.ld + t) : 0.f;
    }
  }
  __syncthreads();
  if (!live) return;
  const float best = best_of[lane], g0 = gates[0][lane];
  float dot = 0.f;
  for (int j = 0; j < p.k; ++j) dot += part[j][lane];
  const bool some = who[0][lane] >= 0;  // a token without experts has no gradient
#pragma unroll 4
  for (int e = warp; e < p.E; e += warps) {
    float v = 0.f;
    if (!p.renorm && some) v = -g0 * expf(load_logit<L>(static_cast<const L*>(p.logits) + (int64_t)e * p.ld + t) - best) * dot;
    if (mask[e] >> lane & 1u) {
      for (int j = 0; j < p.k; ++j)
        if (who[j][lane] == e) v += p.renorm ? part[j][lane] - gates[j][lane] * dot : part[j][lane];
    }
    static_cast<L*>(p.dlogits)[(int64_t)e * p.ldd + t] = round_to<L>(v);
  }
}

template <typename L>
static cudaError_t launch_route(const Params& p, int k, int warps, cudaStream_t s) {
  const dim3 grid((unsigned)p.groups), block(32u * (unsigned)warps);
  cudaError_t e = k <= 1   ? launch_pdl(route_kernel<L, 1>, grid, block, 0, s, p)
                  : k <= 2 ? launch_pdl(route_kernel<L, 2>, grid, block, 0, s, p)
                  : k <= 4 ? launch_pdl(route_kernel<L, 4>, grid, block, 0, s, p)
                  : k <= 8 ? launch_pdl(route_kernel<L, 8>, grid, block, 0, s, p)
                           : launch_pdl(route_kernel<L, 16>, grid, block, 0, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Logits are read and written element by element: rows of any stride.
static nm_status check_logits(const void* p, int64_t ld, int64_t T, int dtype, const char* name) {
  if (!p) return fail(NM_ERR_INVALID_ARG, "%s is null", name);
  if (ld < T) return fail(NM_ERR_INVALID_ARG, "ld of %s < T", name);
  if (!aligned_to(p, (uintptr_t)dtype_bytes(dtype))) return fail(NM_ERR_MISALIGNED, "%s is not aligned to its elements", name);
  return NM_OK;
}

static nm_status check(int64_t E, int64_t T, int64_t k) {
  if (E < 0 || T < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (E < 1) return fail(NM_ERR_INVALID_ARG, "no experts to choose from");
  if (k < 1 || k > E) return fail(NM_ERR_INVALID_ARG, "k=%lld is not in 1..E", (long long)k);
  if (E > kMaxE) return fail(NM_ERR_UNSUPPORTED, "more than %d experts", kMaxE);
  if (k > kMaxK) return fail(NM_ERR_UNSUPPORTED, "more than %d experts of a token", kMaxK);
  if (k * T >= kMaxDim - 4096) return fail(NM_ERR_UNSUPPORTED, "k * T must stay below 2^31");
  return NM_OK;
}
}  // namespace route

}  // namespace nmk

using namespace nmk;

extern "C" nm_status nm_experts_route(const void* logits, int64_t ld, nm_out_dtype dtype, int64_t E, int64_t T, int k,
                                      int renorm, int32_t* expert, float* gate, int32_t* slot, int32_t* source,
                                      int32_t* offsets, void* stream) {
  set_last_error("");
  nm_status st = route::check(E, T, k);
  if (st != NM_OK) return st;
  if (!dtype_ok(dtype)) return fail(NM_ERR_INVALID_ARG, "bad logits dtype");
  if (!offsets) return fail(NM_ERR_INVALID_ARG, "offsets is null");
  if (T > 0 && (!expert || !gate || !slot || !source))
    return fail(NM_ERR_INVALID_ARG, "expert, gate, slot or source is null");
  st = T > 0 ? route::check_logits(logits, ld, T, dtype, "logits") : NM_OK;
  if (st == NM_OK) st = check_words({expert, gate, slot, source, offsets}, "expert, gate, slot, source and offsets");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    const cudaError_t e = cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "offsets");
  }
  route::Params p{logits, ld, (int32_t)E, (int32_t)T, k, renorm, expert, gate, slot, source, offsets, nullptr, 0, 0, 1, 1};
  p.groups = (int32_t)((T + 31) / 32);
  p.pitch = (p.groups + 15) / 16 * 16;
  // A CTA reads all counts, so more of them only as long as there are SMs.
  p.chunk = 1;
  while (p.chunk < route::kMaxChunk && p.chunk * sm_count_current() < p.groups) p.chunk *= 2;
  const int32_t chunks = (p.groups + p.chunk - 1) / p.chunk;
  p.turns = (chunks + 4 * sm_count_current() - 1) / (4 * sm_count_current());
  const int warps = E >= 8 * route::kWarps ? route::kWarps : (int)((E + 7) / 8);  // eight experts a slice at least
  Staged counts(s);
  if (p.groups > 1) {
    cudaError_t e = counts.get((size_t)E * p.pitch);
    if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the experts' counts");
    p.counts = counts.as<uint8_t>();
  }
  cudaError_t e = dtype == NM_OUT_F32 ? route::launch_route<float>(p, k, warps, s)
                                      : route::launch_route<uint16_t>(p, k, warps, s);
  if (e == cudaSuccess && p.groups > 1) {
    static SmemLimit limit;
    e = limit.raise(route::place_kernel, 4u * (route::kMaxE * (route::kMaxChunk + 2) + 1));
    if (e == cudaSuccess) {
      e = launch_pdl(route::place_kernel, dim3((unsigned)((chunks + p.turns - 1) / p.turns)), dim3(route::kPlaceThreads),
                     (size_t)4 * (E * (p.chunk + 2) + 1), s, p);
      count_launch();
      if (e == cudaSuccess) e = cudaGetLastError();
    }
  }
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "router launch");
}

extern "C" nm_status nm_experts_route_grad(const void* logits, int64_t ld, nm_out_dtype dtype, int64_t E, int64_t T, int k,
                                           int renorm, const int32_t* expert, const float* gate, const float* dgate,
                                           void* dlogits, int64_t lddl, void* stream) {
  set_last_error("");
  nm_status st = route::check(E, T, k);
  if (st != NM_OK) return st;
  if (!dtype_ok(dtype)) return fail(NM_ERR_INVALID_ARG, "bad logits dtype");
  if (T == 0) return NM_OK;
  if (!expert || !gate || !dgate) return fail(NM_ERR_INVALID_ARG, "expert, gate or dgate is null");
  st = route::check_logits(logits, ld, T, dtype, "logits");
  if (st == NM_OK) st = route::check_logits(dlogits, lddl, T, dtype, "dlogits");
  if (st == NM_OK) st = check_words({expert, gate, dgate}, "expert, gate and dgate");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  const route::GradParams p{logits, ld, (int32_t)E, (int32_t)T, k, renorm, expert, gate, dgate, dlogits, lddl};
  const dim3 grid((unsigned)((T + 31) / 32)), block(256);
  cudaError_t e = dtype == NM_OUT_F32 ? launch_pdl(route::route_grad_kernel<float>, grid, block, 0, (cudaStream_t)stream, p)
                                      : launch_pdl(route::route_grad_kernel<uint16_t>, grid, block, 0, (cudaStream_t)stream, p);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "router gradient launch");
}
