// nm_lora.cu -- low-rank adapters of many requests beside the shared pruned
// projection: y_t = (W' Pi) x_t + s_a B_a (A_a x_t), a the adapter of token t.
//
// Three products, each over tiles of 64 tokens, on the warp-level bf16 MMA
// (m16n8k16): with ranks of 8 to 128 they move far more bytes than they
// multiply, so operand streaming bounds them and not the tensor pipe.
//   shrink   S[t] = A_a x_t          (and U[t] = B_a^T dy_t in the backward pass)
//   expand   Y = base + s_a B_a S    (and dX = base + s_a A_a^T U)
//   outer    dB_a = s_a sum_t dy_t S[t]^T,  dA_a = s_a sum_t U[t] x_t^T
// A tile lists the distinct adapters of its tokens and takes them one after the
// other; a product for adapter a is kept only in the columns of a's tokens (a
// select, not a multiplication by 0), so an Inf or NaN of one request reaches no
// other request.  Requests side by side have one or two adapters in a tile;
// tokens in any order, up to 64.
// S and U stay fp32 in memory.  As MMA operands they are split into two bf16
// terms (three for fp32 results): 2^-17 (2^-25) of a value is lost instead of
// the 2^-9 of one rounding.  Sums over a reduction leave the MMA accumulator
// every 128 steps and add up in fp32 registers, since the accumulator
// truncates; the CTAs of a cluster share a reduction and join in rank order, so
// results repeat bit for bit.
#include <cstdint>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_lora.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace lora {
constexpr int kThreads = 256;
constexpr int kDepth = 128;      // reduction steps of a shrink stage
constexpr int kRankBlock = 32;   // rank rows of a shrink work item
constexpr int kStages = 3;
constexpr uint32_t kZBytes = kDepth * kTok * 2;
constexpr uint32_t kMBytes = kRankBlock * kDepth * 2;
constexpr uint32_t kShrinkPart = 2 * kRankBlock * (kTok + 1) * 4;
constexpr uint32_t kShrinkSmem = kStages * (kZBytes + kMBytes) + kShrinkPart;
constexpr int kRows = 128;       // rows of an expand or outer tile
constexpr int kOuterRank = 64;   // rank columns of an outer work item
constexpr int kOuterStages = 4;
constexpr uint32_t kOuterM = kRows * kTok * 2;
constexpr uint32_t kOuterV = kTok * kOuterRank * 2;  // one bf16 term
constexpr uint32_t kOuterSmem = kOuterStages * kOuterM + 3 * kOuterV;
static_assert(kRows * (kOuterRank + 1) * 4 <= kOuterStages * kOuterM, "the joined sums reuse the stages");

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Sixteen bytes (eight bf16) of a row into shared memory, zeros from element `valid` on (valid may be <= 0).
// Rows that do not start on 16 bytes (vec = 0) are read element by element.
__device__ __forceinline__ void stage16(uint8_t* dst, const uint16_t* src, int64_t valid, int vec) {
  const int v = valid < 0 ? 0 : valid > 8 ? 8 : (int)valid;
  if (vec) {
    cp_async_16(dst, src, (uint32_t)(2 * v));
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < v) w[j >> 1] |= (uint32_t)__ldg(src + j) << (16 * (j & 1));
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The tile's token adapters (-1: none) and the distinct ones in order of first appearance; all threads call it.
__device__ __forceinline__ int tile_adapters(const int32_t* adapter, int64_t n, int64_t t0, int64_t T, int32_t* s_id,
                                             int32_t* s_list, int* s_count) {
  const int tid = threadIdx.x;
  int32_t id = -1;
  if (tid < kTok) {
    if (adapter && t0 + tid < T) id = __ldg(adapter + t0 + tid);
    if (id < 0 || (int64_t)id >= n) id = -1;
    s_id[tid] = id;
  }
  __syncthreads();
  unsigned firsts = 0;
  bool first = false;
  if (tid < kTok) {
    first = id >= 0;
    for (int j = 0; j < tid; ++j)
      if (s_id[j] == id) first = false;
    firsts = __ballot_sync(0xFFFFFFFFu, first);
    if ((tid & 31) == 0) s_count[tid >> 5] = __popc(firsts);
  }
  __syncthreads();
  if (first) s_list[(tid >= 32 ? s_count[0] : 0) + __popc(firsts & ((1u << (tid & 31)) - 1u))] = id;
  __syncthreads();
  return s_count[0] + s_count[1];
}

// The bf16 terms of v: term p is the rounding of what the terms before it left over.
template <int P>
__device__ __forceinline__ void split_terms(float v, uint16_t (&term)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t b = pack_bf16x2(v, 0.f) & 0xFFFFu;
    term[p] = (uint16_t)b;
    v -= __uint_as_float(b << 16);
  }
}
}  // namespace lora

template <bool TRANS>
__global__ void __launch_bounds__(lora::kThreads) lora_shrink_kernel(const LoraShrink p) {
  using namespace lora;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_id[kTok], s_list[kTok];
  __shared__ int s_count[2];
  float* s_part = reinterpret_cast<float*>(smem + kStages * (kZBytes + kMBytes));  // [K half][32 ranks][65]
  pdl_gate();
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster;
  const int64_t t0 = (int64_t)(blockIdx.x / C) * kTok;
  const int distinct = tile_adapters(p.adapter, p.n, t0, p.T, s_id, s_list, s_count);
  const int rblocks = (p.rank + kRankBlock - 1) / kRankBlock;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = warp & 1, group = warp >> 1;  // K half of a stage, group of 16 tokens
  const int rs = (p.rank + 15) / 16 * 16;
  const int64_t chunks = (p.D + kDepth - 1) / kDepth;
  const int64_t mine = chunks > rank ? (chunks - rank + C - 1) / C : 0;  // chunks rank, rank + C, ...

  for (int item = blockIdx.y; item < distinct * rblocks; item += gridDim.y) {
    const int32_t a = s_list[item / rblocks];
    const int j0 = (item % rblocks) * kRankBlock;
    auto load = [&](int64_t i) {
      uint8_t* z = smem + (i % kStages) * (kZBytes + kMBytes);
      uint8_t* m = z + kZBytes;
      const int64_t d0 = (rank + i * C) * kDepth;
#pragma unroll
      for (int u = tid; u < kDepth * 8; u += kThreads) {  // 128 rows of eight 16-byte units
        const int row = u >> 3, c = u & 7;
        const int64_t d = d0 + row;
        const int64_t valid = d < p.D ? p.T - (t0 + 8 * c) : 0;
        cp_async_16(z + row * 128 + ((c ^ (row & 7)) << 4), valid > 0 ? p.Z + d * p.ldz + t0 + 8 * c : p.Z,
                    (uint32_t)(2 * (valid < 0 ? 0 : valid > 8 ? 8 : valid)));
      }
#pragma unroll
      for (int u = tid; u < kRankBlock * 16; u += kThreads) {
        if (!TRANS) {  // 32 rank rows of sixteen units
          const int j = u >> 4, c = u & 15;
          const int64_t valid = j0 + j < p.rank ? p.D - (d0 + 8 * c) : 0;
          const uint16_t* src = p.M + ((int64_t)a * p.rank + j0 + j) * p.D + d0 + 8 * c;
          stage16(m + j * 256 + ((c ^ (j & 7)) << 4), valid > 0 ? src : p.M, valid, p.vec);
        } else {  // 128 reduction rows of four units
          const int row = u >> 2, c = u & 3;
          const int64_t valid = d0 + row < p.D ? p.rank - (j0 + 8 * c) : 0;
          const uint16_t* src = p.M + ((int64_t)a * p.D + d0 + row) * p.rank + j0 + 8 * c;
          stage16(m + row * 64 + ((c ^ ((row >> 1) & 3)) << 4), valid > 0 ? src : p.M, valid, p.vec);
        }
      }
    };
    bool active = false;  // does any of this warp's 16 tokens use the adapter?
    for (int j = 0; j < 16; ++j) active |= s_id[16 * group + j] == a;

    float sum[2][2][4] = {};
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < mine) load(i);
      cp_commit();
    }
    for (int64_t i = 0; i < mine; ++i) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (i + kStages - 1 < mine) load(i + kStages - 1);
      cp_commit();
      if (!active) continue;
      const uint32_t z = smem_u32(smem + (i % kStages) * (kZBytes + kMBytes)), m = z + kZBytes;
      float acc[2][2][4] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int ks = 4 * half + q, mi = lane >> 3, l8 = lane & 7;
        uint32_t b[4], w[2][4];
        const int zr = 16 * ks + 8 * (mi & 1) + l8;
        ldmatrix_x4_trans(b, z + zr * 128 + (((2 * group + (mi >> 1)) ^ (zr & 7)) << 4));
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if (!TRANS) {
            const int j = 16 * mt + 8 * (mi & 1) + l8;
            ldmatrix_x4(w[mt], m + j * 256 + (((2 * ks + (mi >> 1)) ^ (j & 7)) << 4));
          } else {
            const int row = 16 * ks + 8 * (mi >> 1) + l8;
            ldmatrix_x4_trans(w[mt], m + row * 64 + (((2 * mt + (mi & 1)) ^ ((row >> 1) & 3)) << 4));
          }
          mma_bf16(acc[mt][0], w[mt], b[0], b[1]);
          mma_bf16(acc[mt][1], w[mt], b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[e >> 3][(e >> 2) & 1][e & 3] += acc[e >> 3][(e >> 2) & 1][e & 3];
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * mt + (lane >> 2) + 8 * (e >> 1), t = 16 * group + 8 * nb + 2 * (lane & 3) + (e & 1);
          s_part[(half * kRankBlock + j) * (kTok + 1) + t] = sum[mt][nb][e];
        }
    __syncthreads();
    if (C > 1) cluster_sync();  // every CTA's sums are written
    for (int e = tid + kThreads * (int)rank; e < kRankBlock * kTok; e += kThreads * C) {
      const int j = e & (kRankBlock - 1), t = e / kRankBlock;
      if (s_id[t] != a || j0 + j >= rs) continue;
      float v = 0.f;
      for (int c = 0; c < C; ++c) {
        const uint32_t at = map_to_cta(smem_u32(s_part + j * (kTok + 1) + t), c);
        v += ld_cluster_f32(at) + ld_cluster_f32(at + kRankBlock * (kTok + 1) * 4);
      }
      p.S[(t0 + t) * rs + j0 + j] = v;
    }
    if (C > 1) cluster_sync();  // the sums may be overwritten, and a CTA may leave
    __syncthreads();
  }
}

template <bool TRANS, int P>
__global__ void __launch_bounds__(lora::kThreads) lora_expand_kernel(const LoraExpand p) {
  using namespace lora;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_id[kTok], s_list[kTok];
  __shared__ int s_count[2];
  pdl_gate();
  const int rs = (p.rank + 15) / 16 * 16;
  const uint32_t pitch = (uint32_t)rs * 2 + 16;  // an odd number of 16-byte units: eight rows miss each other's banks
  const uint32_t m_bytes = TRANS ? (uint32_t)rs * 256u : kRows * pitch;
  uint8_t* s_m = smem;                // two buffers of one adapter's tile
  uint8_t* s_s = smem + 2 * m_bytes;  // P terms of 64 tokens x rs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * kRows, t0 = (int64_t)blockIdx.y * kTok;
  const int distinct = tile_adapters(p.adapter, p.n, t0, p.T, s_id, s_list, s_count);

  auto load = [&](int i) {
    uint8_t* m = s_m + (i & 1) * m_bytes;
    const int64_t a = s_list[i];
    if (!TRANS) {
      const int units = rs / 8;
      for (int u = tid; u < kRows * units; u += kThreads) {
        const int row = u / units, c = u - row * units;
        const int64_t valid = r0 + row < p.rows ? p.rank - 8 * c : 0;
        stage16(m + row * pitch + c * 16, valid > 0 ? p.M + (a * p.rows + r0 + row) * p.rank + 8 * c : p.M, valid, p.vec);
      }
    } else {
      for (int u = tid; u < rs * 16; u += kThreads) {
        const int j = u >> 4, c = u & 15;
        const int64_t valid = j < p.rank ? p.rows - (r0 + 8 * c) : 0;
        stage16(m + j * 256 + ((c ^ (j & 7)) << 4), valid > 0 ? p.M + (a * p.rank + j) * p.rows + r0 + 8 * c : p.M, valid,
                p.vec);
      }
    }
  };
  if (distinct > 0) load(0);
  cp_commit();
  // s_a S of the tile's tokens as P bf16 terms (0 for a token without an adapter, whose S is not written)
  for (int u = tid; u < kTok * rs; u += kThreads) {
    const int t = u / rs, j = u - t * rs;
    const int32_t id = s_id[t];
    const float v = id >= 0 ? __ldcg(p.S + (t0 + t) * rs + j) * (p.scale ? __ldg(p.scale + id) : 1.f) : 0.f;
    uint16_t term[P];
    split_terms<P>(v, term);
#pragma unroll
    for (int q = 0; q < P; ++q)
      *reinterpret_cast<uint16_t*>(s_s + ((uint32_t)q * kTok + t) * pitch + 2 * j) = term[q];
  }

  float acc[8][4] = {};
  for (int i = 0; i < distinct; ++i) {
    if (i + 1 < distinct) load(i + 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const int32_t a = s_list[i];
    const uint32_t m = smem_u32(s_m + (i & 1) * m_bytes);
    uint32_t used = 0;  // pairs of 8-token blocks with a token of the adapter
    {
      const unsigned lo = __ballot_sync(0xFFFFFFFFu, s_id[lane] == a), hi = __ballot_sync(0xFFFFFFFFu, s_id[32 + lane] == a);
      for (int b = 0; b < 2; ++b) {
        if (lo & (0xFFFFu << (16 * b))) used |= 1u << b;
        if (hi & (0xFFFFu << (16 * b))) used |= 4u << b;
      }
    }
    const int mi = lane >> 3, l8 = lane & 7;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (!(used & (1u << b))) continue;
      float d[2][4] = {};
      for (int ks = 0; ks < rs / 16; ++ks) {
        uint32_t w[4];
        if (!TRANS) {
          ldmatrix_x4(w, m + (16 * warp + 8 * (mi & 1) + l8) * pitch + (2 * ks + (mi >> 1)) * 16);
        } else {
          const int j = 16 * ks + 8 * (mi >> 1) + l8;
          ldmatrix_x4_trans(w, m + j * 256 + (((2 * warp + (mi & 1)) ^ (j & 7)) << 4));
        }
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint32_t f[4];  // tokens 0-7 (k 0-7, 8-15), tokens 8-15
          ldmatrix_x4(f, smem_u32(s_s) + ((uint32_t)q * kTok + 16 * b + 8 * (mi >> 1) + l8) * pitch + (2 * ks + (mi & 1)) * 16);
          mma_bf16(d[0], w, f[0], f[1]);
          mma_bf16(d[1], w, f[2], f[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s_id[16 * b + 8 * h + 2 * (lane & 3) + (e & 1)] == a) acc[2 * b + h][e] += d[h][e];
    }
    __syncthreads();
  }

#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + 16 * warp + (lane >> 2) + 8 * h;
    if (row >= p.rows) continue;
    const int64_t brow = p.base_row ? (int64_t)__ldg(p.base_row + row) : row;
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const int64_t t = t0 + 8 * nb + 2 * (lane & 3);
      if (t >= p.T) continue;
      float2 v = make_float2(0.f, 0.f);
      if (brow >= 0) {
        for (int q = 0; q < p.splits; ++q) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(p.base + q * p.split_stride + brow * p.ldb + t));
          v.x += x.x;
          v.y += x.y;
        }
      }
      v.x += acc[nb][2 * h];
      v.y += acc[nb][2 * h + 1];
      if (p.out_f32) {
        float* y = static_cast<float*>(p.Y) + row * p.ldy + t;
        if (t + 1 < p.T)
          *reinterpret_cast<float2*>(y) = v;
        else
          *y = v.x;
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.Y) + row * p.ldy + t;
        const uint32_t w = pack_bf16x2(v.x, v.y);
        if (t + 1 < p.T)
          *reinterpret_cast<uint32_t*>(y) = w;
        else
          *y = (uint16_t)(w & 0xFFFFu);
      }
    }
  }
}

// The tiles that hold tokens of adapter blockIdx.x, ascending, and their number.
__global__ void __launch_bounds__(256) lora_plan_kernel(const int32_t* adapter, int64_t T, int32_t* tiles,
                                                        int32_t* counts) {
  using namespace lora;
  __shared__ int s_warp[8];
  pdl_gate();
  const int32_t a = (int32_t)blockIdx.x;
  const int64_t all = (T + kTok - 1) / kTok;
  int32_t* out = tiles + (int64_t)a * all;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int found = 0;
  for (int64_t base = 0; base < all; base += 256) {
    const int64_t tile = base + threadIdx.x;
    bool has = false;
    if (tile < all)
      for (int64_t t = tile * kTok; t < (tile + 1) * kTok && t < T; ++t) has |= __ldg(adapter + t) == a;
    const unsigned votes = __ballot_sync(0xFFFFFFFFu, has);
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int before = found, total = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    if (has) out[before + __popc(votes & ((1u << lane) - 1u))] = (int32_t)tile;
    found += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) counts[a] = found;
}

template <bool BY_RANK, int P>
__global__ void __launch_bounds__(lora::kThreads) lora_outer_kernel(const LoraOuter p) {
  using namespace lora;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_id[2][kTok];
  uint8_t* s_v = smem + kOuterStages * kOuterM;  // P terms of [64 tokens][64 ranks], swizzled 128-byte rows
  pdl_gate();
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster;
  const int64_t r0 = (int64_t)(blockIdx.x / C) * kRows;
  const int rblocks = (p.rank + kOuterRank - 1) / kOuterRank;
  const int32_t a = (int32_t)(blockIdx.y / rblocks);
  const int j0 = (int)(blockIdx.y % rblocks) * kOuterRank;
  const int rs = (p.rank + 15) / 16 * 16;
  const int cols = rs - j0 < kOuterRank ? rs - j0 : kOuterRank;  // rank columns of this item, a multiple of 16
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* list = p.tiles + (int64_t)a * ((p.T + kTok - 1) / kTok);
  const int count = __ldcg(p.counts + a);
  const int mine = count > (int)rank ? (count - (int)rank + C - 1) / C : 0;  // tiles rank, rank + C, ... of the list

  auto load = [&](int i) {
    uint8_t* m = smem + (i % kOuterStages) * kOuterM;
    const int64_t t0 = (int64_t)__ldcg(list + rank + (int64_t)i * C) * kTok;
#pragma unroll
    for (int u = tid; u < kRows * 8; u += kThreads) {
      const int row = u >> 3, c = u & 7;
      const int64_t valid = r0 + row < p.rows ? p.T - (t0 + 8 * c) : 0;
      cp_async_16(m + row * 128 + ((c ^ (row & 7)) << 4), valid > 0 ? p.Z + (r0 + row) * p.ldz + t0 + 8 * c : p.Z,
                  (uint32_t)(2 * (valid < 0 ? 0 : valid > 8 ? 8 : valid)));
    }
  };
  float sum[8][4] = {};
  for (int i = 0; i < kOuterStages - 1; ++i) {
    if (i < mine) load(i);
    cp_commit();
  }
  for (int i = 0; i < mine; ++i) {
    const int64_t t0 = (int64_t)__ldcg(list + rank + (int64_t)i * C) * kTok;
    if (tid < kTok) s_id[i & 1][tid] = t0 + tid < p.T ? __ldg(p.adapter + t0 + tid) : -1;
    cp_wait<kOuterStages - 2>();
    __syncthreads();  // the stage has landed, the ids are there, and the products of the tile before are done
    if (i + kOuterStages - 1 < mine) load(i + kOuterStages - 1);
    cp_commit();
    for (int u = tid; u < kTok * (cols / 8); u += kThreads) {  // eight ranks of one token at a time
      const int t = u / (cols / 8), c = u - t * (cols / 8);
      uint32_t w[P][4] = {};
      if (s_id[i & 1][t] == a) {
        const float4* src = reinterpret_cast<const float4*>(p.V + (t0 + t) * rs + j0 + 8 * c);
        const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint16_t term[P];
          split_terms<P>(v[e], term);
#pragma unroll
          for (int q = 0; q < P; ++q) w[q][e >> 1] |= (uint32_t)term[q] << (16 * (e & 1));
        }
      }
#pragma unroll
      for (int q = 0; q < P; ++q)
        *reinterpret_cast<uint4*>(s_v + q * kOuterV + t * 128 + ((c ^ (t & 7)) << 4)) =
            make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
    }
    __syncthreads();
    const uint32_t m = smem_u32(smem + (i % kOuterStages) * kOuterM), v = smem_u32(s_v);
    const int mi = lane >> 3, l8 = lane & 7;
    float acc[8][4] = {};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t z[4];
      const int row = 16 * warp + 8 * (mi & 1) + l8;
      ldmatrix_x4(z, m + row * 128 + (((2 * ks + (mi >> 1)) ^ (row & 7)) << 4));
      // other requests' tokens leave the product as zeros of Z too: their Inf or NaN times a 0 of V would stay
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 16 * ks + 8 * h + 2 * (lane & 3);
        const uint32_t keep = (s_id[i & 1][t] == a ? 0xFFFFu : 0u) | (s_id[i & 1][t + 1] == a ? 0xFFFF0000u : 0u);
        z[2 * h] &= keep;
        z[2 * h + 1] &= keep;
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (16 * b >= cols) continue;
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint32_t f[4];
          const int t = 16 * ks + 8 * (mi & 1) + l8;
          ldmatrix_x4_trans(f, v + q * kOuterV + t * 128 + (((2 * b + (mi >> 1)) ^ (t & 7)) << 4));
          mma_bf16(acc[2 * b], z, f[0], f[1]);
          mma_bf16(acc[2 * b + 1], z, f[2], f[3]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) sum[e >> 2][e & 3] += acc[e >> 2][e & 3];
  }
  cp_wait<0>();
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(smem);  // [128 rows][65], over the stages
#pragma unroll
  for (int nb = 0; nb < 8; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s_sum[(16 * warp + (lane >> 2) + 8 * (e >> 1)) * (kOuterRank + 1) + 8 * nb + 2 * (lane & 3) + (e & 1)] = sum[nb][e];
  __syncthreads();
  if (C > 1) cluster_sync();
  const float scale = p.scale ? __ldg(p.scale + a) : 1.f;
  const int part = kRows / C;  // rows that this CTA joins and stores
  const int live = p.rank - j0 < kOuterRank ? p.rank - j0 : kOuterRank;
  for (int e = tid; e < part * live; e += kThreads) {
    const int row = (BY_RANK ? e % part : e / live) + (int)rank * part, j = BY_RANK ? e / part : e % live;
    if (r0 + row >= p.rows) continue;
    float v = 0.f;
    for (int c = 0; c < C; ++c) v += ld_cluster_f32(map_to_cta(smem_u32(s_sum + row * (kOuterRank + 1) + j), c));
    v *= scale;
    const int64_t at = BY_RANK ? ((int64_t)a * p.rank + j0 + j) * p.rows + r0 + row
                               : ((int64_t)a * p.rows + r0 + row) * p.rank + j0 + j;
    if (p.out_f32)
      static_cast<float*>(p.out)[at] = v;
    else
      static_cast<uint16_t*>(p.out)[at] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another still reads its sums
}

__global__ void __launch_bounds__(256) invert_clear_kernel(int64_t K, int32_t* inv) {
  pdl_gate();
  const int64_t k = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (k < K) inv[k] = -1;
}
__global__ void __launch_bounds__(256) invert_map_kernel(const int32_t* idx, int64_t K, int32_t* inv) {
  pdl_gate();
  const int64_t k = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (k >= K) return;
  const int32_t j = __ldg(idx + k);
  if (j >= 0 && (int64_t)j < K) atomicMax(inv + j, (int32_t)k);
}

template <typename Kern, typename Params>
static cudaError_t launch_clustered(Kern kernel, dim3 grid, int cluster, uint32_t smem, uint32_t smem_limit,
                                    const Params& p, cudaStream_t s) {
  // Always the kernel's largest request: calls from several host threads set no smaller limit meanwhile.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_limit);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(lora::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_shrink(LoraShrink& p, bool trans, cudaStream_t s) {
  using namespace lora;
  const int64_t tiles = tiles_of(p.T), chunks = (p.D + kDepth - 1) / kDepth;
  const int64_t target = 2 * (int64_t)sm_count_current();
  // The CTAs of a cluster share the reduction until the grid fills the SMs twice over (two stages each at least)
  p.cluster = 1;
  while (p.cluster < 8 && tiles * p.cluster < target && chunks / (2 * p.cluster) >= 2) p.cluster <<= 1;
  // ... and further CTAs take the tile's adapters side by side when the tiles are few
  const int64_t items = (p.n < kTok ? p.n : kTok) * ((p.rank + kRankBlock - 1) / kRankBlock);
  int64_t y = (target + tiles * p.cluster - 1) / (tiles * p.cluster);
  if (y > items) y = items;
  if (y < 1) y = 1;
  if (tiles * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(tiles * p.cluster), (unsigned)y);
  return trans ? launch_clustered(lora_shrink_kernel<true>, grid, p.cluster, kShrinkSmem, kShrinkSmem, p, s)
               : launch_clustered(lora_shrink_kernel<false>, grid, p.cluster, kShrinkSmem, kShrinkSmem, p, s);
}

cudaError_t launch_lora_expand(const LoraExpand& p, bool trans, cudaStream_t s) {
  using namespace lora;
  const int64_t tiles = tiles_of(p.T), blocks = (p.rows + kRows - 1) / kRows;
  if (tiles > 65535) return cudaErrorInvalidValue;
  const uint32_t rs = (uint32_t)rank_stride(p.rank);
  const uint32_t terms = p.out_f32 ? 3 : 2;
  auto bytes = [&](uint32_t r) { return 2 * (trans ? r * 256u : kRows * (r * 2 + 16)) + terms * kTok * (r * 2 + 16); };
  const dim3 grid((unsigned)blocks, (unsigned)tiles);
  const uint32_t b = bytes(rs), most = bytes(kMaxRank);
  if (trans)
    return p.out_f32 ? launch_clustered(lora_expand_kernel<true, 3>, grid, 1, b, most, p, s)
                     : launch_clustered(lora_expand_kernel<true, 2>, grid, 1, b, most, p, s);
  return p.out_f32 ? launch_clustered(lora_expand_kernel<false, 3>, grid, 1, b, most, p, s)
                   : launch_clustered(lora_expand_kernel<false, 2>, grid, 1, b, most, p, s);
}

cudaError_t launch_lora_plan(const int32_t* adapter, int64_t T, int64_t n, int32_t* tiles, int32_t* counts,
                             cudaStream_t s) {
  cudaError_t e = launch_pdl(lora_plan_kernel, dim3((unsigned)n), dim3(256), 0, s, adapter, T, tiles, counts);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_outer(LoraOuter& p, bool by_rank, cudaStream_t s) {
  using namespace lora;
  const int64_t blocks = (p.rows + kRows - 1) / kRows, tiles = tiles_of(p.T);
  const int64_t items = p.n * ((p.rank + kOuterRank - 1) / kOuterRank);
  if (blocks == 0 || items == 0) return cudaSuccess;
  if (items > 65535) return cudaErrorInvalidValue;
  // CTAs that share an adapter's tokens, until the grid fills the SMs
  p.cluster = 1;
  while (p.cluster < 8 && blocks * items * p.cluster < 2 * (int64_t)sm_count_current() && tiles / (2 * p.cluster) >= 2)
    p.cluster <<= 1;
  if (blocks * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * p.cluster), (unsigned)items);
  const uint32_t b = kOuterSmem;
  if (by_rank)
    return p.out_f32 ? launch_clustered(lora_outer_kernel<true, 3>, grid, p.cluster, b, b, p, s)
                     : launch_clustered(lora_outer_kernel<true, 2>, grid, p.cluster, b, b, p, s);
  return p.out_f32 ? launch_clustered(lora_outer_kernel<false, 3>, grid, p.cluster, b, b, p, s)
                   : launch_clustered(lora_outer_kernel<false, 2>, grid, p.cluster, b, b, p, s);
}

cudaError_t launch_invert_map(const int32_t* idx, int64_t K, int32_t* inv, cudaStream_t s) {
  const dim3 grid((unsigned)((K + 255) / 256));
  cudaError_t e = launch_pdl(invert_clear_kernel, grid, dim3(256), 0, s, K, inv);
  count_launch();
  if (e == cudaSuccess) {
    e = launch_pdl(invert_map_kernel, grid, dim3(256), 0, s, idx, K, inv);
    count_launch();
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

namespace {

struct Adapters {
  const uint16_t *A, *B;
  int64_t n;
  int rank;
  const float* scale;
  const int32_t* adapter;
};

nm_status check_adapters(const Adapters& ad) {
  if (ad.n < 0 || ad.rank < 1) return fail(NM_ERR_INVALID_ARG, "num_adapters must be >= 0 and rank >= 1");
  if (ad.rank > lora::kMaxRank) return fail(NM_ERR_UNSUPPORTED, "rank %d is above %d", ad.rank, lora::kMaxRank);
  if (ad.n > 65535 / 2) return fail(NM_ERR_UNSUPPORTED, "more than 32767 adapters in a call");
  return NM_OK;
}
nm_status check_adapter_pointers(const Adapters& ad, int64_t R, int64_t K, int64_t T) {
  if ((!ad.A && K > 0) || (!ad.B && R > 0) || !ad.adapter) return fail(NM_ERR_INVALID_ARG, "A, B or adapter is null");
  if (!aligned_to(ad.A, 2) || !aligned_to(ad.B, 2)) return fail(NM_ERR_MISALIGNED, "A or B misaligned");
  if (lora::tiles_of(T) > 65535) return fail(NM_ERR_UNSUPPORTED, "more than %d tokens in a call", 65535 * lora::kTok);
  return NM_OK;
}

nm_status shrink(const Adapters& ad, bool trans, int64_t D, const uint16_t* Z, int64_t ldz, int64_t T, float* S,
                 cudaStream_t s) {
  LoraShrink p = {};
  p.M = trans ? ad.B : ad.A;
  p.Z = Z;
  p.ldz = ldz;
  p.adapter = ad.adapter;
  p.n = ad.n;
  p.D = D;
  p.T = T;
  p.rank = ad.rank;
  p.vec = al16(p.M) && (trans ? ad.rank : D) % 8 == 0;
  p.S = S;
  cudaError_t e = launch_lora_shrink(p, trans, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter shrink launch");
}

}  // namespace
}  // namespace nmk

using namespace nmk;

extern "C" {

nm_status nm_spmm_lora(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                       const int32_t* idx, const uint16_t* X, int64_t ldx, int64_t T, const uint16_t* A,
                       const uint16_t* B, int rank, int64_t num_adapters, const float* scale, const int32_t* adapter,
                       void* Y, int64_t ldy, nm_out_dtype y_dtype, void* stream) {
  set_last_error("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Adapters ad{A, B, num_adapters, rank, scale, adapter};
  nm_status st = check_adapters(ad);
  if (st == NM_OK) st = check_spmm(values, meta, n, m, R, K, X, ldx, T, Y, ldy, y_dtype);
  if (st != NM_OK || R == 0 || T == 0) return st;
  if (num_adapters == 0 || K == 0)
    return run_spmm(values, meta, n, m, R, K, idx, X, ldx, T, Y, ldy, y_dtype, nullptr, s);
  st = check_adapter_pointers(ad, R, K, T);
  if (st != NM_OK) return st;
  Staged low(s), sum(s), partials(s);
  const int64_t ldb = (T + 3) / 4 * 4;
  cudaError_t e = low.get((size_t)(T * lora::rank_stride(rank) * 4));
  if (e == cudaSuccess) e = sum.get((size_t)(R * ldb * 4));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the projection");
  st = shrink(ad, false, K, X, ldx, T, low.as<float>(), s);
  GemmPartials raw{&partials, 1, 0, 0};
  if (st == NM_OK) st = run_spmm(values, meta, n, m, R, K, idx, X, ldx, T, sum.as<float>(), ldb, NM_OUT_F32, &raw, s);
  if (st != NM_OK) return st;
  LoraExpand p = {};
  p.M = B;
  p.S = low.as<float>();
  p.adapter = adapter;
  p.scale = scale;
  p.n = num_adapters;
  p.rows = R;
  p.T = T;
  p.rank = rank;
  p.vec = al16(B) && rank % 8 == 0;
  p.base = raw.splits > 1 ? partials.as<float>() : sum.as<float>();
  p.splits = raw.splits;
  p.split_stride = raw.split_stride;
  p.ldb = raw.splits > 1 ? raw.ld : ldb;
  p.Y = Y;
  p.ldy = ldy;
  p.out_f32 = y_dtype == NM_OUT_F32;
  e = launch_lora_expand(p, false, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter expand launch");
}

nm_status nm_spmm_lora_t(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                         const int32_t* idx, const uint16_t* dY, int64_t lddy, int64_t T, const uint16_t* A,
                         const uint16_t* B, int rank, int64_t num_adapters, const float* scale,
                         const int32_t* adapter, void* dX, int64_t lddx, nm_out_dtype dtype, void* stream) {
  set_last_error("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Adapters ad{A, B, num_adapters, rank, scale, adapter};
  nm_status st = check_adapters(ad);
  if (st == NM_OK) st = check_spmm_t(values, meta, n, m, R, K, dY, lddy, T, dX, lddx, dtype);
  if (st != NM_OK || K == 0 || T == 0) return st;
  if (R == 0) return run_spmm_t(values, meta, n, m, R, K, nullptr, dY, lddy, T, dX, lddx, dtype, s);
  if (num_adapters > 0) st = check_adapter_pointers(ad, R, K, T);
  if (st != NM_OK) return st;
  Staged low(s), sum(s), inverse(s);
  const int64_t ldb = (T + 3) / 4 * 4;
  cudaError_t e = low.get((size_t)(T * lora::rank_stride(rank) * 4));
  if (e == cudaSuccess) e = sum.get((size_t)(K * ldb * 4));
  if (e == cudaSuccess && idx) e = inverse.get((size_t)(K * 4));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the input gradient");
  if (idx) {
    e = launch_invert_map(idx, K, inverse.as<int32_t>(), s);
    if (e != cudaSuccess) return cuda_fail(e, "index map launch");
  }
  if (num_adapters > 0) st = shrink(ad, true, R, dY, lddy, T, low.as<float>(), s);
  if (st == NM_OK) st = run_spmm_t(values, meta, n, m, R, K, nullptr, dY, lddy, T, sum.as<float>(), ldb, NM_OUT_F32, s);
  if (st != NM_OK) return st;
  LoraExpand p = {};
  p.M = A;
  p.S = low.as<float>();
  p.adapter = adapter;
  p.scale = scale;
  p.n = num_adapters;
  p.rows = K;
  p.T = T;
  p.rank = rank;
  p.vec = al16(A) && K % 8 == 0;
  p.base = sum.as<float>();
  p.splits = 1;
  p.ldb = ldb;
  p.base_row = idx ? inverse.as<int32_t>() : nullptr;
  p.Y = dX;
  p.ldy = lddx;
  p.out_f32 = dtype == NM_OUT_F32;
  e = launch_lora_expand(p, true, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter expand launch");
}

nm_status nm_lora_grad(int64_t R, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                       int64_t T, const uint16_t* A, const uint16_t* B, int rank, int64_t num_adapters,
                       const float* scale, const int32_t* adapter, void* dA, void* dB, nm_out_dtype dtype,
                       void* stream) {
  set_last_error("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Adapters ad{A, B, num_adapters, rank, scale, adapter};
  if (R < 0 || K < 0 || T < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  nm_status st = check_adapters(ad);
  if (st != NM_OK) return st;
  if (!dtype_ok(dtype)) return fail(NM_ERR_INVALID_ARG, "bad output dtype");
  if (R >= kMaxDim || K >= kMaxDim || T >= kMaxDim) return fail(NM_ERR_UNSUPPORTED, "dimensions must stay below 2^31");
  if (num_adapters == 0 || (R == 0 && K == 0)) return NM_OK;
  if (!dA && !dB) return fail(NM_ERR_INVALID_ARG, "dA and dB are both null");
  const int64_t esize = dtype_bytes(dtype);
  if (!aligned_to(dA, esize) || !aligned_to(dB, esize)) return fail(NM_ERR_MISALIGNED, "dA or dB misaligned");
  if (T == 0) {  // empty sums
    st = require_device();
    if (st != NM_OK) return st;
    cudaError_t e = cudaSuccess;
    if (dA && K > 0) e = launch_fill_zero(dA, num_adapters * rank, K, K, (int)esize, s);
    if (e == cudaSuccess && dB && R > 0) e = launch_fill_zero(dB, num_adapters * R, rank, rank, (int)esize, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "zero fill");
  }
  st = check_adapter_pointers(ad, R, K, T);
  if (st == NM_OK && R > 0) st = check_matrix(dY, lddy, T, 2, "dY");
  if (st == NM_OK && K > 0) st = check_matrix(X, ldx, T, 2, "X");
  if (st == NM_OK) st = require_device();
  if (st != NM_OK) return st;
  Staged low(s), up(s), plan(s);
  const size_t bytes = (size_t)(T * lora::rank_stride(rank) * 4);
  const int64_t tiles = lora::tiles_of(T);
  cudaError_t e = plan.get((size_t)((tiles + 1) * num_adapters * 4));
  if (e == cudaSuccess && dB) e = low.get(bytes);
  if (e == cudaSuccess && dA) e = up.get(bytes);
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the adapter gradients");
  LoraOuter p = {};
  p.adapter = adapter;
  p.scale = scale;
  p.n = num_adapters;
  p.T = T;
  p.rank = rank;
  p.counts = plan.as<int32_t>();
  p.tiles = plan.as<int32_t>() + num_adapters;
  p.out_f32 = dtype == NM_OUT_F32;
  e = launch_lora_plan(adapter, T, num_adapters, plan.as<int32_t>() + num_adapters, plan.as<int32_t>(), s);
  if (e != cudaSuccess) return cuda_fail(e, "adapter plan launch");
  if (dB && R > 0) {
    st = shrink(ad, false, K, X, ldx, T, low.as<float>(), s);
    if (st != NM_OK) return st;
    p.Z = dY;
    p.ldz = lddy;
    p.V = low.as<float>();
    p.rows = R;
    p.out = dB;
    e = launch_lora_outer(p, false, s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter gradient launch");
  }
  if (dA && K > 0) {
    st = shrink(ad, true, R, dY, lddy, T, up.as<float>(), s);
    if (st != NM_OK) return st;
    p.Z = X;
    p.ldz = ldx;
    p.V = up.as<float>();
    p.rows = K;
    p.out = dA;
    e = launch_lora_outer(p, true, s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter gradient launch");
  }
  return NM_OK;
}

}  // extern "C"
