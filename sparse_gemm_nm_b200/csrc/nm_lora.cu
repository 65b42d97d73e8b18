// nm_lora.cu -- low-rank adapters of many requests beside the shared pruned
// projection: y_t = (W' Pi) x_t + s_a B_a (A_a x_t), a the adapter of token t.
//
// Three products, each over tiles of 64 tokens:
//   shrink   S[t] = A_a x_t          (and U[t] = B_a^T dy_t in the backward pass)
//   expand   Y = base + s_a B_a S    (and dX = base + s_a A_a^T U)
//   outer    dB_a = s_a sum_t dy_t S[t]^T,  dA_a = s_a sum_t U[t] x_t^T
// With ranks of 8 to 128 they move far more bytes than they multiply.  Shrink and
// expand, whose tiles hold several adapters' tokens in any order, run on the
// warp-level bf16 MMA (m16n8k16), which takes blocks of 16 ranks and 8 tokens;
// outer, whose reduction is the adapter's tokens, on tcgen05 with both operands
// as TMA brings them (128 rows x the terms side by side, up to 3 x 64 columns, so
// that the rows are read from shared memory once for all terms).
// A tile lists the distinct adapters of its tokens and takes them one after the
// other; a product for adapter a is kept only in the columns of a's tokens (a
// select, not a multiplication by 0), so an Inf or NaN of one request reaches no
// other request.  Requests side by side have one or two adapters in a tile;
// tokens in any order, up to 64.
// Where the SM-pair GEMM serves the projection (and for every input gradient),
// the expand product is not a pass of its own: the adapters' second factors
// stand side by side in one matrix, shrink leaves s_a S as blocks that are 0
// outside an adapter's tokens, and the GEMM takes the blocks that a column tile
// uses as further reduction steps, so Y is rounded once and written once.
// S and U are fp32 sums.  As MMA operands they are split into two bf16 terms
// (three for fp32 results): 2^-17 (2^-25) of a value is lost instead of the 2^-9
// of one rounding.  Sums over a reduction leave the MMA accumulator
// every 128 steps and add up in fp32 registers, since the accumulator
// truncates; the CTAs of a cluster share a reduction and join in rank order, so
// results repeat bit for bit.
//
// Measured (floor): 13824 x 5120 x 16 with 16 adapters of rank 16 35 us (14 us
// of weights; shrink 9 us beside the GEMM's 18, expand 8); 4096 x 4096 x 2048, 8 of
// rank 16 57 us (the sparse product alone 35); input gradient 4096 x 11008 x 2048, 2
// of rank 32 169 us (the dense product alone 110, decompression beside the
// shrink; 193 us in a loop under the power cap); gradients 11008 x 4096 x 2048, 4 of rank 64 74 us (13 us of bytes;
// latency of the copies: a CTA has 9 tiles between its first load and its join.
// The outer product on warp-level MMAs, whose fragment loads and thirds of the rate
// of three terms set its time: 95 us).
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "nm_host.h"
#include "nm_internal.h"
#include "nm_lora.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace lora {
constexpr int kThreads = 256;
constexpr int kDepth = 128;      // reduction steps of a shrink stage
constexpr int kMaxStages = 6;
constexpr uint32_t kZBytes = kDepth * kTok * 2;
// A shrink work item takes 32 rank rows, or 64 of a rank above 32 (one reading of Z for them instead of two).
__host__ __device__ constexpr int rank_block(int rank) { return rank > 32 ? 64 : 32; }
__host__ __device__ constexpr uint32_t m_bytes(int rb) { return (uint32_t)(rb * kDepth * 2); }
__host__ __device__ constexpr uint32_t sum_words(int rb) { return (uint32_t)(kTok * (rb + 1) + rb); }  // either layout
__host__ __device__ constexpr uint32_t shrink_smem(int stages, int rb) {
  return (uint32_t)stages * (kZBytes + m_bytes(rb)) + 1024;
}
static_assert(sum_words(32) * 4 <= kZBytes + m_bytes(32) && sum_words(64) * 4 <= kZBytes + m_bytes(64),
              "the sums reuse the first stage");
constexpr int kRows = 128;       // rows of an expand or outer tile
constexpr uint32_t kExpandBatch = 96 * 1024;  // bytes of adapters' tiles in flight
constexpr int kOuterRank = 64;   // rank columns of an outer work item
constexpr uint32_t kOuterM = kRows * kTok * 2;
constexpr uint32_t kOuterV = kTok * kOuterRank * 2;  // one bf16 term
// Two CTAs to an SM, one working while the other waits for copies or joins (tiles of 256 rows, one CTA to an SM with
// four stages: 11008 x 4096 x 2048, 4 of rank 64 took 90 us instead of 74).  Z comes from HBM and has a ring of three
// stages; three terms leave room for two stages of V, which the L2 holds.
constexpr int kOuterZ = 3;
__host__ __device__ constexpr int outer_v(int planes) { return planes == 3 ? 2 : 3; }
__host__ __device__ constexpr uint32_t outer_smem(int planes) {
  return kOuterZ * kOuterM + (uint32_t)(outer_v(planes) * planes) * kOuterV + 1024;
}
constexpr int kOuterPitch = kOuterRank + 4;  // floats of a row of joined sums
constexpr int kOuterGroup = 3;  // tiles whose products one accumulator takes (it truncates): 192 tokens
// Rank columns of a work item as an MMA's N and a box: 16, 32 or 64 (a swizzle's width).
__host__ __device__ constexpr int outer_box(int rank) { return rank > 32 ? 64 : rank > 16 ? 32 : 16; }
static_assert(kRows * kOuterPitch * 4 <= kOuterZ * kOuterM, "the joined sums reuse the stages");
constexpr uint64_t kWaitNs = 2000000000ull;

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
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
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

// The tile's token adapters (-1: none) and the distinct ones, the first half's before the second's; all threads call
// it, the first warp works: matches within each half, then the first half's adapters are struck from the second's.
__device__ __forceinline__ int tile_adapters(const int32_t* adapter, int64_t n, int64_t t0, int64_t T, int32_t* s_id,
                                             int32_t* s_list, int* s_count) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int32_t id[2];
    bool first[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      id[h] = adapter && t0 + 32 * h + lane < T ? __ldg(adapter + t0 + 32 * h + lane) : -1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (id[h] < 0 || (int64_t)id[h] >= n) id[h] = -1;
      s_id[32 * h + lane] = id[h];
      const unsigned same = __match_any_sync(0xFFFFFFFFu, id[h]);  // every lane takes part, those without an adapter too
      first[h] = id[h] >= 0 && __ffs(same) - 1 == lane;
    }
    const unsigned f0 = __ballot_sync(0xFFFFFFFFu, first[0]);
    for (unsigned left = f0; left; left &= left - 1)
      if (__shfl_sync(0xFFFFFFFFu, id[0], __ffs(left) - 1) == id[1]) first[1] = false;
    const unsigned f1 = __ballot_sync(0xFFFFFFFFu, first[1]);
    const unsigned below = (1u << lane) - 1u;
    if (first[0]) s_list[__popc(f0 & below)] = id[0];
    if (first[1]) s_list[__popc(f0) + __popc(f1 & below)] = id[1];
    if (lane == 0) *s_count = __popc(f0) + __popc(f1);
  }
  __syncthreads();
  return *s_count;
}

// The bf16 terms of v: term p is the rounding of what the terms before it left over.
template <int P>
__device__ __forceinline__ void split_terms(float v, uint16_t (&term)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t b = pack_bf16x2(v, 0.f) & 0xFFFFu;
    term[p] = (uint16_t)b;
    v = (b & 0x7F80u) == 0x7F80u ? 0.f : v - __uint_as_float(b << 16);  // nothing is left over of an Inf or NaN
  }
}
}  // namespace lora

template <bool TRANS, int OUT, int P, int RB>
__global__ void __launch_bounds__(lora::kThreads, RB == 32 ? 3 : 2) lora_shrink_kernel(const __grid_constant__ LoraShrink p) {
  using namespace lora;
  constexpr int kRankBlock = RB;
  constexpr int kMT = RB / 16;
  constexpr uint32_t kMBytes = m_bytes(RB);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int32_t s_id[kTok], s_list[kTok];
  __shared__ int s_count, s_abort;
  __shared__ uint32_t s_present[kMaxCat / 32];
  __shared__ uint64_t s_full[kMaxStages];
  float* s_part = reinterpret_cast<float*>(smem);  // joined sums, over the first stages
  const int stages = p.stages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&s_full[i], 1);
    s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    if (p.D > 0) tma_prefetch_desc(&p.tm_z);
    if (p.vec) tma_prefetch_desc(&p.tm_m);
  }
  pdl_enter(p.early != 0);
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster;
  const int64_t tile = blockIdx.x / C;
  const int64_t t0 = tile * kTok;
  const int distinct = tile_adapters(p.adapter, p.n, t0, p.T, s_id, s_list, &s_count);
  const int rblocks = (p.rank + kRankBlock - 1) / kRankBlock;
  const int half = warp & 1, group = warp >> 1;  // K half of a stage, group of 16 tokens
  const int rs = (p.rank + 15) / 16 * 16;
  const int chunks = (int)((p.D + kDepth - 1) / kDepth);
  const int mine = chunks > (int)rank ? (chunks - (int)rank + C - 1) / C : 0;  // chunks rank, rank + C, ...
  int next_slot = 0, slot = 0;  // ring slots of the next load and of the next chunk to be read
  uint32_t phase = 0;           // of that chunk

  for (int item = blockIdx.y; item < distinct * rblocks; item += gridDim.y) {
    const int32_t a = s_list[item / rblocks];
    const int j0 = (item % rblocks) * kRankBlock;
    const int live = p.rank - j0 < kRankBlock ? p.rank - j0 : kRankBlock;
    auto load = [&](int i) {  // all threads; chunk i of this CTA into the next ring slot
      const int at = next_slot;
      if (++next_slot == stages) next_slot = 0;
      uint8_t* z = smem + at * (kZBytes + kMBytes);
      uint8_t* m = z + kZBytes;
      const int d0 = ((int)rank + i * C) * kDepth;
      if (tid == 0) {
        mbar_arrive_expect_tx(&s_full[at], kZBytes + (p.vec ? kMBytes : 0u));
        tma_load_2d(z, &p.tm_z, &s_full[at], (int32_t)t0, d0);
        if (p.vec) {
          if (TRANS) {
            tma_load_3d(m, &p.tm_m, &s_full[at], j0, d0, a);
          } else {
            tma_load_3d(m, &p.tm_m, &s_full[at], d0, j0, a);
            tma_load_3d(m + kMBytes / 2, &p.tm_m, &s_full[at], d0 + kDepth / 2, j0, a);
          }
        }
      }
      if (!p.vec) {  // rows off 16 bytes: element by element; read at the earliest after two more barriers
        for (int u = tid; u < kRankBlock * 16; u += kThreads) {
          if (!TRANS) {
            const int j = u >> 4, c = u & 15;
            const int64_t valid = j < live ? p.D - (d0 + 8 * c) : 0;
            stage16(m + (c >> 3) * (kMBytes / 2) + j * 128 + (((c & 7) ^ (j & 7)) << 4),
                    p.M + ((int64_t)a * p.rank + j0 + j) * p.D + d0 + 8 * c, valid, 0);
          } else {
            const int row = u / (RB / 8), c = u % (RB / 8);
            const int64_t valid = d0 + row < p.D ? p.rank - (j0 + 8 * c) : 0;
            stage16(RB == 32 ? m + row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : m + row * 128 + ((c ^ (row & 7)) << 4),
                    p.M + ((int64_t)a * p.D + d0 + row) * p.rank + j0 + 8 * c, valid, 0);
          }
        }
      }
    };
    unsigned serves;  // does any of this warp's 16 tokens use the adapter?
    {
      const unsigned lo = __ballot_sync(0xFFFFFFFFu, s_id[lane] == a), hi = __ballot_sync(0xFFFFFFFFu, s_id[32 + lane] == a);
      serves = ((group & 2 ? hi : lo) >> (16 * (group & 1))) & 0xFFFFu;
    }
    float sum[kMT][2][4] = {};
    for (int i = 0; i < stages - 1 && i < mine; ++i) load(i);
    for (int i = 0; i < mine; ++i) {
      mbar_wait(&s_full[slot], phase, &s_abort, p.status, kWaitNs);
      __syncthreads();  // the slot of chunk i - 1 is free, and element-wise loads have landed
      if (i + stages - 1 < mine) load(i + stages - 1);
      const uint32_t z = smem_u32(smem + slot * (kZBytes + kMBytes)), m = z + kZBytes;
      if (++slot == stages) {
        slot = 0;
        phase ^= 1u;
      }
      if (!serves) continue;
      float acc[kMT][2][4] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int ks = 4 * half + q, mi = lane >> 3, l8 = lane & 7;
        uint32_t b[4], w[4];
        const int zr = 16 * ks + 8 * (mi & 1) + l8;
        ldmatrix_x4_trans(b, z + zr * 128 + (((2 * group + (mi >> 1)) ^ (zr & 7)) << 4));
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          if (16 * mt >= live) continue;
          if (!TRANS) {
            const int j = 16 * mt + 8 * (mi & 1) + l8;
            ldmatrix_x4(w, m + half * (kMBytes / 2) + j * 128 + (((2 * q + (mi >> 1)) ^ (j & 7)) << 4));
          } else {
            const int row = 16 * ks + 8 * (mi >> 1) + l8;
            ldmatrix_x4_trans(w, RB == 32 ? m + row * 64 + (((2 * mt + (mi & 1)) ^ ((row >> 1) & 3)) << 4)
                                           : m + row * 128 + (((2 * mt + (mi & 1)) ^ (row & 7)) << 4));
          }
          mma_bf16(acc[mt][0], w, b[0], b[1]);
          mma_bf16(acc[mt][1], w, b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8 * kMT; ++e) sum[e >> 3][(e >> 2) & 1][e & 3] += acc[e >> 3][(e >> 2) & 1][e & 3];
    }
    __syncthreads();  // every warp is done with the stages
    // The sums, in the order of the output (ranks of a token, or tokens of a rank row, side by side): lanes that read
    // another CTA's shared memory at neighbouring addresses share a transfer (reading it across rows took 14 us of a
    // 25 us item).  The second K half's warps leave theirs, the first half's add them to their own.
    auto part_at = [](int j, int t) { return OUT == SHRINK_BLOCKS ? j * (kTok + 1) + t : t * (kRankBlock + 1) + j; };
#pragma unroll
    for (int h = 1; h >= 0; --h) {
      if (half == h) {
#pragma unroll
        for (int e = 0; e < 8 * kMT; ++e) {
          const int mt = e >> 3, nb = (e >> 2) & 1, f = e & 3;
          const int at = part_at(16 * mt + (lane >> 2) + 8 * (f >> 1), 16 * group + 8 * nb + 2 * (lane & 3) + (f & 1));
          s_part[at] = h == 1 ? sum[mt][nb][f] : sum[mt][nb][f] + s_part[at];
        }
      }
      __syncthreads();
    }
    if (C > 1) cluster_sync();  // every CTA's sums are written
    // Output e belongs to one CTA of the cluster: nobody else reads its place in that CTA's own sums, so the joined
    // value goes back there and leaves after the others have been told that their sums are done with.
    for (int e = tid + kThreads * (int)rank; C > 1 && e < kRankBlock * kTok; e += kThreads * C) {
      const int j = OUT == SHRINK_BLOCKS ? e / kTok : e % kRankBlock, t = OUT == SHRINK_BLOCKS ? e % kTok : e / kRankBlock;
      float* place = s_part + part_at(j, t);
      const uint32_t mine_at = smem_u32(place);
      float part[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) part[c] = c < C ? ld_cluster_f32(map_to_cta(mine_at, c)) : 0.f;
      *place = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
    }
    if (C > 1) cluster_arrive();  // the stores below need not be waited for
    for (int e = tid + kThreads * (int)rank; e < kRankBlock * kTok; e += kThreads * C) {
      const int j = OUT == SHRINK_BLOCKS ? e / kTok : e % kRankBlock, t = OUT == SHRINK_BLOCKS ? e % kTok : e / kRankBlock;
      const bool own = s_id[t] == a;
      if (OUT == SHRINK_BLOCKS ? (j >= live || t0 + t >= p.ldp) : (!own || j0 + j >= rs)) continue;
      float v = s_part[part_at(j, t)];
      if (OUT == SHRINK_F32) {
        p.S[(t0 + t) * rs + j0 + j] = v;
      } else {
        if (OUT == SHRINK_BLOCKS && p.scale) v *= __ldg(p.scale + a);
        uint16_t term[P];
        split_terms<P>(v, term);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          if (OUT == SHRINK_TERMS)
            p.terms[((int64_t)q * p.T + t0 + t) * rs + j0 + j] = term[q];
          else
            p.terms[((int64_t)q * p.cat + (int64_t)a * p.rank + j0 + j) * p.ldp + t0 + t] = own ? term[q] : (uint16_t)0;
        }
      }
    }
    if (C > 1) cluster_wait();  // the sums may be overwritten, and a CTA may leave
    fence_proxy_async_smem();   // ... by the next item's copies, which take their place: ordinary accesses come first
    __syncthreads();
  }

  if (OUT == SHRINK_BLOCKS && blockIdx.y == 0) {  // the rows of adapters that the tile does not use, and the tile's mask
    if (tid < kMaxCat / 32) s_present[tid] = 0;
    __syncthreads();
    if (tid < distinct) {
      const int32_t a = s_list[tid];
      if (a < kMaxCat) atomicOr(&s_present[a >> 5], 1u << (a & 31));
    }
    __syncthreads();
    for (int64_t u = tid + kThreads * (int64_t)rank; u < p.cat * 8; u += (int64_t)kThreads * C) {
      const int row = (int)(u >> 3), c = (int)(u & 7);
      const int a = row / p.rank;
      if (a < p.n && ((s_present[a >> 5] >> (a & 31)) & 1u)) continue;
      if (t0 + 8 * c >= p.ldp) continue;
#pragma unroll
      for (int q = 0; q < P; ++q)
        *reinterpret_cast<uint4*>(p.terms + ((int64_t)q * p.cat + row) * p.ldp + t0 + 8 * c) = make_uint4(0, 0, 0, 0);
    }
    if (rank == 0 && tid == 0) {
      uint32_t mask = 0;
      for (int i = 0; i < distinct; ++i) {
        const int first = (int)s_list[i] * p.rank / 64, last = ((int)s_list[i] * p.rank + p.rank - 1) / 64;
        for (int b = first; b <= last; ++b) mask |= 1u << b;
      }
      p.masks[tile] = mask;
    }
  }
  pdl_leave(p.early != 0);
  if (p.inv) {  // after the wait: the launch before presets inv
    const int64_t all = (int64_t)gridDim.x * gridDim.y * kThreads;
    for (int64_t k = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + tid; k < p.idx_n; k += all) {
      const int32_t j = __ldg(p.idx + k);
      if (j >= 0 && (int64_t)j < p.idx_n) atomicMax(p.inv + j, (int32_t)k);
    }
  }
}

template <bool TRANS, int P>
__global__ void __launch_bounds__(lora::kThreads) lora_expand_kernel(const LoraExpand p) {
  using namespace lora;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_id[kTok], s_list[kTok];
  __shared__ int s_count;
  pdl_gate();
  const int rs = (p.rank + 15) / 16 * 16;
  const uint32_t pitch = (uint32_t)rs * 2 + 16;  // an odd number of 16-byte units: eight rows miss each other's banks
  const uint32_t m_bytes = TRANS ? (uint32_t)rs * 256u : kRows * pitch;
  uint8_t* s_m = smem;                      // p.batch adapters' tiles
  uint8_t* s_s = smem + p.batch * m_bytes;  // P terms of 64 tokens x rs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * kRows, t0 = (int64_t)blockIdx.y * kTok;

  const int tokens = p.T - t0 < kTok ? (int)(p.T - t0) : kTok;
  const int distinct = tile_adapters(p.adapter, p.n, t0, p.T, s_id, s_list, &s_count);

  const int unit_bits = rs <= 16 ? 1 : rs <= 32 ? 2 : rs <= 64 ? 3 : 4;  // 16-byte units of a row, to a power of two
  auto load = [&](int i, int at) {
    uint8_t* m = s_m + at * m_bytes;
    const int64_t a = s_list[i];
    if (!TRANS) {
      for (int u = tid; u < kRows << unit_bits; u += kThreads) {
        const int row = u >> unit_bits, c = u & ((1 << unit_bits) - 1);
        if (8 * c >= rs) continue;
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
  for (int i = 0; i < p.batch && i < distinct; ++i) load(i, i);
  cp_commit();
  // s_a S of the tile's tokens as P bf16 terms (0 for a token without an adapter, whose S is not written)
  for (int u = tid; u < tokens * (rs / 4); u += kThreads) {
    const int t = u / (rs / 4), j = 4 * (u - t * (rs / 4));
    const int32_t id = s_id[t];
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (id >= 0) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p.S + (t0 + t) * rs + j));
      const float sc = p.scale ? __ldg(p.scale + id) : 1.f;
      v[0] = x.x * sc;
      v[1] = x.y * sc;
      v[2] = x.z * sc;
      v[3] = x.w * sc;
    }
    uint16_t term[4][P];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_terms<P>(v[e], term[e]);
#pragma unroll
    for (int q = 0; q < P; ++q)
      *reinterpret_cast<uint2*>(s_s + ((uint32_t)q * kTok + t) * pitch + 2 * j) =
          make_uint2((uint32_t)term[0][q] | (uint32_t)term[1][q] << 16, (uint32_t)term[2][q] | (uint32_t)term[3][q] << 16);
  }

  // The base, while the adapters' tiles are on their way.  Several K ranges' sums are added on the way into shared
  // memory, four ranges in flight for every 16 bytes.
  float acc[8][4];
  if (p.splits > 1) {
    float* s_base = reinterpret_cast<float*>(smem + p.base_off);
    const int quads = (int)p.ldb / 4;  // rows of a K range's sums: 16, 32 or 64 columns (one tile of tokens)
#pragma unroll 2
    for (int u = tid; u < kRows * quads; u += kThreads) {
      const int row = u / quads, c = u - row * quads;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r0 + row < p.rows) {
        const float* src = p.base + (r0 + row) * p.ldb + 4 * c;
        for (int q0 = 0; q0 < p.splits; q0 += 4) {
          float4 x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            x[q] = q0 + q < p.splits ? __ldcg(reinterpret_cast<const float4*>(src + (q0 + q) * p.split_stride))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v.x += x[q].x;
            v.y += x[q].y;
            v.z += x[q].z;
            v.w += x[q].w;
          }
        }
      }
      *reinterpret_cast<float4*>(s_base + row * (p.ldb + 4) + 4 * c) = v;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nb = 0; nb < 8; ++nb) {
        const int t = 8 * nb + 2 * (lane & 3);
        float2 v = make_float2(0.f, 0.f);
        if (t < tokens)
          v = *reinterpret_cast<const float2*>(s_base + (16 * warp + (lane >> 2) + 8 * h) * (p.ldb + 4) + t);
        acc[nb][2 * h] = v.x;
        acc[nb][2 * h + 1] = v.y;
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (p.splits > 1) break;
    const int64_t row = r0 + 16 * warp + (lane >> 2) + 8 * h;
    int64_t brow = row < p.rows ? row : -1;
    if (p.base_row && brow >= 0) brow = __ldcg(p.base_row + row);
    const float* src = p.base + brow * p.ldb + t0 + 2 * (lane & 3);
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const bool in = brow >= 0 && 8 * nb + 2 * (lane & 3) < tokens;
      const float2 v = in ? __ldcg(reinterpret_cast<const float2*>(src + 8 * nb)) : make_float2(0.f, 0.f);
      acc[nb][2 * h] = v.x;
      acc[nb][2 * h + 1] = v.y;
    }
  }
  for (int i = 0, at = 0; i < distinct; ++i, ++at) {
    if (at == p.batch) {  // the next batch of adapters' tiles, all in flight together
      __syncthreads();
      at = 0;
      for (int u = 0; u < p.batch && i + u < distinct; ++u) load(i + u, u);
      cp_commit();
    }
    if (at == 0) {
      cp_wait<0>();
      __syncthreads();  // the batch has landed (and S, at first)
    }
    const int32_t a = s_list[i];
    const uint32_t m = smem_u32(s_m + at * m_bytes);
    const unsigned lo = __ballot_sync(0xFFFFFFFFu, s_id[lane] == a), hi = __ballot_sync(0xFFFFFFFFu, s_id[32 + lane] == a);
    const int mi = lane >> 3, l8 = lane & 7;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const unsigned used = ((b & 2 ? hi : lo) >> (16 * (b & 1))) & 0xFFFFu;  // this block's tokens of the adapter
      if (!used) continue;
      __syncwarp();  // lanes kept other columns of the last block
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
          if ((used >> (8 * h + 2 * (lane & 3) + (e & 1))) & 1u) acc[2 * b + h][e] += d[h][e];
    }
  }

#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + 16 * warp + (lane >> 2) + 8 * h;
    if (row >= p.rows) continue;
    const int64_t at = row * p.ldy + t0 + 2 * (lane & 3);
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const int t = 8 * nb + 2 * (lane & 3);
      if (t >= tokens) continue;
      if (p.out_f32) {
        float* y = static_cast<float*>(p.Y) + at + 8 * nb;
        if (t + 1 < tokens)
          *reinterpret_cast<float2*>(y) = make_float2(acc[nb][2 * h], acc[nb][2 * h + 1]);
        else
          *y = acc[nb][2 * h];
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.Y) + at + 8 * nb;
        const uint32_t w = pack_bf16x2(acc[nb][2 * h], acc[nb][2 * h + 1]);
        if (t + 1 < tokens)
          *reinterpret_cast<uint32_t*>(y) = w;
        else
          *y = (uint16_t)(w & 0xFFFFu);
      }
    }
  }
}

// The second factors of all adapters side by side (see LoraCat).
template <bool BY_RANK>
__global__ void __launch_bounds__(256) lora_cat_kernel(const LoraCat p) {
  pdl_gate();
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
  if (p.inv)
    for (int64_t k = first; k < p.rows; k += all) p.inv[k] = -1;
  const int live = (int)p.n * p.rank;
  const int64_t lines = BY_RANK ? live : p.rows, units = p.ldc / 8;
  bool bad = false;
  for (int64_t u = first; u < lines * units; u += all) {
    const int64_t line = u / units;
    const int64_t c = (u - line * units) * 8;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t v = 0;
      if (BY_RANK) {
        if (c + e < p.rows) {
          const int64_t k = p.idx ? (int64_t)__ldg(p.idx + c + e) : c + e;
          if (k >= 0 && k < p.rows) v = __ldg(p.M + line * p.rows + k);
        }
      } else if (c + e < live) {
        const int col = (int)c + e, a = col / p.rank;
        v = __ldg(p.M + ((int64_t)a * p.rows + line) * p.rank + col - a * p.rank);
      }
      if ((v & 0x7F80u) == 0x7F80u) {
        bad = true;
        v = 0;
      }
      w[e >> 1] |= v << (16 * (e & 1));
    }
    *reinterpret_cast<uint4*>(p.out + line * p.ldc + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.flags[blockIdx.x] = any ? 1u : 0u;
}

// Plain loads, every row and token as soon as one weight of any adapter is flagged: the other requests' results stay as
// they are, but wait for it (4096 x 4096 x 2048 with eight adapters of rank 16 69 us, with one Inf among them 2.2 ms; input
// gradient 4096 x 11008 x 2048 178 us and 2.9 ms).  Such an adapter is broken, and its user has to be told anyway.
template <bool TRANS>
__global__ void __launch_bounds__(256) lora_mend_kernel(const LoraMend p) {
  pdl_gate();
  bool set = false;
  for (int i = threadIdx.x; i < p.nflags; i += 256) set |= __ldcg(p.flags + i) != 0;
  const int64_t r0 = (int64_t)blockIdx.x * 128;
  bool orphan = false;
  if (p.inv && threadIdx.x < 128 && r0 + threadIdx.x < p.rows) orphan = __ldcg(p.inv + r0 + threadIdx.x) < 0;
  const int flagged = __syncthreads_or(set), orphans = __syncthreads_or(orphan);
  if (!flagged && !orphans) return;
  for (int64_t row = r0 + (threadIdx.x >> 5); row < r0 + 128 && row < p.rows; row += 8) {
    const bool whole = p.inv && __ldcg(p.inv + row) < 0;
    if (!whole && !flagged) continue;
    for (int64_t t = threadIdx.x & 31; t < p.T; t += 32) {
      const int32_t a = __ldg(p.adapter + t);
      float v = 0.f;
      bool any = whole;
      if (a >= 0 && (int64_t)a < p.n) {
        for (int j = 0; j < p.rank; ++j) {
          const uint32_t b = TRANS ? __ldg(p.M + ((int64_t)a * p.rank + j) * p.rows + row)
                                   : __ldg(p.M + ((int64_t)a * p.rows + row) * p.rank + j);
          if (!whole && (b & 0x7F80u) != 0x7F80u) continue;
          any = true;
          float s = 0.f;
          for (int q = 0; q < p.planes; ++q)
            s += __uint_as_float((uint32_t)__ldcg(p.blocks + ((int64_t)q * p.cat + (int64_t)a * p.rank + j) * p.ldp + t) << 16);
          v += __uint_as_float(b << 16) * s;
        }
      }
      if (!any) continue;
      if (p.out_f32) {
        float* y = static_cast<float*>(p.Y) + row * p.ldy + t;
        *y = whole ? v : *y + v;
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.Y) + row * p.ldy + t;
        const float f = whole ? v : __uint_as_float((uint32_t)*y << 16) + v;
        *y = (uint16_t)(pack_bf16x2(f, 0.f) & 0xFFFFu);
      }
    }
  }
}

// The tiles that hold tokens of adapter blockIdx.x, ascending, and their number.  A warp votes on four tiles at a time.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* adapter, int64_t T, int32_t* tiles,
                                                         int32_t* counts) {
  using namespace lora;
  __shared__ int s_has[128], s_votes[4];
  pdl_gate();
  const int32_t a = (int32_t)blockIdx.x;
  const int64_t all = (T + kTok - 1) / kTok;
  int32_t* out = tiles + (int64_t)a * all;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int found = 0;
  for (int64_t base = 0; base < all; base += 128) {
    int32_t id[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = (base + 4 * warp) * kTok + 32 * i + lane;
      id[i] = t < T ? __ldg(adapter + t) : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool has = __any_sync(0xFFFFFFFFu, id[2 * i] == a || id[2 * i + 1] == a);
      if (lane == 0) s_has[4 * warp + i] = has;
    }
    __syncthreads();
    bool has = false;
    unsigned votes = 0;
    if (threadIdx.x < 128) {
      has = s_has[threadIdx.x] != 0;
      votes = __ballot_sync(0xFFFFFFFFu, has);
      if (lane == 0) s_votes[warp] = __popc(votes);
    }
    __syncthreads();
    int before = found, total = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) before += s_votes[w];
      total += s_votes[w];
    }
    if (has) out[before + __popc(votes & ((1u << lane) - 1u))] = (int32_t)(base + threadIdx.x);
    found += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) counts[a] = found;
}

template <bool BY_RANK, int P>
__global__ void __launch_bounds__(lora::kThreads, 2) lora_outer_kernel(const __grid_constant__ LoraOuter p) {
  using namespace lora;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kV = outer_v(P);                  // stages of V: P terms of [64 tokens][up to 64 ranks]
  constexpr uint32_t kVStage = P * kOuterV;
  constexpr uint32_t kCols = P == 3 ? 256 : 128;  // TMEM columns: the terms' products side by side, 64 each at most
  uint8_t* s_v = smem + kOuterZ * kOuterM;
  __shared__ int32_t s_id[kOuterZ][kTok];
  __shared__ uint64_t s_fz[kOuterZ], s_fv[kV], s_done[kOuterZ];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kOuterZ; ++i) {
      mbar_init(&s_fz[i], 1);
      mbar_init(&s_done[i], 1);
    }
    for (int i = 0; i < kV; ++i) mbar_init(&s_fv[i], 1);
    s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&p.tm_z);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 4) {
    tmem_alloc(&s_tmem, kCols);
    tmem_relinquish();
  }
  pdl_enter(p.early != 0);
  const uint32_t rank = cluster_ctarank();
  const int C = p.cluster;
  const int64_t r0 = (int64_t)(blockIdx.x / C) * kRows;
  const int rblocks = (p.rank + kOuterRank - 1) / kOuterRank;
  const int32_t a = (int32_t)(blockIdx.y / rblocks);
  const int j0 = (int)(blockIdx.y % rblocks) * kOuterRank;
  const int box = outer_box(p.rank);  // rank columns that a box brings, N of the MMAs (past the rank: zeros)
  const int32_t* list = p.tiles + (int64_t)a * ((p.T + kTok - 1) / kTok);
  const int count = __ldcg(p.counts + a);
  int32_t first[kOuterZ];  // read beside the count (places past it hold no tile and are not used)
#pragma unroll
  for (int d = 0; d < kOuterZ; ++d) {
    const int64_t at = rank + (int64_t)d * C;
    first[d] = at < (p.T + kTok - 1) / kTok ? __ldcg(list + at) : 0;
  }
  const int mine = count > (int)rank ? (count - (int)rank + C - 1) / C : 0;  // tiles rank, rank + C, ... of the list
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Tile i of this CTA: Z and its tokens' adapters into ring slot i % kOuterZ, V into slot i % kV.  The tile numbers come
  // from the list two turns earlier, so that no load waits for the list.
  auto load_z = [&](int i, int32_t tile) {
    const int slot = i % kOuterZ;
    const int64_t t0 = (int64_t)tile * kTok;
    if (tid == 0) {
      mbar_arrive_expect_tx(&s_fz[slot], kOuterM);
      tma_load_2d(smem + slot * kOuterM, &p.tm_z, &s_fz[slot], (int32_t)t0, (int32_t)r0);
    } else if (tid >= 64 && tid < 64 + kTok) {
      const int t = tid - 64;
      s_id[slot][t] = t0 + t < p.T ? __ldg(p.adapter + t0 + t) : -1;
    }
  };
  auto load_v = [&](int i, int32_t tile) {
    if (tid != 32) return;
    const int slot = i % kV;
    mbar_arrive_expect_tx(&s_fv[slot], (uint32_t)(P * kTok * box * 2));
#pragma unroll
    for (int q = 0; q < P; ++q)
      tma_load_3d(s_v + slot * kVStage + q * kOuterV, &p.tm_v, &s_fv[slot], j0, tile * kTok, q);
  };
  // The products of tile i are complete (its slots are free, its accumulator may be read).
  auto done = [&](int i) {
    return mbar_wait(&s_done[i % kOuterZ], (uint32_t)(i / kOuterZ) & 1u, &s_abort, p.status, kWaitNs);
  };
  // next[d]: the tile that is d turns ahead
  int32_t next[kOuterZ];
#pragma unroll
  for (int d = 0; d < kOuterZ; ++d) next[d] = d < mine ? first[d] : 0;
#pragma unroll
  for (int d = 0; d < kOuterZ - 1; ++d)
    if (d < mine) load_z(d, next[d]);
#pragma unroll
  for (int d = 0; d < kV - 1; ++d)
    if (d < mine) load_v(d, next[d]);
  const uint32_t idesc = idesc_bf16_major((uint32_t)(P * box), (uint32_t)kRows, false, true);
  const uint32_t v_row = (uint32_t)box * 2u;  // bytes of a token's ranks, the swizzle's width
  const uint32_t v_swz = box == 64 ? SWZ_128B : box == 32 ? SWZ_64B : SWZ_32B;
  // This thread's part of the sums: row 32 (warp % 4) + lane, 32 ranks from 32 (warp / 4).
  const uint32_t my_tmem = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32u * (uint32_t)(warp >> 2);
  float sum[32] = {};
  auto flush = [&] {  // adds the accumulators of a group of tiles, whose products are complete
    tc_fence_after();
#pragma unroll
    for (int q = 0; q < P; ++q) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(my_tmem + (uint32_t)(q * box), v);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) sum[e] += __uint_as_float(v[e]);
    }
    tc_fence_before();  // the next __syncthreads lets the next group overwrite them
  };
  __syncthreads();  // the first tiles' adapters are there
  bool ok = true;
  for (int i = 0; i < mine && ok; ++i) {
    const int slot = i % kOuterZ;
    uint8_t* z = smem + slot * kOuterM;
    uint8_t* v = s_v + (i % kV) * kVStage;
    ok = mbar_wait(&s_fz[slot], (uint32_t)(i / kOuterZ) & 1u, &s_abort, p.status, kWaitNs) &&
         mbar_wait(&s_fv[i % kV], (uint32_t)(i / kV) & 1u, &s_abort, p.status, kWaitNs);
    const unsigned lo = __ballot_sync(0xFFFFFFFFu, s_id[slot][lane] == a);
    const unsigned hi = __ballot_sync(0xFFFFFFFFu, s_id[slot][32 + lane] == a);
    if ((lo & hi) != 0xFFFFFFFFu) {
      // Tokens that are not the adapter's leave both operands: their Inf or NaN in one would survive a 0 in the other, and
      // S of a token without an adapter is not written at all.
#pragma unroll
      for (int u = 0; u < kRows * 8 / kThreads; ++u) {
        const int e = tid + u * kThreads, row = e >> 3, c = e & 7;  // tokens 8 c ..
        const unsigned used = ((c & 4 ? hi : lo) >> (8 * (c & 3))) & 0xFFu;
        if (used == 0xFFu) continue;
        uint4* at = reinterpret_cast<uint4*>(z + row * 128 + ((c ^ (row & 7)) << 4));
        uint4 w = *at;
        auto keep = [&](int j) { return (used >> j & 1u ? 0xFFFFu : 0u) | (used >> j & 2u ? 0xFFFF0000u : 0u); };
        w.x &= keep(0);
        w.y &= keep(2);
        w.z &= keep(4);
        w.w &= keep(6);
        *at = w;
      }
      const int units = box / 8;  // 16-byte units of a token, swizzled within it
      for (int e = tid; e < P * kTok * units; e += kThreads) {
        const int q = e / (kTok * units), t = (e - q * kTok * units) / units, c = e % units;
        if (((t & 32 ? hi : lo) >> (t & 31)) & 1u) continue;
        *reinterpret_cast<uint4*>(v + q * kOuterV + t * v_row + c * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
    }
    if (i > 0 && i % kOuterGroup == 0) {
      const bool complete = __all_sync(0xFFFFFFFFu, done(i - 1));
      if (complete) flush();
      ok = ok && complete;
    }
    ok = !__syncthreads_or(!ok);  // every thread leaves together when a copy did not come
    if (tid == 0 && ok) {
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < kTok / 16; ++ks)  // the terms are P atoms of the second operand: Z is read once for all
        tc_mma(tmem, smem_desc(smem_u32(z) + 32 * ks, 16, 1024, SWZ_128B),
               smem_desc(smem_u32(v) + ks * 16 * v_row, kOuterV, 8 * v_row, v_swz), idesc,
               i % kOuterGroup > 0 || ks > 0 ? 1u : 0u);
      tc_commit(&s_done[slot]);
    }
    if (!ok) break;
    if (i >= 1 && (tid == 0 || tid == 32)) done(i - 1);  // the slots of tile i - 1 are free
    if (i + kOuterZ - 1 < mine) load_z(i + kOuterZ - 1, next[kOuterZ - 1]);
    if (i + kV - 1 < mine) load_v(i + kV - 1, next[kV - 1]);
#pragma unroll
    for (int d = 0; d + 1 < kOuterZ; ++d) next[d] = next[d + 1];
    next[kOuterZ - 1] = i + kOuterZ < mine ? __ldcg(list + rank + (int64_t)(i + kOuterZ) * C) : 0;
  }
  if (mine > 0 && ok && __all_sync(0xFFFFFFFFu, done(mine - 1))) flush();
  if (*static_cast<volatile int*>(&s_abort)) sleep_about_ns(200000ull);  // what is in flight lands before its place is reused
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(smem);  // [128 rows][kOuterPitch], over the stages
#pragma unroll
  for (int e = 0; e < 32; e += 4)
    *reinterpret_cast<float4*>(s_sum + (32 * (warp & 3) + lane) * kOuterPitch + 32 * (warp >> 2) + e) =
        make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  if (C > 1) cluster_sync();
  const float scale = p.scale ? __ldg(p.scale + a) : 1.f;
  const int part = kRows / C;  // rows that this CTA joins and stores
  const int live = p.rank - j0 < kOuterRank ? p.rank - j0 : kOuterRank;
  // Four neighbouring ranks of a row at a time.  Rank-contiguous outputs leave from here.  For row-contiguous ones the
  // joined values go back to this CTA's own sums (whose rows nobody else reads) and leave row by row.
  float* own = s_sum + (int)rank * part * kOuterPitch;
  const int64_t out0 = (int64_t)a * p.rows * p.rank;
  const bool vec = !BY_RANK && p.out_f32 && p.rank % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0;
#pragma unroll 2
  for (int e = tid; e < part * (kOuterRank / 4); e += kThreads) {
    const int row = e / (kOuterRank / 4), j = 4 * (e % (kOuterRank / 4));
    float* place = own + row * kOuterPitch + j;
    const uint32_t at = smem_u32(place);
    float4 got[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) got[c] = ld_cluster_f32x4(map_to_cta(at, c));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= C) continue;
      v.x += got[c].x;
      v.y += got[c].y;
      v.z += got[c].z;
      v.w += got[c].w;
    }
    v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    const int64_t r = r0 + (int)rank * part + row;
    if (BY_RANK) {
      *reinterpret_cast<float4*>(place) = v;
    } else if (r < p.rows && j < live) {
      const int64_t to = out0 + r * p.rank + j0 + j;
      if (vec) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = v;
      } else {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (j + u >= live) continue;
          if (p.out_f32)
            static_cast<float*>(p.out)[to + u] = f[u];
          else
            static_cast<uint16_t*>(p.out)[to + u] = (uint16_t)(pack_bf16x2(f[u], 0.f) & 0xFFFFu);
        }
      }
    }
  }
  if (C > 1) cluster_arrive();  // done with the other CTAs' sums
  if (BY_RANK) {
    __syncthreads();
    const int bits = 31 - __clz(part);  // a power of two
#pragma unroll 4
    for (int e = tid; e < part * live; e += kThreads) {
      const int row = e & (part - 1), j = e >> bits;
      const int64_t r = r0 + (int)rank * part + row;
      if (r >= p.rows) continue;
      const float v = own[row * kOuterPitch + j];
      const int64_t to = out0 + (int64_t)(j0 + j) * p.rows + r;
      if (p.out_f32)
        static_cast<float*>(p.out)[to] = v;
      else
        static_cast<uint16_t*>(p.out)[to] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
    }
  }
  if (C > 1) cluster_wait();  // no CTA leaves while another still reads its sums
  pdl_leave(p.early != 0);
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

template <auto Kern, typename Params>
static cudaError_t launch_clustered(dim3 grid, int cluster, uint32_t smem, uint32_t smem_limit, const Params& p,
                                    cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(Kern, smem_limit);
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
  e = cudaLaunchKernelEx(&cfg, Kern, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool TRANS, int RB>
static cudaError_t launch_shrink_out(const LoraShrink& p, dim3 grid, cudaStream_t s) {
  using namespace lora;
  const uint32_t b = shrink_smem(p.stages, RB), most = shrink_smem(kMaxStages, RB);
  const int c = p.cluster;
  if (p.out == SHRINK_F32) return launch_clustered<&lora_shrink_kernel<TRANS, SHRINK_F32, 1, RB>>(grid, c, b, most, p, s);
  if (p.out == SHRINK_TERMS)
    return p.planes == 3 ? launch_clustered<&lora_shrink_kernel<TRANS, SHRINK_TERMS, 3, RB>>(grid, c, b, most, p, s)
                         : launch_clustered<&lora_shrink_kernel<TRANS, SHRINK_TERMS, 2, RB>>(grid, c, b, most, p, s);
  return p.planes == 3 ? launch_clustered<&lora_shrink_kernel<TRANS, SHRINK_BLOCKS, 3, RB>>(grid, c, b, most, p, s)
                       : launch_clustered<&lora_shrink_kernel<TRANS, SHRINK_BLOCKS, 2, RB>>(grid, c, b, most, p, s);
}

cudaError_t launch_lora_shrink(LoraShrink& p, bool trans, cudaStream_t s) {
  using namespace lora;
  const int64_t tiles = tiles_of(p.T), chunks = (p.D + kDepth - 1) / kDepth;
  const int64_t target = 2 * (int64_t)sm_count_current();
  // The CTAs of a cluster share the reduction until the grid fills the SMs twice over (two stages each at least)
  p.cluster = 1;
  while (p.cluster < 8 && tiles * p.cluster < target && chunks / (2 * p.cluster) >= 2) p.cluster <<= 1;
  // ... and further CTAs take the tile's adapters side by side when the tiles are few
  const int64_t rblocks = (p.rank + rank_block(p.rank) - 1) / rank_block(p.rank);
  const int64_t items = (p.n < kTok ? p.n : kTok) * rblocks;
  int64_t y = (target + tiles * p.cluster - 1) / (tiles * p.cluster);
  if (y < rblocks) y = rblocks;
  if (y > items) y = items;
  if (tiles * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  // Two or three CTAs to an SM in a full grid (three stages); with an SM to itself a CTA has all its chunks in flight.
  p.stages = tiles * p.cluster * y <= sm_count_current() ? kMaxStages : 3;
  const dim3 grid((unsigned)(tiles * p.cluster), (unsigned)y);
  if (rank_block(p.rank) == 64)
    return trans ? launch_shrink_out<true, 64>(p, grid, s) : launch_shrink_out<false, 64>(p, grid, s);
  return trans ? launch_shrink_out<true, 32>(p, grid, s) : launch_shrink_out<false, 32>(p, grid, s);
}

cudaError_t launch_lora_expand(LoraExpand& p, bool trans, cudaStream_t s) {
  using namespace lora;
  const int64_t tiles = tiles_of(p.T), blocks = (p.rows + kRows - 1) / kRows;
  if (tiles > 65535) return cudaErrorInvalidValue;
  const uint32_t terms = p.out_f32 ? 3 : 2;
  const uint32_t r = (uint32_t)rank_stride(p.rank), tile = trans ? r * 256u : kRows * (r * 2 + 16);
  int64_t batch = kExpandBatch / tile;  // at least 2
  if (batch > p.n) batch = p.n > 0 ? p.n : 1;
  if (batch > kTok) batch = kTok;
  p.batch = (int)batch;
  const dim3 grid((unsigned)blocks, (unsigned)tiles);
  p.base_off = (uint32_t)batch * tile + terms * kTok * (r * 2 + 16);
  const uint32_t b = p.base_off + (p.splits > 1 ? (uint32_t)(kRows * (p.ldb + 4) * 4) : 0u);
  const uint32_t most = kExpandBatch + 3 * kTok * (kMaxRank * 2 + 16) + kRows * (kTok + 4) * 4;
  if (trans)
    return p.out_f32 ? launch_clustered<&lora_expand_kernel<true, 3>>(grid, 1, b, most, p, s)
                     : launch_clustered<&lora_expand_kernel<true, 2>>(grid, 1, b, most, p, s);
  return p.out_f32 ? launch_clustered<&lora_expand_kernel<false, 3>>(grid, 1, b, most, p, s)
                   : launch_clustered<&lora_expand_kernel<false, 2>>(grid, 1, b, most, p, s);
}

int lora_cat_blocks() { return 2 * sm_count_current(); }

cudaError_t launch_lora_cat(LoraCat& p, bool by_rank, cudaStream_t s) {
  p.blocks = lora_cat_blocks();
  cudaError_t e = by_rank ? launch_pdl(lora_cat_kernel<true>, dim3((unsigned)p.blocks), dim3(256), 0, s, p)
                          : launch_pdl(lora_cat_kernel<false>, dim3((unsigned)p.blocks), dim3(256), 0, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_mend(const LoraMend& p, bool trans, cudaStream_t s) {
  const dim3 grid((unsigned)((p.rows + 127) / 128));
  cudaError_t e = trans ? launch_pdl(lora_mend_kernel<true>, grid, dim3(256), 0, s, p)
                        : launch_pdl(lora_mend_kernel<false>, grid, dim3(256), 0, s, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_plan(const int32_t* adapter, int64_t T, int64_t n, int32_t* tiles, int32_t* counts,
                             cudaStream_t s) {
  cudaError_t e = launch_pdl(lora_plan_kernel, dim3((unsigned)n), dim3(1024), 0, s, adapter, T, tiles, counts);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_outer(LoraOuter& p, bool by_rank, cudaStream_t s) {
  using namespace lora;
  const int64_t blocks = (p.rows + kRows - 1) / kRows, tiles = tiles_of(p.T);
  const int64_t items = p.n * ((p.rank + kOuterRank - 1) / kOuterRank);
  if (blocks == 0 || items == 0) return cudaSuccess;
  if (items > 65535) return cudaErrorInvalidValue;
  // CTAs that share an adapter's tokens, until every SM has one (until it has three: 8 us more of the 74 above)
  p.cluster = 1;
  while (p.cluster < 8 && blocks * items * p.cluster < (int64_t)sm_count_current() && tiles / (2 * p.cluster) >= 2)
    p.cluster <<= 1;
  if (blocks * p.cluster >= (1ll << 31)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * p.cluster), (unsigned)items);
  const uint32_t b = outer_smem(p.out_f32 ? 3 : 2);
  if (by_rank)
    return p.out_f32 ? launch_clustered<&lora_outer_kernel<true, 3>>(grid, p.cluster, b, b, p, s)
                     : launch_clustered<&lora_outer_kernel<true, 2>>(grid, p.cluster, b, b, p, s);
  return p.out_f32 ? launch_clustered<&lora_outer_kernel<false, 3>>(grid, p.cluster, b, b, p, s)
                   : launch_clustered<&lora_outer_kernel<false, 2>>(grid, p.cluster, b, b, p, s);
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
  return check_words({ad.scale, ad.adapter}, "scale and adapter");
}
nm_status check_operand(const uint16_t* values, const uint32_t* meta, const int32_t* idx) {
  if (!aligned_to(values, 2)) return fail(NM_ERR_MISALIGNED, "values misaligned");
  return check_words({meta, idx}, "meta and idx");
}
nm_status check_adapter_pointers(const Adapters& ad, int64_t R, int64_t K, int64_t T) {
  if ((!ad.A && K > 0) || (!ad.B && R > 0) || !ad.adapter) return fail(NM_ERR_INVALID_ARG, "A, B or adapter is null");
  if (!aligned_to(ad.A, 2) || !aligned_to(ad.B, 2)) return fail(NM_ERR_MISALIGNED, "A or B misaligned");
  if (lora::tiles_of(T) > 65535) return fail(NM_ERR_UNSUPPORTED, "more than %d tokens in a call", 65535 * lora::kTok);
  return NM_OK;
}

// The shrink product of Z (D x T) into the form that `p` asks for.
nm_status shrink(const Adapters& ad, bool trans, int64_t D, const uint16_t* Z, int64_t ldz, int64_t T, LoraShrink& p,
                 cudaStream_t s) {
  using namespace lora;
  p.M = trans ? ad.B : ad.A;
  p.adapter = ad.adapter;
  p.scale = ad.scale;
  p.n = ad.n;
  p.D = D;
  p.T = T;
  p.rank = ad.rank;
  p.vec = D > 0 && al16(p.M) && (trans ? ad.rank : D) % 8 == 0;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  nm_status st = NM_OK;
  if (D > 0) st = make_tmap(&p.tm_z, Z, (uint64_t)T, (uint64_t)D, (uint64_t)ldz * 2, kTok, kDepth, 128, "tokens");
  if (st == NM_OK && p.vec) {
    const int rb = rank_block(ad.rank);
    const uint64_t inner = trans ? (uint64_t)ad.rank : (uint64_t)D, rows = trans ? (uint64_t)D : (uint64_t)ad.rank;
    st = make_tmap3(&p.tm_m, p.M, inner, rows, (uint64_t)ad.n, inner * 2, inner * rows * 2, trans ? (uint32_t)rb : 64u,
                    trans ? (uint32_t)kDepth : (uint32_t)rb, trans && rb == 32 ? 64 : 128, "adapters");
  }
  if (st != NM_OK) return st;
  cudaError_t e = launch_lora_shrink(p, trans, s);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter shrink launch");
}

// The adapters in the projection's own reduction: a GEMM that serves the shape takes, after its own steps, the blocks
// of 64 rank rows that a column tile's tokens use.  Returns what that GEMM and the mending pass need.
struct InGemm {
  Staged buf;
  GemmExt ext{};
  LoraMend mend{};
  InGemm(cudaStream_t s) : buf(s) {}
};
bool adapters_fit_gemm(const Adapters& ad) { return ad.n > 0 && ad.n * ad.rank <= lora::kMaxCat; }
nm_status adapters_for_gemm(const Adapters& ad, bool trans, int64_t D, int64_t rows, const uint16_t* Z, int64_t ldz,
                            int64_t T, const int32_t* idx, bool f32, InGemm& g, cudaStream_t s) {
  using namespace lora;
  const int64_t cat = (ad.n * ad.rank + 63) / 64 * 64, ldp = (T + 7) / 8 * 8, ldc = trans ? (rows + 7) / 8 * 8 : cat;
  const int planes = f32 ? 3 : 2, nflags = lora_cat_blocks();
  Parts parts;
  const int64_t at_cat = parts.take((trans ? ad.n * ad.rank : rows) * ldc * 2), at_blocks = parts.take(planes * cat * ldp * 2);
  const int64_t at_flags = parts.take(nflags * 4), at_masks = parts.take(tiles_of(T) * 4);
  const int64_t at_inv = parts.take(idx ? rows * 4 : 0);
  cudaError_t e = g.buf.get(parts.size());
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the adapters");
  uint32_t* flags = g.buf.as<uint32_t>(at_flags);
  uint32_t* masks = g.buf.as<uint32_t>(at_masks);
  int32_t* inv = idx ? g.buf.as<int32_t>(at_inv) : nullptr;
  LoraCat c = {};
  c.M = trans ? ad.A : ad.B;
  c.n = ad.n;
  c.rows = rows;
  c.rank = ad.rank;
  c.cat = cat;
  c.ldc = ldc;
  c.idx = idx;
  c.out = g.buf.as<uint16_t>(at_cat);
  c.flags = flags;
  c.inv = inv;
  e = launch_lora_cat(c, trans, s);
  if (e != cudaSuccess) return cuda_fail(e, "adapter layout launch");
  LoraShrink p = {};
  p.out = SHRINK_BLOCKS;
  p.planes = planes;
  p.terms = g.buf.as<uint16_t>(at_blocks);
  p.cat = cat;
  p.ldp = ldp;
  p.masks = masks;
  p.idx = idx;
  p.idx_n = rows;
  p.inv = inv;
  p.early = 1;  // reads nothing of the layout launch (inv is taken at its end)
  nm_status st = shrink(ad, trans, D, Z, ldz, T, p, s);
  if (st != NM_OK) return st;
  g.ext = GemmExt{c.out, trans ? ad.n * ad.rank : rows, trans ? rows : cat, ldc, p.terms, cat, ldp, planes, masks};
  LoraMend& m = g.mend;
  m.M = c.M;
  m.adapter = ad.adapter;
  m.n = ad.n;
  m.rows = rows;
  m.T = T;
  m.rank = ad.rank;
  m.blocks = p.terms;
  m.planes = planes;
  m.cat = cat;
  m.ldp = ldp;
  m.flags = flags;
  m.nflags = nflags;
  m.inv = inv;
  m.out_f32 = f32;
  return NM_OK;
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
  if (st == NM_OK) st = check_operand(values, meta, idx);
  if (st == NM_OK) st = check_spmm(values, meta, n, m, R, K, X, ldx, T, Y, ldy, y_dtype);
  if (st != NM_OK || R == 0 || T == 0) return st;
  if (num_adapters == 0 || K == 0)
    return run_spmm(values, meta, n, m, R, K, idx, X, ldx, T, Y, ldy, y_dtype, nullptr, s);
  st = check_adapter_pointers(ad, R, K, T);
  if (st != NM_OK) return st;
  if (spmm_pair_serves(values, meta, n, m, K, T) && adapters_fit_gemm(ad)) {
    InGemm g(s);
    st = adapters_for_gemm(ad, false, K, R, X, ldx, T, nullptr, y_dtype == NM_OUT_F32, g, s);
    if (st == NM_OK) st = run_spmm(values, meta, n, m, R, K, idx, X, ldx, T, Y, ldy, y_dtype, nullptr, s, &g.ext);
    if (st != NM_OK) return st;
    g.mend.Y = Y;
    g.mend.ldy = ldy;
    cudaError_t e = launch_lora_mend(g.mend, false, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter mending launch");
  }
  Staged low(s), sum(s), partials(s);
  const int64_t ldb = (T + 3) / 4 * 4;
  cudaError_t e = low.get((size_t)(T * lora::rank_stride(rank) * 4));
  if (e == cudaSuccess) e = sum.get((size_t)(R * ldb * 4));
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the projection");
  LoraShrink sh = {};
  sh.out = SHRINK_F32;
  sh.S = low.as<float>();
  st = shrink(ad, false, K, X, ldx, T, sh, s);
  GemmPartials raw{&partials, true, 1, 0, 0};
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
  if (st == NM_OK) st = check_operand(values, meta, idx);
  if (st == NM_OK) st = check_spmm_t(values, meta, n, m, R, K, dY, lddy, T, dX, lddx, dtype);
  if (st != NM_OK || K == 0 || T == 0) return st;
  if (R == 0) return run_spmm_t(values, meta, n, m, R, K, nullptr, dY, lddy, T, dX, lddx, dtype, s);
  if (num_adapters > 0) st = check_adapter_pointers(ad, R, K, T);
  if (st != NM_OK) return st;
  if (adapters_fit_gemm(ad)) {
    InGemm g(s);
    st = adapters_for_gemm(ad, true, R, K, dY, lddy, T, idx, dtype == NM_OUT_F32, g, s);
    if (st == NM_OK) st = run_spmm_t(values, meta, n, m, R, K, idx, dY, lddy, T, dX, lddx, dtype, s, &g.ext);
    if (st != NM_OK) return st;
    g.mend.Y = dX;
    g.mend.ldy = lddx;
    cudaError_t e = launch_lora_mend(g.mend, true, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "adapter mending launch");
  }
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
  LoraShrink sh = {};
  sh.out = SHRINK_F32;
  sh.S = low.as<float>();
  if (num_adapters > 0) st = shrink(ad, true, R, dY, lddy, T, sh, s);
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
  Staged buf(s);
  const int planes = dtype == NM_OUT_F32 ? 3 : 2;
  const int64_t rs = lora::rank_stride(rank), tiles = lora::tiles_of(T);
  Parts parts;
  const int64_t at_plan = parts.take((tiles + 1) * num_adapters * 4);
  const int64_t at_terms[2] = {parts.take(planes * T * rs * 2), parts.take(planes * T * rs * 2)};
  cudaError_t e = buf.get(parts.size());
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer for the adapter gradients");
  LoraOuter p = {};
  p.adapter = adapter;
  p.scale = scale;
  p.n = num_adapters;
  p.T = T;
  p.rank = rank;
  int32_t* counts = buf.as<int32_t>(at_plan);
  p.counts = counts;
  p.tiles = counts + num_adapters;
  p.out_f32 = dtype == NM_OUT_F32;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  e = launch_lora_plan(adapter, T, num_adapters, counts + num_adapters, counts, s);
  if (e != cudaSuccess) return cuda_fail(e, "adapter plan launch");
  const uint32_t box = (uint32_t)lora::outer_box(rank);
  // S = A X for dB and U = B^T dY for dA, then the two gradients: within each pair the second launch needs nothing of
  // the first and runs beside it.
  const bool want[2] = {dB && R > 0, dA && K > 0};
  for (int which = 0; which < 2; ++which) {
    if (!want[which]) continue;
    LoraShrink sh = {};
    sh.out = SHRINK_TERMS;
    sh.planes = planes;
    sh.terms = buf.as<uint16_t>(at_terms[which]);
    sh.early = 1;
    st = which ? shrink(ad, true, R, dY, lddy, T, sh, s) : shrink(ad, false, K, X, ldx, T, sh, s);
    if (st != NM_OK) return st;
  }
  for (int which = 0; which < 2; ++which) {
    if (!want[which]) continue;
    const int64_t rows = which ? K : R;
    st = make_tmap(&p.tm_z, which ? X : dY, (uint64_t)T, (uint64_t)rows, (uint64_t)(which ? ldx : lddy) * 2, lora::kTok,
                   lora::kRows, 128, "tokens");
    if (st == NM_OK)
      st = make_tmap3(&p.tm_v, buf.as<uint16_t>(at_terms[which]), (uint64_t)rs, (uint64_t)T,
                      (uint64_t)planes, (uint64_t)rs * 2, (uint64_t)(T * rs) * 2, box, lora::kTok,
                      box == 64 ? 128 : box == 32 ? 64 : 32, "adapter terms");
    if (st != NM_OK) return st;
    p.rows = rows;
    p.out = which ? dA : dB;
    p.early = which && want[0];
    e = launch_lora_outer(p, which != 0, s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter gradient launch");
  }
  return NM_OK;
}

}  // extern "C"
