// nm_experts_grad.cu -- the two gradients of products grouped by expert (nm_experts.cu), with expert e's columns s:
//   dX[:, s] = W'_e^T dY[:, s]          (experts_t_kernel), and
//   dV_e = the survivors' entries of sum_s dY[:, s] X[:, s]^T   (experts_dv_kernel).
// W'^T is 2:4 along its output axis and the product for dV has no sparse operand, so both are dense MMAs on SM pairs
// (M = 256, N up to 256, two accumulators).
//
// experts_t_kernel reads the compressed weights and expands them on the way to the tensor core: a dense copy of all experts
// would be staged at 16 bits a weight and written and read again, 4.6 times the bytes of the compressed operand (721 MB
// staged for eight experts of 11008 x 4096).  Per CTA and stage of 64 reduction rows (R), TMA brings 64 x 64 stored values
// (8 KB) and their metadata (1 KB) into a ring of their own; eight warps expand them into the MN-major operand tile (two
// strips of 64 columns, 64 rows of 128 bytes each, 128-byte swizzle): a group of four is two byte permutations of its pair
// of values, whose selectors come from a table by the group's nibble.  dY's rows arrive by TMA beside it.
//
// experts_dv_kernel reduces over an expert's columns, which start and end anywhere.  Its stages of 128 columns start as the
// tiles of nm_experts.cuh do; in a tile's first and last stage two warps of each CTA zero the columns outside the expert (of
// both operands: a zero times a neighbour's Inf would be NaN) before the MMA may read them, and these stages issue only the
// MMAs (16 columns each) that hold columns of the expert.  An expert without columns has a gradient of zeros.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "nm_experts.cuh"
#include "nm_experts.h"
#include "nm_host.h"
#include "nm_internal.h"
#include "nm_ptx.cuh"

namespace nmk {

namespace grpt {
// Warps 0 raw copies, 1 MMA, 2 copies of dY, 4-7 epilogue, 8 on expansion.
constexpr uint32_t kVals = 8192, kMeta = 1024;
constexpr uint32_t kA = 16384;  // 64 reduction rows x 128 columns, in strips of 8 KB
constexpr uint32_t kStrip = 8192;
constexpr uint32_t kTmemCols = 512;
constexpr int kWide = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
// Many columns: up to 512 of them a tile, so that weights expanded once meet two accumulators: expansion, copies and operand
// reads together fill shared memory's bandwidth (256 columns: 710 us for 8192 of 11008 x 4096, 512: 600 us).
// FEW: up to 128, K-contiguous; the weights' bytes decide, so their ring is the deep one.
template <bool FEW>
struct Cfg {
  static constexpr int kGroups = 2;  // of four expanding warps, a stage each
  static constexpr int kThreads = 256 + 128 * kGroups;
  static constexpr int kRaw = FEW ? 10 : 4, kStages = FEW ? 4 : 3;
  // A group meets the same slots of the ring of values again and again, so that its parity tells it which turn it sees.
  static_assert(kRaw % kGroups == 0, "whole turns");
  static constexpr uint32_t kB = FEW ? 8192 : 32768;
  static constexpr uint32_t kOffB = kStages * kA, kOffVals = kOffB + kStages * kB, kOffMeta = kOffVals + kRaw * kVals;
  static constexpr uint32_t kOffEpi = kOffMeta + kRaw * kMeta;
  static constexpr uint32_t kOffBar = kOffEpi + 4 * kBoxBytes;
  static constexpr uint32_t kOffTable = kOffBar + (2 * kStages + 2 * kRaw + 5) * 8 + 8;
  static constexpr uint32_t kOffFirst = kOffTable + 128;
  static_assert(kOffTable % 8 == 0, "eight bytes an entry");
  static constexpr uint32_t bytes(int E) { return kOffFirst + 4u * (uint32_t)(2 * E + 1) + 1024u; }
  static_assert(kOffFirst + 4 * (2 * kMaxExperts + 1) + 1024 <= 232448, "shared memory");
};
}  // namespace grpt

// Four weights from their two stored values, as two words, are two byte permutations; their selectors, by the group's nibble
// p0 | p1 << 2: of a half's selector bytes 0x44 picks zeros, 0x10 the first value, 0x32 the second.
__device__ __forceinline__ uint2 selectors(uint32_t nib) {
  const uint32_t sel = 0x44444444u ^ (0x54u << (8u * (nib & 3u))) ^ (0x76u << (8u * (nib >> 2)));
  return make_uint2(sel, sel >> 16);
}
// One row's 16 weights: eight values and, in the low 16 bits of `pos` shifted right by SHIFT, their positions, to two 16-byte
// units.  The selectors come from a table in shared memory (16 entries: lanes meet different banks or the same word), half
// the instructions of making them.
template <int SHIFT>
__device__ __forceinline__ void expand_row(const uint4& v, uint32_t pos, const uint8_t* table, uint4& a, uint4& b) {
  auto group = [&](int g, uint32_t w, uint32_t& lo, uint32_t& hi) {
    const int right = SHIFT + 4 * g - 3;  // eight bytes an entry
    const uint2 sel = *reinterpret_cast<const uint2*>(table + ((right < 0 ? pos << -right : pos >> right) & 0x78u));
    lo = __byte_perm(w, 0u, sel.x);
    hi = __byte_perm(w, 0u, sel.y);
  };
  group(0, v.x, a.x, a.y);
  group(1, v.y, a.z, a.w);
  group(2, v.z, b.x, b.y);
  group(3, v.w, b.z, b.w);
}

template <bool FEW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(grpt::Cfg<FEW>::kThreads, 1)
    experts_t_kernel(const __grid_constant__ ExpertsParams p) {
  using namespace grpt;
  using C = Cfg<FEW>;
  constexpr int kRaw = C::kRaw, kStages = C::kStages;
  constexpr uint32_t kB = C::kB, kOffB = C::kOffB, kOffVals = C::kOffVals, kOffMeta = C::kOffMeta;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* raw_full = empty + kStages;
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* acc_full = raw_empty + kRaw;  // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint64_t* spare = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(spare + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* first = reinterpret_cast<int32_t*>(smem + C::kOffFirst);

  const uint32_t rank = cluster_ctarank();  // 0: leader (issues the MMAs)
  const int pair_id = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + 8);  // dY's bytes, and the expanding warps of both CTAs
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 8);
    }
    mbar_init(spare, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 3 && lane < 16) reinterpret_cast<uint2*>(smem + C::kOffTable)[lane] = selectors((uint32_t)lane);
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&p.tm_vals);
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_meta);
  }
  cluster_sync();  // the allocation takes columns in both SMs: the peer has started
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_enter(FEW);  // no global memory touched before this point; few columns: nothing that the launch before writes
  if (warp == 0) {
    if (FEW)
      list_tiles<ON_UNITS>(p.offsets, p.E, p.S, kSlotCols, p.tiles_m, first, lane);
    else
      list_wide_tiles<kWide>(p.offsets, p.E, p.S, p.tiles_m, first, lane);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const uint32_t lead_full0 = map_to_cta(smem_u32(&full[0]), 0);
  const uint32_t lead_acc_empty0 = map_to_cta(smem_u32(acc_empty), 0);
  bool ok = true;
  auto w = [&] {
    if constexpr (FEW)
      return TileWalk<true, ON_UNITS>(first, p.offsets, p.E, p.S, kSlotCols, p.k_tiles, p.tiles_m, pair_id, npairs);
    else
      return WideWalk<kWide>(first, p.offsets, p.E, p.S, p.k_tiles, p.tiles_m, pair_id, npairs);
  }();

  if (warp == 0) {
    // ------------------------------------------------- values and metadata
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      while (ok && w.next()) {
        const int32_t m0 = w.tm * 256 + 128 * (int)rank;
        for (int kt = w.k0; kt < w.k1; ++kt) {
          ok = mbar_wait(&raw_empty[s], ph ^ 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          mbar_arrive_expect_tx(&raw_full[s], kVals + kMeta);
          tma_load_3d(smem + kOffVals + s * kVals, &p.tm_vals, &raw_full[s], m0 >> 1, kt * 64, w.e);
          tma_load_3d(smem + kOffMeta + s * kMeta, &p.tm_meta, &raw_full[s], 0, m0 >> 7, w.e * p.meta_rblocks + kt * 4);
          if (++s == kRaw) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ dY
    if (lane == 0) {
      if (FEW) pdl_wait();  // the columns laid out by the launch before
      int s = 0;
      uint32_t ph = 0;
      while (ok && w.next()) {
        // Columns in parts of 256, each half to a CTA, in strips of 64.
        const int32_t n0 = min(w.n, 256), n1 = w.n - n0;
        const int32_t col0 = w.x0 + (n0 >> 1) * (int32_t)rank, col1 = w.x0 + 256 + (n1 >> 1) * (int32_t)rank;
        const int s0 = n0 > 128 ? 2 : 1, s1 = (n1 + 127) >> 7;
        for (int kt = w.k0; kt < w.k1; ++kt) {
          ok = mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], FEW ? 128u * (uint32_t)w.n : 2u * (uint32_t)(s0 + s1) * kStrip);
          uint8_t* b = smem + kOffB + s * kB;
          if constexpr (FEW) {  // this CTA's columns, 16 of them a box
            for (int i = 0; i < (n0 >> 1); i += 16)
              tma_load_2d_pair(b + i * 128, &p.tm_x, lead_full0 + 8u * s, kt * 64, col0 + i);
          } else {
            const uint32_t bar = lead_full0 + 8u * s;
            tma_load_2d_pair(b, &p.tm_x, bar, col0, kt * 64);
            if (s0 == 2) tma_load_2d_pair(b + kStrip, &p.tm_x, bar, col0 + 64, kt * 64);
            if (s1 >= 1) tma_load_2d_pair(b + 2 * kStrip, &p.tm_x, bar, col1, kt * 64);
            if (s1 == 2) tma_load_2d_pair(b + 3 * kStrip, &p.tm_x, bar, col1 + 64, kt * 64);
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA (leader)
    if (rank == 0 && lane == 0) {
      // Descriptors of the first slots: their start address counts 16 bytes.
      const uint64_t desc_a = smem_desc(smem_u32(smem), kStrip, 1024, SWZ_128B);
      const uint64_t desc_b = smem_desc(smem_u32(smem + kOffB), FEW ? 16 : kStrip, 1024, SWZ_128B);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      while (ok && w.next()) {
        const int parts = w.n > 256 ? 2 : 1;
        for (int j = 0; j < parts && ok; ++j)
          ok = mbar_wait(&acc_empty[acc ^ j], ((aph >> (acc ^ j)) & 1u) ^ 1u, abort_flag, p.status, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + 256u * (uint32_t)acc, d1 = tmem_base + 256u * (uint32_t)(acc ^ 1);
        const uint32_t idesc0 = idesc_bf16_major((uint32_t)min(w.n, 256), 256, true, !FEW);
        const uint32_t idesc1 = idesc_bf16_major((uint32_t)max(w.n - 256, 32), 256, true, true);
        for (int kt = w.k0; kt < w.k1; ++kt) {
          ok = mbar_wait(&full[s], ph, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = desc_a + (uint64_t)(s * (kA >> 4)), bd = desc_b + (uint64_t)(s * (kB >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_pair(d0, ad + 128u * kk, bd + (FEW ? 2u : 128u) * kk, idesc0, (kt > w.k0 || kk > 0) ? 1u : 0u);
          if (parts == 2) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_pair(d1, ad + 128u * kk, bd + (2 * kStrip >> 4) + 128u * kk, idesc1, (kt > w.k0 || kk > 0) ? 1u : 0u);
          }
          tc_commit_pair(&empty[s], 0x3);
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        for (int j = 0; j < parts; ++j) {
          tc_commit_pair(&acc_full[acc], 0x3);
          aph ^= 1u << acc;
          acc ^= 1;
        }
      }
      if (!ok) {
        tc_commit_pair(spare, 0x1);
        volatile int dummy = 0;
        mbar_wait(spare, 0, &dummy, p.status, 100000000ull);
      }
    }
  } else if (warp >= 8) {
    // ----------------------------------------------------------- expansion
    // Four warps to a stage, two stages at a time (one group alone takes longer than a stage's MMAs; three or four groups
    // are no faster: 135 us with few columns, 145 and 140).  A warp takes 16 rows: two words of metadata a lane, each of a
    // row and its partner eight below.  Eight lanes take four 16-byte units of the values (a half of the columns) in two
    // rows whose numbers differ by 5 in their bits: the swizzle then puts their units of values, and of weights (every other
    // one of a strip), in different banks.
    const int q = (lane & 1) + 2 * ((lane >> 3) & 1), h = (lane >> 1) & 1, rb = warp & 3, mine = (warp - 8) >> 2;
    const int flip = (lane >> 2) & 1 ? 5 : 0, rlow = lane >> 4;
    const uint8_t* table = smem + C::kOffTable;
    const uint32_t u0 = (uint32_t)(4 * (q & 1) + 2 * h);
    const uint32_t out_at = (uint32_t)(q >> 1) * kStrip + (uint32_t)rb * 2048u;
    int s = 0, r = 0, turn = 0;
    uint32_t ph = 0, rph = 0;
    while (ok && w.next()) {
      for (int kt = w.k0; kt < w.k1; ++kt) {
        if (turn == mine) {
          ok = mbar_wait_warp(&raw_full[r], rph, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          uint4 out[2][2][2];  // word, row, unit
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = (rlow + 2 * i) ^ flip;
            const uint8_t* vals = smem + kOffVals + r * kVals + rb * 2048 + rr * 128 + (((2 * q + h) ^ rr) << 4);
            const uint32_t word =
                *reinterpret_cast<const uint32_t*>(smem + kOffMeta + r * kMeta + rb * 256 + 4 * (4 * (rr + 8 * h) + q));
            const uint4 v0 = *reinterpret_cast<const uint4*>(vals), v1 = *reinterpret_cast<const uint4*>(vals + 1024);
            expand_row<0>(v0, word, table, out[i][0][0], out[i][0][1]);
            expand_row<16>(v1, word, table, out[i][1][0], out[i][1][1]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[r]);
          ok = mbar_wait_warp(&empty[s], ph ^ 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t rr = (uint32_t)((rlow + 2 * i) ^ flip);
            uint8_t* a = smem + s * kA + out_at + rr * 128u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              *reinterpret_cast<uint4*>(a + ((u0 ^ rr) << 4) + 1024 * j) = out[i][j][0];
              *reinterpret_cast<uint4*>(a + (((u0 + 1u) ^ rr) << 4) + 1024 * j) = out[i][j][1];
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(lead_full0 + 8u * s);
        }
        if (++turn == C::kGroups) turn = 0;
        if (++s == kStages) { s = 0; ph ^= 1u; }
        if (++r == kRaw) { r = 0; rph ^= 1u; }
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    uint8_t* box = smem + C::kOffEpi + quarter * kBoxBytes;
    uint32_t aph = 0;
    int acc = 0;
    const bool notes = FEW && rank == 0 && quarter == 0 && lane == 0;
    bool noted = false;
    while (ok && w.next()) {
      if constexpr (FEW) {
        if (notes && note_cut(p, w, pair_id, npairs)) noted = true;
      }
      for (int32_t x = 0; x < w.n; x += 256) {  // the parts
        ok = mbar_wait_warp(&acc_full[acc], (aph >> acc) & 1u, abort_flag, p.status, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t_addr = tmem_base + 256u * (uint32_t)acc + ((uint32_t)(quarter * 32) << 16);
        const int row = 128 * (int)rank + quarter * 32;
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(lead_acc_empty0 + 8u * (uint32_t)acc);
        };
        bool whole = true;
        if constexpr (FEW) {
          whole = w.whole();
          if (!whole) store_part(p.parts + (int64_t)(2 * pair_id + w.slot) * kSlotFloats, w, t_addr, row, lane, release);
        }
        if (whole)
          store_tile(p, w.x0 + x, min(w.n - x, 256), w.c0, w.c1, t_addr, box, w.tm * 256 + row, lane, release);
        aph ^= 1u << acc;
        acc ^= 1;
      }
    }
    if (FEW && notes && !noted) p.cuts[pair_id].pairs = 0;
    if (lane == 0) bulk_wait_group<0>();  // every store of this warp has landed
  }

  // -------------------------------------------------------------- teardown
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) sleep_about_ns(200000ull);
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
  cluster_sync();  // ... and so does the deallocation: neither CTA leaves before both are through it
  pdl_leave(FEW);
}

// ------------------------------------------------------------ survivors' gradient
namespace grpv {
constexpr int kThreads = 384;  // warp 0 copies, 1 MMA, 2, 3 columns outside the expert, 4-11 epilogue
constexpr int kStages = 3;
constexpr uint32_t kA = 32768, kB = 32768;  // 128 rows x 128 columns each, in halves of 64 columns
constexpr uint32_t kHalf = 16384;
// Column tiles of a strip, at most: 43 (two experts of 4096 x 11008, 8192 columns each) in strips of 8 993 us, in one
// 1135; 16 (11008 x 4096, eight experts of 1024 columns) in strips of 8 581, in one 572.
constexpr int kAcross = 16;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kOffEpi = kStages * (kA + kB);
constexpr uint32_t kOffBar = kOffEpi + 8 * kBoxBytes;
constexpr uint32_t kSmemBytes = kOffBar + (4 * kStages + 5) * 8 + 8 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

// The stages of one expert's reduction, from its first column rounded down.
struct Reduction {
  int e;
  int32_t c0, c1, a0;
  int stages;
  __device__ __forceinline__ Reduction() : e(-1) {}
  __device__ __forceinline__ void at(const ExpertsGradParams& p, int expert) {
    if (expert == e) return;
    const ExpertCols x = expert_cols(p.offsets, expert, p.S, 256);
    e = expert;
    c0 = x.c0;
    c1 = x.c1;
    a0 = x.a0;
    stages = c1 > c0 ? (c1 - a0 + 127) / 128 : 0;
  }
  // The expert's columns of stage kt, from the stage's first; MMAs take 16 of them each.
  __device__ __forceinline__ int32_t from(int kt) const { return kt == 0 ? c0 - a0 : 0; }  // below 64
  __device__ __forceinline__ int32_t to(int kt) const { return min(c1 - a0 - 128 * kt, 128); }
  // Do the stage's MMAs meet columns of another expert (or behind the matrix)?
  __device__ __forceinline__ bool ragged(int kt) const { return ((from(kt) | to(kt)) & 15) != 0; }
};
}  // namespace grpv

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(grpv::kThreads, 1)
    experts_dv_kernel(const __grid_constant__ ExpertsGradParams p) {
  using namespace grpv;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* landed = empty + kStages;   // a ragged stage's bytes, in each CTA
  uint64_t* masked = landed + kStages;  // ... its columns, in both: stands in for full
  uint64_t* acc_full = masked + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint64_t* spare = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(spare + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();  // 0: leader (issues the MMAs)
  const int pair_id = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
      mbar_init(&masked[s], 4);  // two warps of each CTA
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);
    }
    mbar_init(spare, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&p.tm_a);
    tma_prefetch_desc(&p.tm_b);
  }
  cluster_sync();  // the allocation takes columns in both SMs: the peer has started
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_gate();  // no global memory touched before this point
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const uint32_t lead_full0 = map_to_cta(smem_u32(&full[0]), 0);
  const uint32_t lead_masked0 = map_to_cta(smem_u32(&masked[0]), 0);
  const uint32_t lead_acc_empty0 = map_to_cta(smem_u32(acc_empty), 0);
  const int per_expert = p.tiles_m * p.tiles_n, tiles = p.E * per_expert, wide = strip_width(p.tiles_n, kAcross);
  bool ok = true;
  Reduction red;

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int tile = pair_id; tile < tiles && ok; tile += npairs) {
        red.at(p, tile / per_expert);
        int tm, tn;
        tile_in_strip(tile % per_expert, p.tiles_m, p.tiles_n, wide, tm, tn);
        const int32_t m0 = tm * 256 + 128 * (int)rank, n0 = tn * 256 + 128 * (int)rank;
        for (int kt = 0; kt < red.stages; ++kt) {
          ok = mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          uint8_t* a = smem + s * (kA + kB);
          const int halves = red.to(kt) > 64 ? 2 : 1;
          const uint32_t tx = (uint32_t)halves * 2u * kHalf;  // this CTA's bytes
          const bool ragged = red.ragged(kt);
          if (ragged)
            mbar_arrive_expect_tx(&landed[s], tx);
          else if (rank == 0)
            mbar_arrive_expect_tx(&full[s], 2u * tx);
          const int32_t k0 = red.a0 + kt * 128;
          // Written out for whole stages: by a loop of as many turns as there are halves, a stage's last copies were issued
          // too late (8192 columns of 11008 x 4096 in experts of whole stages: 547 us, written out 503).
          if (ragged) {
            for (int i = 0; i < halves; ++i) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint8_t* to = a + i * kHalf + h * 8192;
                tma_load_2d(to, &p.tm_a, &landed[s], k0 + 64 * i, m0 + 64 * h);
                tma_load_2d(to + kA, &p.tm_b, &landed[s], k0 + 64 * i, n0 + 64 * h);
              }
            }
          } else {
            const uint32_t bar = lead_full0 + 8u * s;
            auto load = [&](int i, int h) {
              uint8_t* to = a + i * kHalf + h * 8192;
              tma_load_2d_pair(to, &p.tm_a, bar, k0 + 64 * i, m0 + 64 * h);
              tma_load_2d_pair(to + kA, &p.tm_b, bar, k0 + 64 * i, n0 + 64 * h);
            };
            load(0, 0);
            load(0, 1);
            if (halves == 2) {
              load(1, 0);
              load(1, 1);
            }
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------- columns outside the expert (of A, of B)
    int s = 0;
    uint32_t lph = 0;  // bit s: phase of landed[s]
    for (int tile = pair_id; tile < tiles && ok; tile += npairs) {
      red.at(p, tile / per_expert);
      for (int kt = 0; kt < red.stages; ++kt) {
        if (red.ragged(kt)) {
          ok = mbar_wait_warp(&landed[s], (lph >> s) & 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          lph ^= 1u << s;
          const int lo = red.from(kt), hi = red.to(kt);
          uint8_t* operand = smem + s * (kA + kB) + (warp - 2) * kA;
          // The two 16-byte units of the MMA step where the columns start, and of the one where they end.
          const int unit = (lane >> 4 ? (hi - 1) >> 4 : lo >> 4) * 2;
          const bool touch = (lane >> 4) == 0 ? (lo & 15) != 0 || (lo >> 4) == ((hi - 1) >> 4)
                                              : (hi & 15) != 0 && (lo >> 4) != ((hi - 1) >> 4);
          if (touch) {
            uint32_t keep[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 8 * unit + 2 * i;
              keep[i >> 2][i & 3] = (k >= lo && k < hi ? 0xFFFFu : 0u) | (k + 1 >= lo && k + 1 < hi ? 0xFFFF0000u : 0u);
            }
#pragma unroll 4
            for (int r = lane & 15; r < 128; r += 16) {
              uint8_t* row = operand + (unit >> 3) * kHalf + r * 128;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint4* at = reinterpret_cast<uint4*>(row + ((((unit & 7) + j) ^ (r & 7)) << 4));
                uint4 u = *at;
                u.x &= keep[j][0];
                u.y &= keep[j][1];
                u.z &= keep[j][2];
                u.w &= keep[j][3];
                *at = u;
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(lead_masked0 + 8u * s);
        }
        if (++s == kStages) s = 0;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA (leader)
    if (rank == 0 && lane == 0) {
      constexpr uint32_t kIdesc = idesc_bf16_major(256, 256, false, false);
      const uint64_t desc = smem_desc(smem_u32(smem), 16, 1024, SWZ_128B);  // its start address counts 16 bytes
      int s = 0, acc = 0;
      uint32_t fph = 0, mph = 0, aph = 0;  // bit s: phase of full[s], of masked[s]
      for (int tile = pair_id; tile < tiles && ok; tile += npairs) {
        red.at(p, tile / per_expert);
        if (red.stages == 0) continue;
        ok = mbar_wait(&acc_empty[acc], ((aph >> acc) & 1u) ^ 1u, abort_flag, p.status, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + 256u * (uint32_t)acc;
        for (int kt = 0; kt < red.stages; ++kt) {
          const bool ragged = red.ragged(kt);
          ok = mbar_wait(ragged ? &masked[s] : &full[s], ((ragged ? mph : fph) >> s) & 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          (ragged ? mph : fph) ^= 1u << s;
          tc_fence_after();
          const uint64_t ad = desc + (uint64_t)(s * ((kA + kB) >> 4)), bd = ad + (kA >> 4);
          const int step0 = red.from(kt) >> 4, steps = (red.to(kt) + 15) >> 4;
          auto step = [&](int kk) {
            const uint32_t at = (uint32_t)(kk >> 2) * (kHalf >> 4) + (uint32_t)(kk & 3) * 2u;
            tc_mma_pair(d_tmem, ad + at, bd + at, kIdesc, (kt > 0 || kk > step0) ? 1u : 0u);
          };
          if (steps - step0 == 8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) step(kk);
          } else {
#pragma unroll 1
            for (int kk = step0; kk < steps; ++kk) step(kk);
          }
          tc_commit_pair(&empty[s], 0x3);
          if (++s == kStages) s = 0;
        }
        if (!ok) break;
        tc_commit_pair(&acc_full[acc], 0x3);
        aph ^= 1u << acc;
        acc ^= 1;
      }
      if (!ok) {
        tc_commit_pair(spare, 0x1);
        volatile int dummy = 0;
        mbar_wait(spare, 0, &dummy, p.status, 100000000ull);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    // A warp takes 32 rows by half of the tile's columns: 64 survivors of every row, through its staging tile as one TMA
    // store (stored by the lanes, a row each, every 16 bytes were a line of L1 of their own: 290 us of 11008 x 4096, eight
    // experts of one column, by four warps); with a release at cluster scope for each accumulator 174 us, without 133).
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    uint8_t* box = smem + kOffEpi + (warp - 4) * kBoxBytes;
    uint32_t aph = 0;
    int acc = 0;
    // The positions of a tile's survivors in this row: asked for a tile ahead.
    uint32_t word[2][4], next[2][4];
    auto positions = [&](int tile, uint32_t (&w)[2][4]) {
      const int e = tile / per_expert;
      int tm, tn;
      tile_in_strip(tile - e * per_expert, p.tiles_m, p.tiles_n, wide, tm, tn);
      const int64_t row = (int64_t)tm * 256 + 128 * rank + quarter * 32 + lane, n0 = (int64_t)tn * 256 + 128 * half;
      const uint32_t* mb = p.meta + e * p.meta_words + ((row >> 4) * p.meta_cblocks + (n0 >> 7)) * 64 + 4 * (row & 7);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in_w = tile < tiles && row < p.R && n0 + 32 * c < p.K;
        w[0][c] = in_w ? __ldcg(mb + c) : 0u;
        w[1][c] = in_w ? __ldcg(mb + c + 32) : 0u;
      }
    };
    positions(pair_id, next);
    for (int tile = pair_id; tile < tiles && ok; tile += npairs) {
      red.at(p, tile / per_expert);
      int tm, tn;
      tile_in_strip(tile % per_expert, p.tiles_m, p.tiles_n, wide, tm, tn);
      const int32_t wrow0 = tm * 256 + 128 * (int)rank + quarter * 32;
      const int64_t row = wrow0 + lane, n0 = (int64_t)tn * 256 + 128 * half;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) word[i][c] = next[i][c];
      positions(tile + npairs, next);
      const bool some = red.stages > 0;
      if (some) {
        ok = mbar_wait_warp(&acc_full[acc], (aph >> acc) & 1u, abort_flag, p.status, kWaitNs);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t t_addr = tmem_base + 256u * (uint32_t)acc + 128u * (uint32_t)half + ((uint32_t)(quarter * 32) << 16);
      const int sh = 16 * (int)((row >> 3) & 1);
      auto take = [&](int c, uint32_t (&v)[32]) {
        if (some) {
          tmem_ld_32x32b_x32(t_addr + c * 32, v);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
      };
      auto stage = [&](int unit, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
        *reinterpret_cast<uint4*>(box + lane * 128 + ((unit ^ (lane & 7)) << 4)) = make_uint4(x, y, z, u);
      };
      auto free_box = [&] {
        if (lane == 0) bulk_wait_group_read<0>();  // the previous store has read it
        __syncwarp();
      };
      auto send = [&](int32_t x) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && wrow0 < p.R && n0 < p.K) {
          tma_store_3d(&p.tm_dv, box, x, wrow0, red.e);
          bulk_commit_group();
        }
      };
      auto release = [&] {
        if (!some) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(lead_acc_empty0 + 8u * (uint32_t)acc);
        aph ^= 1u << acc;
        acc ^= 1;
      };
      if (p.out_f32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          take(c, v);
          if (c == 3) release();
          if (!(c & 1)) free_box();
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t nib = (word[i >> 2][c] >> (sh + 4 * ((i + j) & 3))) & 0xFu;
              const uint32_t p0 = nib & 3u, p1 = nib >> 2;
              const uint32_t* g = v + 4 * (i + j);
              o[2 * j] = p0 == 0 ? g[0] : (p0 == 1 ? g[1] : g[2]);
              o[2 * j + 1] = p1 == 3 ? g[3] : (p1 == 2 ? g[2] : g[1]);
            }
            stage(4 * (c & 1) + (i >> 1), o[0], o[1], o[2], o[3]);
          }
          if (c & 1) send((int32_t)n0 + 64 * (c >> 1));  // 32 survivors a box, two 16-bit units each
        }
      } else {
        free_box();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          take(c, v);
          if (c == 3) release();
          // Rounded first: one byte permutation of a group's four values then picks both survivors (position q is the
          // bytes 2q and 2q + 1).
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t nib = word[i >> 2][c] >> (sh + 4 * (i & 3));
            const uint32_t pick = (nib & 3u) * 0x22u + (nib >> 2 & 3u) * 0x2200u + 0x1010u;
            o[i] = __byte_perm(pack_bf16x2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])),
                               pack_bf16x2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), pick);
          }
          stage(2 * c, o[0], o[1], o[2], o[3]);
          stage(2 * c + 1, o[4], o[5], o[6], o[7]);
        }
        send((int32_t)(n0 >> 1));
      }
    }
    if (lane == 0) bulk_wait_group<0>();  // every store of this warp has landed
  }

  // -------------------------------------------------------------- teardown
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) sleep_about_ns(200000ull);
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
  cluster_sync();  // ... and so does the deallocation: neither CTA leaves before both are through it
}

}  // namespace nmk

using namespace nmk;

extern "C" nm_status nm_experts_spmm_t(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t E, int64_t R,
                                       int64_t K, const uint16_t* dY, int64_t lddy, int64_t S, const int32_t* offsets,
                                       void* dX, int64_t lddx, nm_out_dtype dtype, void* stream) {
  set_last_error("");
  nm_status st = check_experts(n, m, E, R, K, S, offsets);
  if (st != NM_OK) return st;
  if (!dtype_ok(dtype)) return fail(NM_ERR_INVALID_ARG, "bad output dtype");
  if (R < 1) return fail(NM_ERR_INVALID_ARG, "R must be positive");
  if (E == 0 || S == 0) return NM_OK;
  if (!values || !meta) return fail(NM_ERR_INVALID_ARG, "values or meta is null");
  st = check_matrix(dY, lddy, S, 2, "dY");
  if (st == NM_OK) st = check_matrix(dX, lddx, S, dtype_bytes(dtype), "dX");
  if (st != NM_OK) return st;
  if (!al16(values) || !al16(meta)) return fail(NM_ERR_MISALIGNED, "values and meta must be 16-byte aligned");
  st = require_device();
  if (st != NM_OK) return st;
  ExpertsParams p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.Y = dX;
  p.ldy = lddx;
  p.M = (int32_t)K;
  p.S = (int32_t)S;
  p.E = (int32_t)E;
  p.k_tiles = (int32_t)((R + 63) / 64);
  p.tiles_m = (int32_t)((K + 255) / 256);
  p.meta_rblocks = (int32_t)meta_row_blocks(R);
  p.out_f32 = dtype == NM_OUT_F32;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  st = make_tmap3(&p.tm_vals, values, (uint64_t)(K / 2), (uint64_t)R, (uint64_t)E, (uint64_t)K, (uint64_t)(R * K), 64, 64, 128,
                  "values");
  if (st == NM_OK) st = make_meta_tmap(&p.tm_meta, meta, E * meta_row_blocks(R), meta_col_blocks(K), 4);
  if (st == NM_OK) st = make_experts_store_map(p, dX, K, S, lddx);
  if (st != NM_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (few_columns(p, 0.41, 0.44)) {
    Staged staged(s);
    st = stage_few(p, dY, lddy, R, staged, s);
    if (st != NM_OK) return st;
    static SmemLimit limit;
    e = limit.raise(experts_t_kernel<true>, grpt::Cfg<true>::bytes(kMaxExperts));
    if (e == cudaSuccess) {
      e = launch_pdl(experts_t_kernel<true>, dim3(2 * (unsigned)(sm_count_current() / 2)), dim3(grpt::Cfg<true>::kThreads),
                     grpt::Cfg<true>::bytes(p.E), s, p);
      count_launch();
    }
    return e == cudaSuccess ? join_few(p, s) : cuda_fail(e, "grouped input gradient launch");
  }
  st = make_tmap(&p.tm_x, dY, (uint64_t)S, (uint64_t)R, (uint64_t)lddy * 2, 64, 64, 128, "dY");
  if (st != NM_OK) return st;
  static SmemLimit limit;
  e = limit.raise(experts_t_kernel<false>, grpt::Cfg<false>::bytes(kMaxExperts));
  if (e != cudaSuccess) return cuda_fail(e, "grouped input gradient");
  const int pairs = experts_pairs(p, grpt::kWide);
  e = launch_pdl(experts_t_kernel<false>, dim3(2 * pairs), dim3(grpt::Cfg<false>::kThreads),
                 grpt::Cfg<false>::bytes(p.E), s, p);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "grouped input gradient launch");
}

extern "C" nm_status nm_experts_sddmm(const uint32_t* meta, int n, int m, int64_t E, int64_t R, int64_t K, const uint16_t* dY,
                                      int64_t lddy, const uint16_t* X, int64_t ldx, int64_t S, const int32_t* offsets,
                                      void* dV, nm_out_dtype dtype, void* stream) {
  set_last_error("");
  nm_status st = check_experts(n, m, E, R, K, S, offsets);
  if (st != NM_OK) return st;
  if (!dtype_ok(dtype)) return fail(NM_ERR_INVALID_ARG, "bad output dtype");
  if (E == 0 || R == 0) return NM_OK;
  if (!meta || !dV) return fail(NM_ERR_INVALID_ARG, "meta or dV is null");
  if (!al16(dV)) return fail(NM_ERR_MISALIGNED, "dV must be 16-byte aligned");
  st = check_words({meta}, "meta");
  if (st == NM_OK && S > 0) st = check_matrix(dY, lddy, S, 2, "dY");
  if (st == NM_OK && S > 0) st = check_matrix(X, ldx, S, 2, "X");
  if (st != NM_OK) return st;
  const int64_t tiles_m = (R + 255) / 256, tiles_n = (K + 255) / 256;
  if (E * tiles_m * tiles_n >= kMaxDim - 1024) return fail(NM_ERR_UNSUPPORTED, "too many tiles");
  st = require_device();
  if (st != NM_OK) return st;
  if (S == 0) {  // no columns: zeros (offsets may be null)
    const cudaError_t e = cudaMemsetAsync(dV, 0, (size_t)(E * R * (K / 2) * dtype_bytes(dtype)), (cudaStream_t)stream);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "zero gradient");
  }
  ExpertsGradParams p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.meta = meta;
  p.dV = dV;
  p.R = R;
  p.K = K;
  p.S = (int32_t)S;
  p.E = (int32_t)E;
  p.tiles_m = (int32_t)tiles_m;
  p.tiles_n = (int32_t)tiles_n;
  p.meta_cblocks = (int32_t)meta_col_blocks(K);
  p.meta_words = meta_words(R, K, 2, 4);
  p.out_f32 = dtype == NM_OUT_F32;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  st = make_tmap(&p.tm_a, dY, (uint64_t)S, (uint64_t)R, (uint64_t)lddy * 2, 64, 64, 128, "dY");
  if (st == NM_OK) st = make_tmap(&p.tm_b, X, (uint64_t)S, (uint64_t)K, (uint64_t)ldx * 2, 64, 64, 128, "X");
  const int64_t units = p.out_f32 ? K : K / 2;  // 16-bit units of a row
  if (st == NM_OK)
    st = make_tmap3(&p.tm_dv, dV, (uint64_t)units, (uint64_t)R, (uint64_t)E, (uint64_t)units * 2, (uint64_t)(R * units) * 2, 64,
                    32, 128, "dV");
  if (st != NM_OK) return st;
  static SmemLimit limit;
  cudaError_t e = limit.raise(experts_dv_kernel, grpv::kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e, "grouped survivor gradient");
  const int64_t tiles = E * tiles_m * tiles_n;
  const int pairs_avail = sm_count_current() / 2;
  const int pairs = tiles < pairs_avail ? (int)tiles : pairs_avail;
  e = launch_pdl(experts_dv_kernel, dim3(2 * pairs), dim3(grpv::kThreads), (size_t)grpv::kSmemBytes, (cudaStream_t)stream, p);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "grouped survivor gradient launch");
}
