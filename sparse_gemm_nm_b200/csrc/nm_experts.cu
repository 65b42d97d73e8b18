// nm_experts.cu -- products grouped by expert: Y[:, s] = W'_e X[:, s] for the columns s of expert e, W'_e the expert's 2:4
// weight, from the compressed operand on the sparse tensor cores of SM pairs.
//
// One persistent launch covers all experts.  The pairs derive the list of tiles from the device's offsets
// (nm_experts.cuh), so no count is needed on the host.  A tile is 256 rows of one expert by up to 256 of its columns; its
// width is a run-time operand of the MMA, in steps of 32, so that an expert with few columns costs few MMA cycles, and its
// X copies only the 64-column strips that the width reaches.
//
// Per CTA and stage of 128 logical K (as in nm_spmm_pair.cu, whose layouts these are): A 128 rows of compressed values
// (16 KB), E their metadata (2 KB), B 128 rows of X by this CTA's half of the columns, in strips of 64 (16 KB each).  The
// boxes of values come from a map of three axes, so rows past an expert's last read as zeros and not as the next expert's.
// K may end inside a stage: values and X read as zeros there, and the padded metadata is valid.
//
// Forms (MAXN columns a tile, ACC accumulators):
//   256, 1  many columns.  As in nm_spmm_pair.cu the whole accumulator leaves TMEM for registers before it is stored.
//   224, 2  the same for short K, where the hand-over of the accumulator is a large part of a tile.
//   128, 2  few columns per expert: bound by reading the weights once, so six stages of 34 KB instead of four of 50 KB.
//
// Stores: 64-column boxes that lie inside the expert's columns leave as TMA stores; in the boxes that hold an expert's
// first and last columns, lanes store 16-byte units, and the units that two experts share element by element.
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

namespace grp {
constexpr int kThreads = 320;  // warps 0, 2 values; 3, 4 X; 5 metadata; 1 MMA; 6-9 epilogue
constexpr uint32_t kA = 16384, kE = 2048;
constexpr uint32_t kStrip = 16384;  // 128 rows x 64 columns of X
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

template <int MAXN, int ACC>
struct Cfg {
  static constexpr int kStrips = MAXN > 128 ? 2 : 1;  // of one CTA
  static constexpr int kStages = kStrips == 2 ? 4 : 6;
  static constexpr uint32_t kB = kStrips * kStrip;
  static constexpr uint32_t kECol = ACC == 1 ? 256u : 256u + (MAXN + 31) / 32 * 32;  // TMEM column of the metadata
  static constexpr uint32_t kOffB = kStages * kA, kOffE = kOffB + kStages * kB, kOffEpi = kOffE + kStages * kE;
  static constexpr uint32_t kOffBar = kOffEpi + 4 * kBoxBytes;
  static constexpr uint32_t kOffFirst = kOffBar + (2 * kStages + 5) * 8 + 8;
  static constexpr uint32_t bytes(int E) { return kOffFirst + 4u * (uint32_t)(E + 1) + 1024u; }
  static_assert(kECol + 4 * kStages <= kTmemCols, "TMEM columns");
  static_assert(kOffFirst + 4 * (kMaxExperts + 1) + 1024 <= 232448, "shared memory");
};

}  // namespace grp

template <int MAXN, int ACC, bool FEW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(grp::kThreads, 1)
    experts_pair_kernel(const __grid_constant__ ExpertsParams p) {
  using namespace grp;
  using C = Cfg<MAXN, ACC>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2]
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
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
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
  if (warp == 0) list_tiles<FEW ? ON_UNITS : FEWEST_TILES>(p.offsets, p.E, p.S, MAXN, p.tiles_m, first, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const uint32_t lead_full0 = map_to_cta(smem_u32(&full[0]), 0);
  const uint32_t lead_acc_empty0 = map_to_cta(smem_u32(acc_empty), 0);
  bool ok = true;
  TileWalk<FEW, FEW ? ON_UNITS : FEWEST_TILES> w(first, p.offsets, p.E, p.S, MAXN, p.k_tiles, p.tiles_m, pair_id, npairs);

  if (warp == 1) {
    // ---------------------------------------------------------- MMA (leader)
    if (rank == 0 && lane == 0) {
      // Descriptors of the first slots: their start address counts 16 bytes.
      const uint64_t desc_a = smem_desc(smem_u32(smem), 16, 1024, SWZ_128B);
      const uint64_t desc_b = smem_desc(smem_u32(smem + C::kOffB), FEW ? 16 : kStrip, 1024, SWZ_128B);
      const uint64_t desc_e = smem_desc(smem_u32(smem + C::kOffE), 2048, 128, SWZ_NONE);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;  // aph bit a: phase of accumulator a
      while (ok && w.next()) {
        ok = mbar_wait(&acc_empty[acc], ((aph >> acc) & 1u) ^ 1u, abort_flag, p.status, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + 256u * (uint32_t)acc;
        const uint32_t idesc = idesc_bf16((uint32_t)w.n, true, 256) & ~(FEW ? 1u << 16 : 0u);  // B's major axis
        for (int kt = w.k0; kt < w.k1; ++kt) {
          ok = mbar_wait(&full[s], ph, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = desc_a + (uint64_t)(s * (kA >> 4)), bd = desc_b + (uint64_t)(s * (C::kB >> 4));
          const uint32_t e_tmem = tmem_base + C::kECol + 4u * (uint32_t)s;
          tc_cp_128x128b_pair(e_tmem, desc_e + (uint64_t)(s * (kE >> 4)));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_sp_pair(d_tmem, ad + 2u * kk, bd + (FEW ? (kk >> 1) * 512u + (kk & 1) * 4u : kk * 256u),
                           e_tmem + (uint32_t)(kk & 2), idesc | (uint32_t)(kk & 1), (kt > w.k0 || kk > 0) ? 1u : 0u);
          tc_commit_pair(&empty[s], 0x3);
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(&acc_full[acc], 0x3);
        aph ^= 1u << acc;
        if (ACC == 2) acc ^= 1;
      }
      if (!ok) {
        tc_commit_pair(spare, 0x1);
        volatile int dummy = 0;
        mbar_wait(spare, 0, &dummy, p.status, 100000000ull);
      }
    }
  } else if (warp < 6) {
    // ------ copies, each warp a part of every stage: 0, 2 halves of the values, 3, 4 K halves of X, 5 the metadata
    if (lane == 0) {
      if (FEW && (warp == 3 || warp == 4)) pdl_wait();  // the columns laid out by the launch before
      int s = 0;
      uint32_t ph = 0;
      while (ok && w.next()) {
        const int32_t row0 = w.tm * 256 + 128 * (int)rank;
        const int32_t col0 = w.x0 + (w.n >> 1) * (int32_t)rank;
        const int strips = C::kStrips == 2 && w.n > 128 ? 2 : 1;
        for (int kt = w.k0; kt < w.k1; ++kt) {
          ok = mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, kWaitNs);
          if (!ok) break;
          const uint32_t bar = lead_full0 + 8u * s;
          if (warp == 0 || warp == 2) {
            const int h = warp >> 1;
            if (rank == 0 && h == 0)
              mbar_arrive_expect_tx(&full[s], 2u * (kA + kE + (FEW ? 128u * (uint32_t)w.n : (uint32_t)strips * kStrip)));
            tma_load_3d_pair(smem + s * kA + h * 8192, &p.tm_vals, bar, kt * 64, row0 + 64 * h, w.e);
          } else if (warp <= 4) {
            const int h = warp - 3;
            uint8_t* b = smem + C::kOffB + s * C::kB + h * 8192;
            if constexpr (FEW) {  // K half h of this CTA's columns, 16 of them a box
              for (int i = 0; i < (w.n >> 1); i += 16)
                tma_load_2d_pair(b + i * 128, &p.tm_x, bar, kt * 128 + 64 * h, col0 + i);
              if (++s == kStages) { s = 0; ph ^= 1u; }
              continue;
            }
            tma_load_2d_pair(b, &p.tm_x, bar, col0, kt * 128 + 64 * h);
            if (strips == 2) tma_load_2d_pair(b + kStrip, &p.tm_x, bar, col0 + 64, kt * 128 + 64 * h);
          } else {
            tma_load_3d_pair(smem + C::kOffE + s * kE, &p.tm_meta, bar, 0, kt, w.e * p.meta_rblocks + row0 / 16);
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else {
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
      ok = mbar_wait_warp(&acc_full[acc], (aph >> acc) & 1u, abort_flag, p.status, kWaitNs);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_addr = tmem_base + 256u * (uint32_t)acc + ((uint32_t)(quarter * 32) << 16);
      const int32_t wrow0 = w.tm * 256 + 128 * (int)rank + quarter * 32;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(lead_acc_empty0 + 8u * (uint32_t)acc);
      };
      if constexpr (FEW) {
        if (!w.whole()) {
          store_part(p.parts + (int64_t)(2 * pair_id + w.slot) * kSlotFloats, w, t_addr, wrow0 & 255, lane, release);
          aph ^= 1u << acc;
          if (ACC == 2) acc ^= 1;
          continue;
        }
      }
      if (ACC == 2 || p.out_f32) {
        store_tile(p, w.x0, w.n, w.c0, w.c1, t_addr, box, wrow0, lane, release);
      } else {
        const int32_t end = min(w.c1, w.x0 + w.n);
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (64 * c < w.n) {
            take_bf16(t_addr + c * 64, v[c]);
            take_bf16(t_addr + c * 64 + 32, v[c] + 16);
          }
        }
        release();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (64 * c < w.n) store_chunk<uint16_t>(p, v[c], box, w.x0 + 64 * c, w.c0, end, wrow0, lane);
      }
      aph ^= 1u << acc;
      if (ACC == 2) acc ^= 1;
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

// Tiles that several pairs have parts of: their sums in the order of the stages, rounded and stored.  CTA (pair, slab): the
// tile that this pair has noted, some of its rows, several parts of an element on their way at once.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(256) experts_join_kernel(const __grid_constant__ ExpertsParams p) {
  pdl_gate();
  const int4* at_cut = reinterpret_cast<const int4*>(p.cuts + blockIdx.x);
  const int4 a = __ldcg(at_cut), b = __ldcg(at_cut + 1);
  const int pairs = a.x, slot = a.y, row0 = a.z, x0 = a.w, n = b.x, c0 = b.y, c1 = b.z;
  if (pairs == 0) return;
  const float* head = p.parts + (int64_t)(2 * (int)blockIdx.x + slot) * kSlotFloats;
  const float* rest = p.parts + (int64_t)(2 * (int)blockIdx.x + 2) * kSlotFloats;
  for (int i = threadIdx.x; i < kJoinRows * n; i += 256) {
    const int r = (int)blockIdx.y * kJoinRows + i / n, c = i % n;
    const int64_t row = row0 + r;
    const int32_t col = x0 + c;
    if (row >= p.M || col < c0 || col >= c1) continue;
    const int64_t at = (int64_t)r * n + c;
    float sum = __ldcg(head + at);
    const float* part = rest + at;
    int q = 1;
    for (; q + 4 <= pairs; q += 4, part += 8 * kSlotFloats) {
      const float f0 = __ldcg(part), f1 = __ldcg(part + 2 * kSlotFloats), f2 = __ldcg(part + 4 * kSlotFloats),
                  f3 = __ldcg(part + 6 * kSlotFloats);
      sum = (((sum + f0) + f1) + f2) + f3;
    }
    for (; q < pairs; ++q, part += 2 * kSlotFloats) sum += __ldcg(part);
    if (p.out_f32)
      static_cast<float*>(p.Y)[row * p.ldy + col] = sum;
    else
      static_cast<uint16_t*>(p.Y)[row * p.ldy + col] = (uint16_t)(pack_bf16x2(sum, 0.f) & 0xFFFFu);
  }
}

// XT (S rows of `pitch`, an even number) = X^T (K x S), 64 x 64 a CTA.
__global__ void __launch_bounds__(256) columns_kernel(const uint16_t* X, int64_t ldx, int32_t K, int32_t S, uint16_t* XT,
                                                      int64_t pitch) {
  __shared__ uint16_t tile[64][66];
  const int32_t k0 = (int32_t)blockIdx.x * 64, s0 = (int32_t)blockIdx.y * 64;
  const int wide = min(64, S - s0), deep = min(64, K - k0), two = (wide + 1) >> 1;
  pdl_gate();
#pragma unroll 4
  for (int i = threadIdx.x; i < deep * two; i += 256) {
    const int k = i / two, s = (i - k * two) * 2;
    const uint16_t* at = X + (int64_t)(k0 + k) * ldx + s0 + s;
    const uint32_t v = s + 1 < wide ? __ldcg(reinterpret_cast<const uint32_t*>(at)) : (uint32_t)__ldcg(at);
    tile[s][k] = (uint16_t)v;
    tile[s + 1][k] = (uint16_t)(v >> 16);
  }
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < wide * 32; i += 256) {
    const int s = i >> 5, k = (i & 31) * 2;
    if (k < deep)
      *reinterpret_cast<uint32_t*>(XT + (s0 + s) * pitch + k0 + k) = *reinterpret_cast<const uint32_t*>(&tile[s][k]);
  }
}

template <int MAXN, int ACC, bool FEW>
static cudaError_t launch_experts(const ExpertsParams& p, int pairs, cudaStream_t stream) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(experts_pair_kernel<MAXN, ACC, FEW>, grp::Cfg<MAXN, ACC>::bytes(kMaxExperts));
  if (e != cudaSuccess) return e;
  e = launch_pdl(experts_pair_kernel<MAXN, ACC, FEW>, dim3(2 * pairs), dim3(grp::kThreads), grp::Cfg<MAXN, ACC>::bytes(p.E),
                 stream, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

nm_status stage_few(ExpertsParams& p, const uint16_t* X, int64_t ldx, int64_t K, Staged& staged, cudaStream_t stream) {
  const int64_t pairs = sm_count_current() / 2, pitch = (K + 7) / 8 * 8;
  Parts parts;
  const int64_t at_parts = parts.take(pairs * 2 * kSlotFloats * 4), at_x = parts.take(pitch * p.S * 2),
                at_cuts = parts.take(pairs * (int64_t)sizeof(ExpertsCut));
  cudaError_t e = staged.get(parts.size());
  if (e != cudaSuccess) return cuda_fail(e, "staging buffer of a grouped product");
  p.parts = staged.as<float>(at_parts);
  p.cuts = staged.as<ExpertsCut>(at_cuts);
  uint16_t* XT = staged.as<uint16_t>(at_x);
  nm_status st = make_tmap(&p.tm_x, XT, (uint64_t)K, (uint64_t)p.S, (uint64_t)pitch * 2, 64, 16, 128, "X (K contiguous)");
  if (st != NM_OK) return st;
  e = launch_pdl(columns_kernel, dim3((unsigned)((K + 63) / 64), (unsigned)((p.S + 63) / 64)), dim3(256), 0, stream, X, ldx,
                 (int32_t)K, p.S, XT, pitch);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "grouped product launch");
}

nm_status join_few(const ExpertsParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)(sm_count_current() / 2), 256 / kJoinRows);
  cudaError_t e = launch_pdl(experts_join_kernel, grid, dim3(256), 0, stream, p);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "grouped product launch");
}

bool few_columns(const ExpertsParams& p, double few_us, double wide_us) {
  if (p.S > 32 * (int64_t)p.E || p.S > (int64_t)p.M / 16 * p.E || (p.S + 63) / 64 >= 65536) return false;
  const int64_t tiles = (int64_t)p.tiles_m * (p.E < p.S ? p.E : p.S), pairs = sm_count_current() / 2;
  const double most_stages = (double)((tiles + pairs - 1) / pairs * p.k_tiles);  // of a pair's whole tiles
  return 9. + few_us * (double)(tiles * p.k_tiles) / (double)pairs < wide_us * most_stages;
}

int experts_pairs(const ExpertsParams& p, int max_n) {
  const int64_t most = (int64_t)p.tiles_m * (p.S / max_n + (p.E < p.S ? p.E : p.S) + 1);
  const int pairs = sm_count_current() / 2;
  return most < pairs ? (int)most : pairs;
}

nm_status make_experts_store_map(ExpertsParams& p, void* Y, int64_t M, int64_t S, int64_t ldy) {
  return p.out_f32 ? make_tmap(&p.tm_y, Y, (uint64_t)S, (uint64_t)M, (uint64_t)ldy * 4, 32, 32, 128, "Y (fp32)",
                               CU_TENSOR_MAP_DATA_TYPE_FLOAT32)
                   : make_tmap(&p.tm_y, Y, (uint64_t)S, (uint64_t)M, (uint64_t)ldy * 2, 64, 32, 128, "Y");
}

nm_status check_experts(int n, int m, int64_t E, int64_t R, int64_t K, int64_t S, const int32_t* offsets) {
  if (E < 0 || R < 0 || K < 0 || S < 0) return fail(NM_ERR_INVALID_ARG, "negative dimension");
  if (!pattern_ok(n, m)) return fail(NM_ERR_INVALID_ARG, "pattern %d:%d not supported", n, m);
  if (K < 1 || K % m != 0) return fail(NM_ERR_INVALID_ARG, "K=%lld is not a positive multiple of M=%d", (long long)K, m);
  if (n != 2 || m != 4) return fail(NM_ERR_UNSUPPORTED, "products grouped by expert take 2:4, not %d:%d", n, m);
  if (K % 16 != 0) return fail(NM_ERR_UNSUPPORTED, "K=%lld is not a multiple of 16", (long long)K);
  if (E > kMaxExperts) return fail(NM_ERR_UNSUPPORTED, "more than %d experts", kMaxExperts);
  const int64_t lim = kMaxDim - 4096;  // tile corners are 32-bit
  if (R >= lim || K >= lim || S >= lim || E * ((R + 15) / 16) >= lim ||
      (S / 128 + E + 1) * ((R > K ? R : K) / 256 + 1) >= lim)
    return fail(NM_ERR_UNSUPPORTED, "dimensions too large");
  if (E > 0 && S > 0 && !offsets) return fail(NM_ERR_INVALID_ARG, "offsets is null");
  return check_words({offsets}, "offsets");
}

}  // namespace nmk

using namespace nmk;

extern "C" nm_status nm_experts_spmm(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t E, int64_t R,
                                     int64_t K, const uint16_t* X, int64_t ldx, int64_t S, const int32_t* offsets, void* Y,
                                     int64_t ldy, nm_out_dtype y_dtype, void* stream) {
  set_last_error("");
  nm_status st = check_experts(n, m, E, R, K, S, offsets);
  if (st != NM_OK) return st;
  if (!dtype_ok(y_dtype)) return fail(NM_ERR_INVALID_ARG, "bad output dtype");
  if (E == 0 || R == 0 || S == 0) return NM_OK;
  if (!values || !meta) return fail(NM_ERR_INVALID_ARG, "values or meta is null");
  st = check_matrix(X, ldx, S, 2, "X");
  if (st == NM_OK) st = check_matrix(Y, ldy, S, dtype_bytes(y_dtype), "Y");
  if (st != NM_OK) return st;
  if (!al16(values) || !al16(meta)) return fail(NM_ERR_MISALIGNED, "values and meta must be 16-byte aligned");
  st = require_device();
  if (st != NM_OK) return st;
  ExpertsParams p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.Y = Y;
  p.ldy = ldy;
  p.M = (int32_t)R;
  p.S = (int32_t)S;
  p.E = (int32_t)E;
  p.k_tiles = (int32_t)((K + 127) / 128);
  p.tiles_m = (int32_t)((R + 255) / 256);
  p.meta_rblocks = (int32_t)meta_row_blocks(R);
  p.out_f32 = y_dtype == NM_OUT_F32;
  p.status = status_word_ptr();
  if (!p.status) return fail(NM_ERR_CUDA, "device status word is unavailable");
  st = make_tmap3(&p.tm_vals, values, (uint64_t)(K / 2), (uint64_t)R, (uint64_t)E, (uint64_t)K, (uint64_t)(R * K), 64, 64, 128,
                  "values");
  if (st == NM_OK) st = make_meta_tmap(&p.tm_meta, meta, E * meta_row_blocks(R), meta_col_blocks(K));
  if (st == NM_OK) st = make_experts_store_map(p, Y, R, S, ldy);
  if (st != NM_OK) return st;
  if (few_columns(p, 0.42, 0.56)) {
    Staged staged((cudaStream_t)stream);
    st = stage_few(p, X, ldx, K, staged, (cudaStream_t)stream);
    if (st != NM_OK) return st;
    const cudaError_t e = launch_experts<128, 2, true>(p, sm_count_current() / 2, (cudaStream_t)stream);
    return e == cudaSuccess ? join_few(p, (cudaStream_t)stream) : cuda_fail(e, "grouped product launch");
  }
  st = make_tmap(&p.tm_x, X, (uint64_t)S, (uint64_t)K, (uint64_t)ldx * 2, 64, 64, 128, "X");
  if (st != NM_OK) return st;
  const cudaError_t e = p.k_tiles <= 8 ? launch_experts<224, 2, false>(p, experts_pairs(p, 224), (cudaStream_t)stream)
                                       : launch_experts<256, 1, false>(p, experts_pairs(p, 256), (cudaStream_t)stream);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "grouped product launch");
}
