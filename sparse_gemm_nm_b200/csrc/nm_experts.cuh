// nm_experts.cuh -- the columns of a product grouped by expert as tiles (internal).
//
// Columns [offsets[e], offsets[e + 1]) of the activations belong to expert e.  The counts are known on the device alone,
// so every CTA derives the same list of tiles from the offsets when it starts: expert e has row_tiles * nt tiles, nt column
// tiles of at most max_n columns.  TMA loads start on a 16-byte unit of the rows, and a box whose rows lie across two
// 128-byte lines costs L2 twice the requests (11008 x 4096, 8192 columns of eight experts: 437 us from multiples of 8,
// 357 us from multiples of 64), so an expert's first tile begins at its first column rounded down to a multiple of 64, or
// of 8 where it has no more than 64 columns (a wider tile would cost more than the lines).  The columns of its neighbours
// that a tile takes along are computed and not stored.
#pragma once
#include <cstdint>

#include "nm_experts.h"
#include "nm_ptx.cuh"

namespace nmk {

struct ExpertCols {
  int32_t c0, c1;  // the expert's columns
  int32_t a0;      // its first tile's first column
  int32_t nt;      // column tiles
};

// Where an expert's first tile starts: on a 16-byte unit, on a 128-byte line (above), or on a line unless a unit saves
// the second of two tiles (eight experts of 4096 x 4096, 250 columns each: 74 us, one tile from a unit 57)
enum Start { ON_UNITS, ON_LINES, FEWEST_TILES };

// Offsets are clamped to the matrix, whatever they hold.
template <Start START = ON_LINES>
__device__ __forceinline__ ExpertCols expert_cols(const int32_t* offsets, int e, int32_t S, int max_n) {
  ExpertCols x;
  x.c0 = min(max(__ldcg(offsets + e), 0), S);
  x.c1 = min(max(__ldcg(offsets + e + 1), x.c0), S);
  x.a0 = x.c0 & (START != ON_UNITS && x.c1 - x.c0 > 64 ? ~63 : ~7);
  x.nt = x.c1 > x.c0 ? (x.c1 - x.a0 + max_n - 1) / max_n : 0;
  if (START == FEWEST_TILES && x.nt == 2 && x.c1 - (x.c0 & ~7) <= max_n) {
    x.a0 = x.c0 & ~7;
    --x.nt;
  }
  return x;
}

// first[e] = number of the first tile of expert e, first[E] = number of tiles.  One warp; `first` is shared memory.
template <Start START = ON_LINES>
__device__ __forceinline__ void list_tiles(const int32_t* offsets, int E, int32_t S, int max_n, int row_tiles, int32_t* first,
                                           int lane) {
  int32_t base = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    int32_t n = e0 + lane < E ? expert_cols<START>(offsets, e0 + lane, S, max_n).nt * row_tiles : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) n += up;
    }
    if (e0 + lane < E) first[e0 + lane + 1] = base + n;
    base += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
  if (lane == 0) first[0] = 0;
}

// An expert's tiles in strips of column tiles, equally wide and `most` at most; in a strip column tiles go fastest, then row
// tiles.  The pairs running together then share a few row blocks of weights and a few column blocks: with all columns in
// one strip 32 column tiles met two row tiles, and L2 gave the columns (one expert 11008 x 4096, 8192 columns: 359 us,
// strips of 4, 8, 12 tiles 332, 326, 322; two of 4096 x 11008 with 8192 each 759 -> 674; input gradient in strips of 4
// tiles of 512 columns 522 -> 501 and 1047 -> 998; experts of one strip as before).  A strip's weights come back from L2.
__host__ __device__ __forceinline__ int strip_width(int nt, int most) {  // nt > 0
  if (nt <= most) return nt;
  const int strips = (nt + most - 1) / most;
  return (nt + strips - 1) / strips;
}
__device__ __forceinline__ void tile_in_strip(int in, int row_tiles, int nt, int wide, int& tm, int& tn) {
  int first = 0, across = nt;
  if (wide < nt) {
    const int strip = in / (row_tiles * wide);
    in -= strip * row_tiles * wide;
    first = strip * wide;
    across = min(nt - first, wide);
  }
  tm = in / across;
  tn = first + in - tm * across;
}

// What a pair works on: tiles pair, pair + pairs, ... whole, or (STREAM) an equal share of all tiles' stages, in one piece: a
// share may start and end inside a tile, whose other stages the neighbouring pairs have.
constexpr int kLeastStages = 4;  // of a share
struct Shares {
  int64_t total;  // stages of all tiles
  int parts;      // shares
  __device__ __forceinline__ Shares(int64_t tiles, int k_tiles, int pairs) {
    total = tiles * k_tiles;
    const int64_t most = total / kLeastStages;
    parts = most < pairs ? (most < 1 ? 1 : (int)most) : pairs;
  }
  __device__ __forceinline__ int64_t start(int part) const { return total * part / parts; }
  // The share that has stage `at`.
  __device__ __forceinline__ int of(int64_t at) const {
    int part = (int)(at * parts / total);
    while (part + 1 < parts && start(part + 1) <= at) ++part;
    return part;
  }
};

template <bool STREAM, Start START = ON_LINES>
struct TileWalk {
  int e, tm;       // expert, row tile
  int32_t x0, n;   // first column, columns (a multiple of 32)
  int32_t c0, c1;  // the expert's columns
  int k0, k1;      // stages
  int slot;        // of partial sums, for a part of a tile: 0 for the pair's first, 1 for its last
  int64_t at, end;  // tile number, or (STREAM) stage number
  const int32_t *first, *offsets;
  int32_t S;
  int E, max_n, k_tiles, step, row_tiles, wide;
  ExpertCols cols;
  int known;

  __device__ __forceinline__ TileWalk(const int32_t* first_, const int32_t* offsets_, int E_, int32_t S_, int max_n_,
                                      int k_tiles_, int row_tiles_, int pair, int pairs)
      : e(0), slot(-1), first(first_), offsets(offsets_), S(S_), E(E_), max_n(max_n_), k_tiles(k_tiles_), step(pairs),
        row_tiles(row_tiles_), known(-1) {
    if (STREAM) {
      const Shares sh(first[E], k_tiles, pairs);
      at = pair < sh.parts ? sh.start(pair) : 0;
      end = pair < sh.parts ? sh.start(pair + 1) : 0;
    } else {
      at = pair - pairs;
      end = first[E];
    }
  }
  // The next tile, or part of one; false behind the last.
  __device__ __forceinline__ bool next() {
    int id;
    if (STREAM) {
      if (slot >= 0) at += k1 - k0;
      if (at >= end) return false;
      id = (int)(at / k_tiles);
      k0 = (int)(at - (int64_t)id * k_tiles);
      k1 = end - at < k_tiles - k0 ? k0 + (int)(end - at) : k_tiles;
      slot = slot < 0 ? 0 : 1;
    } else {
      at += step;
      if (at >= end) return false;
      id = (int)at;
      k0 = 0;
      k1 = k_tiles;
    }
    tile(id);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return !STREAM || (k0 == 0 && k1 == k_tiles); }
  // Sets the members for tile `id` (at least the last one).
  __device__ __forceinline__ void tile(int id) {
    while (id >= first[e + 1]) ++e;
    if (e != known) {
      cols = expert_cols<START>(offsets, e, S, max_n);
      known = e;
      wide = strip_width(cols.nt, 12);
    }
    int tn;
    tile_in_strip(id - first[e], row_tiles, cols.nt, wide, tm, tn);
    c0 = cols.c0;
    c1 = cols.c1;
    x0 = cols.a0 + tn * max_n;
    n = min((cols.c1 - x0 + 31) & ~31, max_n);
  }
};

// Tiles of up to WIDE columns, the whole ones of all experts first and the experts' last, narrower ones behind them: tiles
// are few then, and what is left for the pairs that come through early is small.  first has 2 E + 1 numbers.
template <int WIDE>
__device__ __forceinline__ int32_t wide_tiles(const int32_t* offsets, int v, int E, int32_t S, int row_tiles) {
  const ExpertCols x = expert_cols(offsets, v < E ? v : v - E, S, WIDE);
  const int32_t w = x.c1 > x.c0 ? x.c1 - x.a0 : 0;
  return (v < E ? w / WIDE : (w % WIDE != 0)) * row_tiles;
}
template <int WIDE>
__device__ __forceinline__ void list_wide_tiles(const int32_t* offsets, int E, int32_t S, int row_tiles, int32_t* first,
                                                int lane) {
  int32_t base = 0;
  for (int v0 = 0; v0 < 2 * E; v0 += 32) {
    int32_t n = v0 + lane < 2 * E ? wide_tiles<WIDE>(offsets, v0 + lane, E, S, row_tiles) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) n += up;
    }
    if (v0 + lane < 2 * E) first[v0 + lane + 1] = base + n;
    base += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
  if (lane == 0) first[0] = 0;
}

template <int WIDE>
struct WideWalk {
  int e, tm;       // expert, row tile
  int32_t x0, n;   // first column, columns (a multiple of 32)
  int32_t c0, c1;  // the expert's columns
  int k0, k1;      // stages
  const int32_t *first, *offsets;
  int32_t S;
  int E, v, id, step, row_tiles, known;
  ExpertCols cols;

  __device__ __forceinline__ WideWalk(const int32_t* first_, const int32_t* offsets_, int E_, int32_t S_, int k_tiles,
                                      int row_tiles_, int pair, int pairs)
      : k0(0), k1(k_tiles), first(first_), offsets(offsets_), S(S_), E(E_), v(0), id(pair - pairs), step(pairs),
        row_tiles(row_tiles_), known(-1) {}
  __device__ __forceinline__ bool next() {
    id += step;
    if (id >= first[2 * E]) return false;
    while (id >= first[v + 1]) ++v;
    e = v < E ? v : v - E;
    if (e != known) {
      cols = expert_cols(offsets, e, S, WIDE);
      known = e;
    }
    const int in = id - first[v], whole = (cols.c1 - cols.a0) / WIDE;
    c0 = cols.c0;
    c1 = cols.c1;
    if (v < E) {
      int tn;
      tile_in_strip(in, row_tiles, whole, strip_width(whole, 4), tm, tn);
      x0 = cols.a0 + tn * WIDE;
      n = WIDE;
    } else {
      tm = in;
      x0 = cols.a0 + whole * WIDE;
      n = (cols.c1 - x0 + 31) & ~31;
    }
    return true;
  }
};

// ------------------------------------------------------------------ stores
constexpr uint32_t kBoxBytes = 4096;  // an epilogue warp's staging tile: 32 rows x 128 bytes, 128-byte swizzle

// Elements [from, to) of a 16-byte unit, one by one.
template <typename T>
__device__ __forceinline__ void store_unit_part(const uint4& u, T* dst, int from, int to) {
  constexpr int kPer = 16 / (int)sizeof(T);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i >= from && i < to) dst[i] = sizeof(T) == 2 ? (T)(w[i >> 1] >> (16 * (i & 1))) : (T)w[i & 3];
}

// A warp's staged box (32 rows of 128 bytes, swizzled), columns x .. of rows wrow0 ..: whole by TMA, or its part inside
// [c0, c1) by the lanes.
template <typename T>
__device__ __forceinline__ void store_box(const ExpertsParams& p, const uint8_t* box, int32_t x, int32_t c0, int32_t c1,
                                          int32_t wrow0, int lane) {
  constexpr int kPer = 16 / (int)sizeof(T), kCols = 8 * kPer;
  if (wrow0 >= p.M || x >= c1 || x + kCols <= c0) return;
  if (x >= c0 && x + kCols <= c1) {
    if (lane == 0) {
      tma_store_2d(&p.tm_y, box, x, wrow0);
      bulk_commit_group();
    }
    return;
  }
  const int unit = lane & 7;
  const int32_t u0 = x + unit * kPer;
  const int from = max(c0 - u0, 0), to = min(c1 - u0, kPer);
  if (from >= to) return;
  T* col = static_cast<T*>(p.Y) + u0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    if (wrow0 + r >= p.M) break;
    const uint4 u = *reinterpret_cast<const uint4*>(box + r * 128 + ((unit ^ (r & 7)) << 4));
    T* dst = col + (int64_t)(wrow0 + r) * p.ldy;
    if (from == 0 && to == kPer)
      *reinterpret_cast<uint4*>(dst) = u;
    else
      store_unit_part<T>(u, dst, from, to);
  }
}

// 32 accumulator columns of the warp's 32 rows as bf16 pairs.
__device__ __forceinline__ void take_bf16(uint32_t t_addr, uint32_t* out) {
  uint32_t v[32];
  tmem_ld_32x32b_x32(t_addr, v);
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) out[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// One chunk (128 bytes of each of the warp's 32 rows, a row a lane) through the warp's staging tile.
template <typename T>
__device__ __forceinline__ void store_chunk(const ExpertsParams& p, const uint32_t (&v)[32], uint8_t* box, int32_t x,
                                            int32_t c0, int32_t c1, int32_t wrow0, int lane) {
  if (lane == 0) bulk_wait_group_read<0>();  // the previous store has read it
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  store_box<T>(p, box, x, c0, c1, wrow0, lane);
}

// The warp's 32 rows of a tile, chunk by chunk; `release` is called after the last TMEM load.  Accumulator columns behind
// the tile's hold what an earlier tile left there: they lie behind `end`.
template <typename Release>
__device__ __forceinline__ void store_tile(const ExpertsParams& p, int32_t x0, int32_t n, int32_t c0, int32_t c1,
                                           uint32_t t_addr, uint8_t* box, int32_t wrow0, int lane, Release release) {
  const int32_t end = min(c1, x0 + n);
  const int step = p.out_f32 ? 32 : 64;
#pragma unroll 1
  for (int c = 0; c < n; c += step) {
    uint32_t v[32];
    if (p.out_f32) {
      tmem_ld_32x32b_x32(t_addr + c, v);
      tc_wait_ld();
    } else {
      take_bf16(t_addr + c, v);
      take_bf16(t_addr + c + 32, v + 16);
    }
    if (c + step >= n) release();
    if (p.out_f32)
      store_chunk<uint32_t>(p, v, box, x0 + c, c0, end, wrow0, lane);
    else
      store_chunk<uint16_t>(p, v, box, x0 + c, c0, end, wrow0, lane);
  }
}

// A pair that starts a tile and does not finish it notes it for the join (one thread of the pair; false: not this one).
__device__ __forceinline__ bool note_cut(const ExpertsParams& p, const TileWalk<true, ON_UNITS>& w, int pair, int pairs) {
  if (w.k0 != 0 || w.k1 == w.k_tiles) return false;
  const Shares sh(w.first[w.E], w.k_tiles, pairs);
  const int last = sh.of(w.at + w.k_tiles - 1);
  p.cuts[pair] = ExpertsCut{last - pair + 1, w.slot, w.tm * 256, w.x0, w.n, w.c0, min(w.c1, w.x0 + w.n), 0};
  return true;
}

// Partial sums: the warp's 32 rows (row `row` of the tile on) into the slot's rows of w.n fp32.
template <typename Walk, typename Release>
__device__ __forceinline__ void store_part(float* slot, const Walk& w, uint32_t t_addr, int row, int lane,
                                           Release release) {
  float4* to = reinterpret_cast<float4*>(slot + (int64_t)(row + lane) * w.n);
#pragma unroll 1
  for (int c = 0; c < w.n; c += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(t_addr + c, v);
    tc_wait_ld();
    if (c + 32 >= w.n) release();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      to[c / 4 + q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                  __uint_as_float(v[4 * q + 3]));
  }
}

}  // namespace nmk
