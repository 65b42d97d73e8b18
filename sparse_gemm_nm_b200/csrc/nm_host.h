// nm_host.h -- host helpers of the C entry points that live in several files
// (internal): error reporting, the staging pool, tensor maps, argument checks
// and the GEMM routines that other entry points build on.  Defined in nm_api.cu.
#pragma once
#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/nm.h"
#include "nm_internal.h"
#include "nm_spmm.h"

namespace nmk {

// Records the text of nm_last_error() and returns the status.
nm_status fail(nm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
nm_status cuda_fail(cudaError_t e, const char* what);
void set_last_error(const char* msg);
nm_status require_device();
cudaError_t staging_pool(cudaMemPool_t* out);
nm_status make_tmap(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
                    uint32_t box_inner, uint32_t box_outer, int swizzle_bytes, const char* what,
                    CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);

// 3-D map of {d0, d1, d2} bf16 with strides s1 and s2 bytes, boxes {b0, b1, 1}.
nm_status make_tmap3(CUtensorMap* tm, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2,
                     uint32_t b0, uint32_t b1, int swizzle_bytes, const char* what);
// 3-D map of the tiled 2:4 metadata (boxes of box_rblocks row blocks of one column block).
nm_status make_meta_tmap(CUtensorMap* tm, const void* meta, int64_t rblocks, int64_t cblocks, uint32_t box_rblocks = 8);

class Staged;

// Further dense reduction steps of a GEMM: blocks of 64 rows of `terms` (planes x cat rows x T, row stride ldp) against
// the same 64 columns of `left` (forward: R x cat, K-major) or rows (input gradient: cat x K); a column tile takes the
// blocks in the masks of its 64-token tiles.  left: rows x cols, row stride ldl.
struct GemmExt {
  const uint16_t* left;
  int64_t rows, cols, ldl;
  const uint16_t* terms;
  int64_t cat, ldp;
  int planes;
  const uint32_t* masks;
};

// Where a split-K GEMM may leave its fp32 partial sums instead of adding them up: `splits` matrices (1: the result
// is in Y as usual), `split_stride` elements apart, rows of `ld`.
struct GemmPartials {
  Staged* ws;
  bool beside;  // the call's launches before this GEMM began with pdl_gate(): its first may run beside the last of them
  int splits;
  int64_t split_stride, ld;
};

// nm_spmm / nm_spmm_permuted (idx may be null): the argument checks alone, and the call.
nm_status check_spmm(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                     const uint16_t* X, int64_t ldx, int64_t T, void* Y, int64_t ldy, nm_out_dtype y_dtype);
nm_status run_spmm(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                   const int32_t* idx, const uint16_t* X, int64_t ldx, int64_t T, void* Y, int64_t ldy,
                   nm_out_dtype y_dtype, GemmPartials* partials, cudaStream_t stream, const GemmExt* ext = nullptr);
// nm_spmm_t: the argument checks alone, and the call.
nm_status check_spmm_t(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                       const uint16_t* dY, int64_t lddy, int64_t T, void* dX, int64_t lddx, nm_out_dtype dtype);
nm_status run_spmm_t(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                     const int32_t* idx, const uint16_t* dY, int64_t lddy, int64_t T, void* dX, int64_t lddx,
                     nm_out_dtype dtype, cudaStream_t stream, const GemmExt* ext = nullptr);
// Y = W' X (nm_spmm).
nm_status spmm_rows(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                    const uint16_t* X, int64_t ldx, int64_t T, void* Y, int64_t ldy, nm_out_dtype y_dtype,
                    cudaStream_t stream);
// Does the SM-pair 2:4 kernel serve the shape (directly, or after re-encoding)?  Only then run_spmm_epilogue: the
// product with one of that kernel's epilogues (Y null where the epilogue stores none).
bool spmm_pair_serves(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t K, int64_t T);
nm_status run_spmm_epilogue(const uint16_t* values, const uint32_t* meta, int n, int m, int64_t R, int64_t K,
                            const uint16_t* X, int64_t ldx, int64_t T, void* Y, int64_t ldy, const PairEpiData& epi,
                            cudaStream_t stream);
// nm_sddmm.
nm_status run_sddmm(const uint32_t* meta, int n, int m, int64_t R, int64_t K, const int32_t* idx, const uint16_t* dY,
                    int64_t lddy, const uint16_t* X, int64_t ldx, int64_t T, void* dV, nm_out_dtype dtype,
                    cudaStream_t stream, bool beside = false, int64_t x_tokens = 0);
// beside: as GemmPartials' (without idx).  x_tokens below T: X has that many columns, and dY is two terms of T / 2 columns
// (a multiple of 64), each of which meets X (zeros past x_tokens).
// C (K x T fp32, row stride ldc) = or += W^T D for a dense R x K bf16 W (row stride ldw) and an R x T bf16 D, by
// the SM-pair GEMM; every element takes one addition.
// dense_product: C (R x T fp32, row stride ldc) = W X, X K x T.
nm_status dense_product(const uint16_t* W, int64_t ldw, int64_t R, int64_t K, const uint16_t* X, int64_t ldx, int64_t T,
                        float* C, int64_t ldc, cudaStream_t stream);
// With ranges > 1 the rows of W and D are taken in that many ranges side by side, range i's sum in C + i K ldc.
int dense_t_ranges(int64_t R, int64_t K, int64_t T);  // that fill the SMs
nm_status dense_t_accumulate(const uint16_t* W, int64_t ldw, int64_t R, int64_t K, const uint16_t* D, int64_t ldd,
                             int64_t T, float* C, int64_t ldc, int ranges, bool add, cudaStream_t stream);

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dtype_ok(int d) { return d == NM_OUT_BF16 || d == NM_OUT_F32; }
inline int64_t dtype_bytes(int d) { return d == NM_OUT_F32 ? 4 : 2; }
constexpr int64_t kMaxDim = 1ll << 31;

// A strided matrix of rows x T elements: pointer set, row stride at least T, rows on 16 bytes.
inline nm_status check_matrix(const void* p, int64_t ld, int64_t T, int64_t esize, const char* name) {
  if (!p) return fail(NM_ERR_INVALID_ARG, "%s is null", name);
  if (ld < T) return fail(NM_ERR_INVALID_ARG, "ld of %s < T", name);
  if (!al16(p) || (ld * esize) % 16 != 0) return fail(NM_ERR_MISALIGNED, "%s rows must be 16-byte aligned", name);
  return NM_OK;
}

// 32-bit vectors and words, each on 4 bytes (null where the argument is optional).
inline nm_status check_words(std::initializer_list<const void*> ps, const char* names) {
  for (const void* p : ps)
    if (!aligned_to(p, 4)) return fail(NM_ERR_MISALIGNED, "%s must be 4-byte aligned", names);
  return NM_OK;
}

// Parts of one staging buffer, each on 256 bytes: take() returns a part's offset.
class Parts {
 public:
  int64_t take(int64_t bytes) {
    const int64_t at = size_;
    size_ += (bytes + 255) / 256 * 256;
    return at;
  }
  size_t size() const { return (size_t)size_; }

 private:
  int64_t size_ = 0;
};

// A staging buffer from the library's pool, handed back on its stream when it goes out of scope.
class Staged {
 public:
  explicit Staged(cudaStream_t s) : stream_(s) {}
  ~Staged() { release(); }
  Staged(const Staged&) = delete;
  Staged& operator=(const Staged&) = delete;
  cudaError_t get(size_t bytes) {
    cudaMemPool_t pool = nullptr;
    cudaError_t e = staging_pool(&pool);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&p_, bytes, pool, stream_);
    if (e != cudaSuccess) p_ = nullptr;
    return e;
  }
  void release() {
    if (p_) cudaFreeAsync(p_, stream_);
    p_ = nullptr;
  }
  template <typename T>
  T* as(int64_t offset_bytes = 0) const {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(p_) + offset_bytes);
  }

 private:
  cudaStream_t stream_;
  void* p_ = nullptr;
};

// Raises a kernel's shared-memory limit once per device (always to the same value, its largest request).
struct SmemLimit {
  std::atomic<bool> done[64];  // static storage: false
  template <typename Kern>
  cudaError_t raise(Kern kernel, uint32_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
    return e;
  }
};

}  // namespace nmk
