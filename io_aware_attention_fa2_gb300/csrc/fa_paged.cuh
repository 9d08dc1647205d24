// fa_paged.cuh -- what the paged cache's kernels share: the device error word, reading a block
// table and lengths that were never checked on the host.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged_internal.h"
#include "ptx_sm103.cuh"

namespace fa {
namespace paged {

// Error word of this translation unit's kernels: bit 0 a wait ran past its limit, bit 1 a
// block-table entry or a length named a token outside the cache.
static __device__ int g_error = 0;

constexpr int kTimeoutBit = 1, kPageBit = 2;

__device__ __forceinline__ void record_page_error() { atomicOr(&g_error, kPageBit); }

static __global__ void clear_error_kernel(int bits) { atomicAnd(&g_error, ~bits); }

// Read and clear g_error of the translation unit that calls it; bits are or-ed into *bits. Only
// the bits that were read are cleared, on the device: kernels of other streams may be adding to
// the word (read and then written with a zero, it lost what they added in between).
static inline cudaError_t read_and_clear_error(int* bits) {
  int value = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&value, g_error, sizeof(int));
  if (err != cudaSuccess || value == 0) return err;
  *bits |= value;
  // (the launch's own status: cudaGetLastError may hold that of an earlier call)
  void* args[] = {&value};
  err = cudaLaunchKernel(reinterpret_cast<const void*>(clear_error_kernel), dim3(1), dim3(1), args,
                         0, nullptr);
  return err == cudaSuccess ? cudaStreamSynchronize(nullptr) : err;
}

// Tokens of sequence b that are visible to its newest one.
struct Visible {
  int lo, hi;
};
template <bool RECORD>
__device__ __forceinline__ Visible visible_tokens(const int* seqlens, int b, int capacity,
                                                  int window_left) {
  int len = seqlens[b];
  if (len > capacity || len < 0) {
    if (RECORD) record_page_error();
    len = min(max(len, 0), capacity);
  }
  return {window_left >= 0 ? max(0, len - 1 - window_left) : 0, len};
}

// Loads past L1 that stay where they stand in the program, behind a wait and in front of a
// barrier: the compiler's own intrinsic promises no order with either.
__device__ __forceinline__ int load_l2(const int* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_l2(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_l2(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Programmatic stream serialisation: let the next kernel be launched; wait for the one before.
// A kernel is resident while the one before it may still write its inputs, so none of them is
// read-only for the kernel's life: no input is declared `const T* __restrict__` and none is read
// through the non-coherent path, or the compiler could load it above the wait.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prerequisites() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launch with programmatic stream serialisation: the kernel may be set up while the one before it
// in the stream ends, and waits for it (wait_prerequisites) before it touches any memory that
// others see. Every kernel of the cache is launched so and lets its successor do the same: a
// chain of calls saves 4 to 5 us a decode (B=4 to 64K tokens 60.3 -> 55.9 us, B=16 to 16K 110.9 ->
// 106.3, with weights 131.9 -> 127.9) and 8 us an eviction (B=8 to 4096 73.8 -> 65.9).
// `cluster` CTAs to a cluster (0: no clusters).
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), int64_t grid, int block, size_t smem,
                           cudaStream_t stream, int cluster, const Args&... args) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// launch_chained, under the name by which the files of drafted and forked sequences call it (the
// rules that hold for the callers of either are tested by these names).
template <typename... Params, typename... Args>
cudaError_t launch_paged(void (*kernel)(Params...), int64_t grid, int block, size_t smem,
                         cudaStream_t stream, int cluster, const Args&... args) {
  return launch_chained(kernel, grid, block, smem, stream, cluster, args...);
}

// A kernel whose blocks, at most as many as run at once, wait for one another by the grid's barrier: a
// cooperative launch, which has all of them resident together or fails, and whose barrier is its own,
// so that calls on several streams and captured graphs do not meet. It starts when what is in front
// of it on the stream has ended.
template <typename... Params, typename... Args>
cudaError_t launch_together(void (*kernel)(Params...), int grid, int block, size_t smem,
                            cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr float kLn2 = 0.69314718055994530942f;

// 1 / sum of a row's probabilities: 0 for a row without any, NaN for a NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// k_pages or v_pages as a 5-D TMA map: 64 columns, head, row of the page, 64-column half, page.
// A box is box_rows rows of one page and head, `halves` 64-column halves of them one after the other.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline bool encode_pages(CUtensorMap* map, void* pages, const PagedCache& c, int box_rows,
                                int halves, bool fp16) {
  const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(encode_tiled_entry());
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.Hkv) * c.d * 2;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(c.Hkv),
                              static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.d / 64),
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(c.d) * 2, row, 128, row * c.page_size};
  const cuuint32_t box[5] = {64, 1, static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(halves), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            pages, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Drafted tokens of sequence b: they are its last ones, tokens [base, base + count). A sequence
// whose length is negative, beyond the table or shorter than its draft has count = -1.
struct Draft {
  int base, count;
};
__device__ __forceinline__ Draft draft_of(const int* seqlens, const int* new_lens, int b, int T,
                                          int capacity) {
  const int len = seqlens[b], n = new_lens ? min(max(new_lens[b], 0), T) : T;
  if (len < n || len > capacity) return {0, -1};
  return {len - n, n};
}

}  // namespace paged
}  // namespace fa
