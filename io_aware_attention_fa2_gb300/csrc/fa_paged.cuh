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

}  // namespace paged
}  // namespace fa
