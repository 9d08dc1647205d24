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

// Read and clear g_error of the translation unit that calls it; bits are or-ed into *bits.
static inline cudaError_t read_and_clear_error(int* bits) {
  int value = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&value, g_error, sizeof(int));
  if (err != cudaSuccess) return err;
  *bits |= value;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
}

// Tokens of sequence b that are visible to its newest one.
struct Visible {
  int lo, hi;
};
template <bool RECORD>
__device__ __forceinline__ Visible visible_tokens(const int* __restrict__ seqlens, int b,
                                                  int capacity, int window_left) {
  int len = seqlens[b];
  if (len > capacity || len < 0) {
    if (RECORD) record_page_error();
    len = min(max(len, 0), capacity);
  }
  return {window_left >= 0 ? max(0, len - 1 - window_left) : 0, len};
}

// Programmatic stream serialisation: let the next kernel be launched; wait for the one before.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prerequisites() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace paged
}  // namespace fa
