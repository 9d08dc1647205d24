// fa_paged_internal.h -- declarations shared by the translation units of the paged key-value cache
// (fa_paged_api.cpp: argument checks and C ABI; fa_paged.cu, fa_paged_decode.cu,
// fa_key_weights.cu: kernels and launch) and, for the host-side helpers and the error words,
// fa_api.cpp. Not part of the public ABI.
#pragma once

#include <initializer_list>

#include "fa_internal.h"

namespace fa {

// ---- host-side helpers shared by the C ABI's translation units (fa_api.cpp)
// FA_OK when the current device is sm_103 (its number in *device).
int check_arch(int* device);
// FA_OK when every non-null pointer is device memory usable by `device`, else FA_ERR_POINTER.
int check_device_ptrs(int device, std::initializer_list<const void*> ptrs);
bool overlaps(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes);
// The driver's cuTensorMapEncodeTiled, or null.
void* encode_tiled_entry();
// [B, N, H, d] 16-bit tensor as a 4-D TMA map (d, H, N, B) with box (64, 1, 128, 1).
bool encode_bnhd(CUtensorMap* map, const void* base, int B, int H, int N, int d, bool fp16);

// ---- the paged key-value cache (include/fa.h has the layouts)
struct KeyWeightsParams {
  CUtensorMap tm_q, tm_k;   // [B, N, Hq, d] and [B, N, Hkv, d]
  const float* lse;         // [B, Hq, N]
  float* w;                 // [B, Hkv, N]
  float* part;              // workspace [B, Hq, N] when Hq > Hkv, else null
  int B, Hq, Hkv, N, d;
  int causal, window_left, window_right;   // windows clamped to N, or -1
  const int* seqlens_k;     // device int32 [B] or null
  int fp16;
  float scale_log2;
};
cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream);

struct PagedCache {
  void* k_pages;            // [num_pages, page_size, Hkv, d]
  void* v_pages;
  float* weights;           // [num_pages, Hkv, page_size] or null
  const int* block_table;   // device int32 [B, max_pages]
  const int* seqlens;       // device int32 [B]
  int B, Hkv, d, page_size, num_pages, max_pages;
};

struct AppendParams {
  PagedCache c;
  const void* k;            // [B, N, Hkv, d]
  const void* v;
  const float* w;           // [B, Hkv, N] or null
  const int* new_lens;      // device int32 [B] or null
  int N;
};
cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream);

struct DecodeParams {
  PagedCache c;
  const void* q;            // [B, Hq, d]
  void* o;
  float* lse;               // [B, Hq]
  void* workspace;
  int Hq, window_left, fp16;
  float scale_log2;
};
cudaError_t launch_paged_decode(const DecodeParams& p, cudaStream_t stream);
size_t paged_decode_workspace(int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                              bool with_weights);

struct EvictParams {
  PagedCache c;
  const int* out_table;     // device int32 [B, out_pages]
  int* kept;                // [B, Hkv, budget]
  int* new_seqlens;         // [B]
  int out_pages, budget, recent;
};
cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t stream);

// The error words of these kernels on the current device: read and clear (no synchronisation).
// FA_OK, FA_ERR_TIMEOUT, or FA_ERR_PAGE (where no wait ran out).
cudaError_t read_and_clear_paged_error(int* value);
// Those of two of the translation units, or-ed in: 1 timeout, 2 bad page.
cudaError_t read_and_clear_decode_error(int* bits);
cudaError_t read_and_clear_key_weights_error(int* bits);

}  // namespace fa
