// fa_paged_api.cpp -- the C ABI of the paged key-value cache (include/fa.h): argument checks and
// launch. Host-detected errors return before anything is enqueued, in the order of the other
// entry points: pointers, shape, dtype, scale, workspace, alignment, aliasing, device.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "fa.h"
#include "fa_paged_internal.h"

namespace {

struct Span {
  const void* p;
  uint64_t n;
};

// No output may overlap an input or another output (null spans are absent arguments).
int check_spans(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    if (!a->p || !a->n) continue;
    for (const Span& b : ins)
      if (b.p && b.n && fa::overlaps(a->p, a->n, b.p, b.n)) return FA_ERR_ALIAS;
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (b->p && b->n && fa::overlaps(a->p, a->n, b->p, b->n)) return FA_ERR_ALIAS;
  }
  return FA_OK;
}

bool aligned(std::initializer_list<const void*> ptrs, uintptr_t to) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % to) return false;
  return true;
}

int check_device(std::initializer_list<const void*> ptrs) {
  int device = 0;
  const int rc = fa::check_arch(&device);
  return rc != FA_OK ? rc : fa::check_device_ptrs(device, ptrs);
}

// Shape of a cache. Lengths are int32 with room for the tiles behind the last one (at most 2^30
// tokens a sequence), and the pool's bytes and the kernels' grids stay far inside 64 and 31 bits.
bool cache_shape_ok(int B, int Hkv, int d, int page_size, int num_pages, int max_pages) {
  if (B < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1) return false;
  if (d != 64 && d != 128) return false;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return false;
  if ((int64_t)max_pages * page_size > (1ll << 30)) return false;
  // a page within 2^31 bytes, the pool within 2^62
  const uint64_t page_bytes = (uint64_t)page_size * (uint64_t)Hkv * (uint64_t)d * 2;
  if (page_bytes >= (1ull << 31)) return false;
  return (uint64_t)B * (uint64_t)Hkv < (1ull << 31);
}

// The kernels work in log2 units: scale * log2(e) has to be finite, too.
constexpr float kLog2e = 1.4426950408889634f;
bool scale_ok(float scale) { return isfinite(scale) && isfinite(scale * kLog2e); }

// Query heads over a cache's key heads, for a decode: the grids (a block for each (b, h), and one
// for each 1024 tokens of a (b, key head)) stay within 2^31 - 1.
bool decode_shape_ok(int B, int Hq, int Hkv, int page_size, int max_pages) {
  if (Hq < Hkv || Hq % Hkv) return false;
  const uint64_t tokens = (uint64_t)max_pages * page_size;
  return (uint64_t)B * (uint64_t)Hq * (tokens / 1024 + 2) < (1ull << 31);
}

uint64_t pool_bytes(int Hkv, int d, int page_size, int num_pages) {
  return (uint64_t)num_pages * page_size * Hkv * d * 2;
}

fa::PagedCache make_cache(const void* k_pages, const void* v_pages, float* weights,
                          const int* block_table, const int* seqlens, int B, int Hkv, int d,
                          int page_size, int num_pages, int max_pages) {
  fa::PagedCache c;
  c.k_pages = const_cast<void*>(k_pages);
  c.v_pages = const_cast<void*>(v_pages);
  c.weights = weights;
  c.block_table = block_table;
  c.seqlens = seqlens;
  c.B = B;
  c.Hkv = Hkv;
  c.d = d;
  c.page_size = page_size;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  return c;
}

}  // namespace

extern "C" {

size_t fa_key_weights_workspace_size(int B, int Hq, int Hkv, int N) {
  if (B < 1 || Hkv < 1 || Hq <= Hkv || N < 1) return 0;
  return (size_t)((uint64_t)B * Hq * N * 4);
}

int fa_key_weights(const void* q, const void* k, const float* lse, float* w, int B, int Hq,
                   int Hkv, int N, int d, int causal, int window_left, int window_right,
                   const int* seqlens_k, float scale, int dtype, void* workspace,
                   size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k || !lse || !w) return FA_ERR_NULL;
  if (B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || N < 1 || (d != 64 && d != 128))
    return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!scale_ok(scale)) return FA_ERR_SCALE;
  const uint64_t bh = (uint64_t)B * (uint64_t)Hq;
  // one CTA per (b, query head, 256 keys), at most 2^31 - 1; a key of the last CTA (at most N + 254)
  // plus a window bound (at most N) plus 1 stays an int
  if (bh >= (1ull << 31) || bh * (((uint64_t)N + 127) / 128) >= (1ull << 31) ||
      N > (1 << 30) - 128 || bh * (uint64_t)N > (1ull << 62) / 256)
    return FA_ERR_SHAPE;
  const uint64_t ws_need = fa_key_weights_workspace_size(B, Hq, Hkv, N);
  if (ws_need) {
    if (!workspace) return FA_ERR_NULL;
    if (workspace_bytes < ws_need) return FA_ERR_WORKSPACE;
  } else {
    workspace = nullptr;
  }
  if (!aligned({q, k, workspace}, 16) || !aligned({lse, w, seqlens_k}, 4)) return FA_ERR_ALIGN;
  const uint64_t row = (uint64_t)B * N;
  int rc = check_spans({{q, row * Hq * d * 2}, {k, row * Hkv * d * 2}, {lse, row * Hq * 4},
                        {seqlens_k, (uint64_t)B * 4}},
                       {{w, row * Hkv * 4}, {workspace, ws_need}});
  if (rc != FA_OK) return rc;
  rc = check_device({q, k, lse, w, seqlens_k, workspace});
  if (rc != FA_OK) return rc;

  fa::KeyWeightsParams p;
  const bool fp16 = dtype == FA_FP16;
  if (!fa::encode_bnhd(&p.tm_q, q, B, Hq, N, d, fp16) ||
      !fa::encode_bnhd(&p.tm_k, k, B, Hkv, N, d, fp16))
    return FA_ERR_CUDA;
  p.lse = lse;
  p.w = w;
  p.part = static_cast<float*>(workspace);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.causal = causal ? 1 : 0;
  // a bound wider than the sequence is no narrower than none, and keeps index sums within int
  p.window_left = window_left < 0 ? -1 : std::min(window_left, N);
  p.window_right = window_right < 0 ? -1 : std::min(window_right, N);
  p.seqlens_k = seqlens_k;
  p.fp16 = fp16 ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  return fa::launch_key_weights(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

int fa_paged_append(const void* k, const void* v, const float* w, void* k_pages, void* v_pages,
                    float* weights, const int* block_table, const int* seqlens,
                    const int* new_lens, int B, int N, int Hkv, int d, int page_size,
                    int num_pages, int max_pages, int dtype, fa_stream_t stream) {
  if (!k || !v || !k_pages || !v_pages || !block_table || !seqlens) return FA_ERR_NULL;
  if (w && !weights) return FA_ERR_NULL;
  if (N < 1 || !cache_shape_ok(B, Hkv, d, page_size, num_pages, max_pages)) return FA_ERR_SHAPE;
  if ((uint64_t)B * (uint64_t)N >= (1ull << 31)) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!aligned({k, v, k_pages, v_pages, weights}, 16) ||
      !aligned({w, block_table, seqlens, new_lens}, 4))
    return FA_ERR_ALIGN;
  const uint64_t pool = pool_bytes(Hkv, d, page_size, num_pages);
  const uint64_t in = (uint64_t)B * N * Hkv * d * 2, lens = (uint64_t)B * 4;
  int rc = check_spans({{k, in}, {v, in}, {w, (uint64_t)B * N * Hkv * 4},
                        {block_table, lens * max_pages}, {seqlens, lens}, {new_lens, lens}},
                       {{k_pages, pool}, {v_pages, pool}, {weights, pool / d * 2}});
  if (rc != FA_OK) return rc;
  rc = check_device({k, v, w, k_pages, v_pages, weights, block_table, seqlens, new_lens});
  if (rc != FA_OK) return rc;

  fa::AppendParams p;
  p.c = make_cache(k_pages, v_pages, weights, block_table, seqlens, B, Hkv, d, page_size,
                   num_pages, max_pages);
  p.k = k;
  p.v = v;
  p.w = w;
  p.new_lens = new_lens;
  p.N = N;
  return fa::launch_paged_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_paged_decode_workspace_size(int B, int Hq, int Hkv, int d, int page_size,
                                      int max_pages, int with_weights) {
  if (!cache_shape_ok(B, Hkv, d, page_size, 1, max_pages) ||
      !decode_shape_ok(B, Hq, Hkv, page_size, max_pages))
    return 0;
  return fa::paged_decode_workspace(B, Hq, Hkv, d, page_size, max_pages, with_weights != 0);
}

int fa_paged_decode(const void* q, const void* k_pages, const void* v_pages, float* weights,
                    const int* block_table, const int* seqlens, void* o, float* lse, int B,
                    int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                    int window_left, float scale, int dtype, void* workspace,
                    size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k_pages || !v_pages || !block_table || !seqlens || !o || !lse) return FA_ERR_NULL;
  if (!cache_shape_ok(B, Hkv, d, page_size, num_pages, max_pages) ||
      !decode_shape_ok(B, Hq, Hkv, page_size, max_pages))
    return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!scale_ok(scale)) return FA_ERR_SCALE;
  const uint64_t ws_need =
      fa::paged_decode_workspace(B, Hq, Hkv, d, page_size, max_pages, weights != nullptr);
  if (ws_need) {
    if (!workspace) return FA_ERR_NULL;
    if (workspace_bytes < ws_need) return FA_ERR_WORKSPACE;
  } else {
    workspace = nullptr;
  }
  if (!aligned({q, k_pages, v_pages, o, weights, workspace}, 16) ||
      !aligned({block_table, seqlens, lse}, 4))
    return FA_ERR_ALIGN;
  const uint64_t pool = pool_bytes(Hkv, d, page_size, num_pages);
  const uint64_t rows = (uint64_t)B * Hq, lens = (uint64_t)B * 4;
  int rc = check_spans({{q, rows * d * 2}, {k_pages, pool}, {v_pages, pool},
                        {block_table, lens * max_pages}, {seqlens, lens}},
                       {{o, rows * d * 2}, {lse, rows * 4}, {weights, pool / d * 2},
                        {workspace, ws_need}});
  if (rc != FA_OK) return rc;
  rc = check_device({q, k_pages, v_pages, weights, block_table, seqlens, o, lse, workspace});
  if (rc != FA_OK) return rc;

  fa::DecodeParams p;
  p.c = make_cache(k_pages, v_pages, weights, block_table, seqlens, B, Hkv, d, page_size,
                   num_pages, max_pages);
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.workspace = workspace;
  p.Hq = Hq;
  p.window_left = window_left < 0 ? -1 : window_left;
  p.fp16 = dtype == FA_FP16 ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  return fa::launch_paged_decode(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

int fa_paged_evict(void* k_pages, void* v_pages, float* weights, const int* block_table,
                   const int* seqlens, const int* out_table, int* kept, int* new_seqlens, int B,
                   int Hkv, int d, int page_size, int num_pages, int max_pages, int out_pages,
                   int budget, int recent, int dtype, fa_stream_t stream) {
  if (!k_pages || !v_pages || !weights || !block_table || !seqlens || !out_table || !kept ||
      !new_seqlens)
    return FA_ERR_NULL;
  if (!cache_shape_ok(B, Hkv, d, page_size, num_pages, max_pages)) return FA_ERR_SHAPE;
  if (out_pages < 1 || budget < 1 || recent < 0 || recent > budget ||
      (int64_t)out_pages * page_size < budget ||
      (int64_t)out_pages * page_size > (1ll << 30) ||
      (uint64_t)B * (uint64_t)Hkv >= (1ull << 28))   // eight CTAs for each
    return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!aligned({k_pages, v_pages, weights}, 16) ||
      !aligned({block_table, seqlens, out_table, kept, new_seqlens}, 4))
    return FA_ERR_ALIGN;
  const uint64_t pool = pool_bytes(Hkv, d, page_size, num_pages), lens = (uint64_t)B * 4;
  int rc = check_spans({{block_table, lens * max_pages}, {seqlens, lens},
                        {out_table, lens * out_pages}},
                       {{k_pages, pool}, {v_pages, pool}, {weights, pool / d * 2},
                        {kept, lens * Hkv * budget}, {new_seqlens, lens}});
  if (rc != FA_OK) return rc;
  rc = check_device({k_pages, v_pages, weights, block_table, seqlens, out_table, kept,
                     new_seqlens});
  if (rc != FA_OK) return rc;

  fa::EvictParams p;
  p.c = make_cache(k_pages, v_pages, weights, block_table, seqlens, B, Hkv, d, page_size,
                   num_pages, max_pages);
  p.out_table = out_table;
  p.kept = kept;
  p.new_seqlens = new_seqlens;
  p.out_pages = out_pages;
  p.budget = budget;
  p.recent = recent;
  return fa::launch_paged_evict(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
