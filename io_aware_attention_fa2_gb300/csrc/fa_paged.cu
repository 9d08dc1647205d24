// fa_paged.cu -- the paged key-value cache: append, decode, evict (include/fa.h has the layouts
// and the rules for bad block-table entries and lengths).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "ptx_sm103.cuh"

namespace fa {

// Device error word of the paged kernels: bit 0 a wait ran past its limit, bit 1 a block-table
// entry or a length named a token outside the cache.
__device__ int g_paged_error = 0;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kPageError = 2;
constexpr int kErrTimeout = -8, kErrPage = -13;   // FA_ERR_TIMEOUT, FA_ERR_PAGE

__device__ __forceinline__ void record_page_error() { atomicOr(&g_paged_error, kPageError); }

template <bool FP16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if constexpr (FP16) {
    return __half2float(__ushort_as_half(x));
  } else {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
}

template <bool FP16>
__device__ __forceinline__ uint16_t from_float(float x) {
  if constexpr (FP16) {
    return __half_as_ushort(__float2half_rn(x));
  } else {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  }
}

// Page of the table entry at `at`, or -1 (recorded) when it is outside the pool.
__device__ __forceinline__ int page_at(const int* __restrict__ table, int64_t at, int num_pages) {
  const int page = table[at];
  if (page >= 0 && page < num_pages) return page;
  record_page_error();
  return -1;
}

// ---------------------------------------------------------------------------------------------
// Append. One block per new token: its Hkv * d values are contiguous in both layouts.
__global__ void __launch_bounds__(128)
    fa_paged_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                           const float* __restrict__ w, uint4* __restrict__ k_pages,
                           uint4* __restrict__ v_pages, float* __restrict__ weights,
                           const int* __restrict__ table, const int* __restrict__ seqlens,
                           const int* __restrict__ new_lens, int N, int Hkv, int d, int page_size,
                           int num_pages, int max_pages) {
  const int b = blockIdx.x / N, i = blockIdx.x % N;
  const int n = new_lens ? min(max(new_lens[b], 0), N) : N;
  if (i >= n) return;
  const int64_t t = static_cast<int64_t>(seqlens[b]) - n + i;
  if (t < 0 || t >= static_cast<int64_t>(max_pages) * page_size) {
    record_page_error();
    return;
  }
  const int page =
      page_at(table, static_cast<int64_t>(b) * max_pages + t / page_size, num_pages);
  if (page < 0) return;
  const int row = static_cast<int>(t % page_size);
  const int chunks = Hkv * d / 8;
  const int64_t src = static_cast<int64_t>(blockIdx.x) * chunks;
  const int64_t dst = (static_cast<int64_t>(page) * page_size + row) * chunks;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    k_pages[dst + c] = k[src + c];
    v_pages[dst + c] = v[src + c];
  }
  if (weights)
    for (int h = threadIdx.x; h < Hkv; h += blockDim.x)
      weights[(static_cast<int64_t>(page) * Hkv + h) * page_size + row] =
          w ? w[(static_cast<int64_t>(b) * Hkv + h) * N + i] : 0.f;
}

// ---------------------------------------------------------------------------------------------
// Decode. One block per (b, query head); each warp takes every fourth visible token with the
// running maximum and sum of an online softmax, and the four are merged at the end.
struct Visible {
  int lo, hi;
};
__device__ __forceinline__ Visible visible_tokens(const int* __restrict__ seqlens, int b,
                                                  int capacity, int window_left) {
  int len = seqlens[b];
  if (len > capacity || len < 0) {
    record_page_error();
    len = min(max(len, 0), capacity);
  }
  const int lo = window_left >= 0 ? max(0, len - 1 - window_left) : 0;
  return {lo, len};
}

template <int D, bool FP16>
__global__ void __launch_bounds__(128)
    fa_paged_decode_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k_pages,
                           const uint16_t* __restrict__ v_pages, const int* __restrict__ table,
                           const int* __restrict__ seqlens, uint16_t* __restrict__ o,
                           float* __restrict__ lse, int Hq, int Hkv, int page_size, int num_pages,
                           int max_pages, int window_left, float scale_log2) {
  constexpr int E = D / 32;
  const int b = blockIdx.x / Hq, h = blockIdx.x % Hq, hk = h / (Hq / Hkv);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Visible vis = visible_tokens(seqlens, b, max_pages * page_size, window_left);
  float qr[E], acc[E];
  for (int e = 0; e < E; ++e) {
    qr[e] = to_float<FP16>(q[static_cast<int64_t>(blockIdx.x) * D + lane + 32 * e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = vis.lo + warp; t < vis.hi; t += 4) {
    const int page =
        page_at(table, static_cast<int64_t>(b) * max_pages + t / page_size, num_pages);
    if (page < 0) continue;
    const int64_t at =
        ((static_cast<int64_t>(page) * page_size + t % page_size) * Hkv + hk) * D + lane;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(qr[e], to_float<FP16>(k_pages[at + 32 * e]), s);
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= scale_log2;
    const float m_new = fmaxf(m, s), m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m - m_use), p = exp2f(s - m_use);
    m = m_new;
    l = l * alpha + p;
    for (int e = 0; e < E; ++e)
      acc[e] = acc[e] * alpha + p * to_float<FP16>(v_pages[at + 32 * e]);
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float sum = 0.f, f[4];
  for (int x = 0; x < 4; ++x) {
    f[x] = mx == -INFINITY ? 0.f : exp2f(sm[x] - mx);
    sum += sl[x] * f[x];
  }
  for (int c = threadIdx.x; c < D; c += 128) {
    float a = 0.f;
    for (int x = 0; x < 4; ++x) a += so[x][c] * f[x];
    o[static_cast<int64_t>(blockIdx.x) * D + c] = from_float<FP16>(sum > 0.f ? a / sum : 0.f);
  }
  if (threadIdx.x == 0)
    lse[blockIdx.x] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// weights[page, hk, row] += sum over the group's heads of exp(s - LSE): one warp per token.
template <int D, bool FP16>
__global__ void __launch_bounds__(256)
    fa_paged_weights_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k_pages,
                            float* __restrict__ weights, const int* __restrict__ table,
                            const int* __restrict__ seqlens, const float* __restrict__ lse, int Hq,
                            int Hkv, int page_size, int num_pages, int max_pages,
                            int window_left, float scale_log2) {
  constexpr int E = D / 32;
  const int b = blockIdx.y / Hkv, hk = blockIdx.y % Hkv, G = Hq / Hkv;
  const int lane = threadIdx.x % 32;
  const Visible vis = visible_tokens(seqlens, b, max_pages * page_size, window_left);
  for (int t = vis.lo + blockIdx.x * 8 + threadIdx.x / 32; t < vis.hi; t += gridDim.x * 8) {
    const int page =
        page_at(table, static_cast<int64_t>(b) * max_pages + t / page_size, num_pages);
    if (page < 0) continue;
    const int row = t % page_size;
    const int64_t at = ((static_cast<int64_t>(page) * page_size + row) * Hkv + hk) * D + lane;
    float kr[E], sum = 0.f;
    for (int e = 0; e < E; ++e) kr[e] = to_float<FP16>(k_pages[at + 32 * e]);
    for (int g = 0; g < G; ++g) {
      const int64_t hrow = static_cast<int64_t>(b) * Hq + hk * G + g;
      float s = 0.f;
      for (int e = 0; e < E; ++e) s = fmaf(kr[e], to_float<FP16>(q[hrow * D + lane + 32 * e]), s);
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float l = lse[hrow];
      if (l != -INFINITY) sum += exp2f(s * scale_log2 - l * kLog2e);
    }
    if (lane == 0)
      atomicAdd(&weights[(static_cast<int64_t>(page) * Hkv + hk) * page_size + row], sum);
  }
}

template <int D, bool FP16>
cudaError_t decode_impl(const DecodeParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  const uint16_t* q = static_cast<const uint16_t*>(p.q);
  const uint16_t* k = static_cast<const uint16_t*>(c.k_pages);
  fa_paged_decode_kernel<D, FP16><<<c.B * p.Hq, 128, 0, stream>>>(
      q, k, static_cast<const uint16_t*>(c.v_pages), c.block_table, c.seqlens,
      static_cast<uint16_t*>(p.o), p.lse, p.Hq, c.Hkv, c.page_size, c.num_pages, c.max_pages,
      p.window_left, p.scale_log2);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !c.weights) return err;
  // (b, hk) on the grid's second axis: at most 65535 rows there
  if (static_cast<int64_t>(c.B) * c.Hkv > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(64, c.B * c.Hkv);
  fa_paged_weights_kernel<D, FP16><<<grid, 256, 0, stream>>>(
      q, k, c.weights, c.block_table, c.seqlens, p.lse, p.Hq, c.Hkv, c.page_size, c.num_pages,
      c.max_pages, p.window_left, p.scale_log2);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Evict. One block per (b, hk).
constexpr int kEvictThreads = 1024;

// Weights as unsigned numbers in the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum of `x` over the threads before this one, and over all of them.
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t* scratch, uint32_t* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t inc = x;
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int i = 0; i < kEvictThreads / 32; ++i) {
    if (i < warp) before += scratch[i];
    all += scratch[i];
  }
  *total = all;
  return before + inc - x;
}

__global__ void __launch_bounds__(kEvictThreads)
    fa_paged_evict_kernel(uint4* __restrict__ k_pages, uint4* __restrict__ v_pages,
                          float* __restrict__ weights, const int* __restrict__ table,
                          const int* __restrict__ seqlens, const int* __restrict__ out_table,
                          int* __restrict__ kept_all, int* __restrict__ new_seqlens, int Hkv,
                          int d, int page_size, int num_pages, int max_pages, int out_pages,
                          int budget, int recent) {
  __shared__ uint32_t hist[256], scratch[32];
  __shared__ uint32_t s_digit, s_before;
  __shared__ int s_bad;
  const int b = blockIdx.x / Hkv, hk = blockIdx.x % Hkv, tid = threadIdx.x;
  const int* src_table = table + static_cast<int64_t>(b) * max_pages;
  const int* dst_table = out_table + static_cast<int64_t>(b) * out_pages;
  int* kept = kept_all + static_cast<int64_t>(blockIdx.x) * budget;
  const int raw_len = seqlens[b];
  if (tid == 0) s_bad = raw_len < 0 || raw_len > max_pages * page_size;
  __syncthreads();
  const int len = s_bad ? 0 : raw_len, new_len = min(len, budget);
  const int src_used = (len + page_size - 1) / page_size;
  const int dst_used = (new_len + page_size - 1) / page_size;
  __syncthreads();
  for (int i = tid; i < src_used; i += kEvictThreads)
    if (src_table[i] < 0 || src_table[i] >= num_pages) s_bad = 1;
  for (int i = tid; i < dst_used; i += kEvictThreads) {
    const int page = dst_table[i];
    if (page < 0 || page >= num_pages) s_bad = 1;
    for (int j = i + 1; j < src_used; ++j)
      if (src_table[j] == page) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    for (int i = tid; i < budget; i += kEvictThreads) kept[i] = -1;
    if (tid == 0) {
      record_page_error();
      if (hk == 0) new_seqlens[b] = raw_len;
    }
    return;
  }
  if (tid == 0 && hk == 0) new_seqlens[b] = new_len;
  auto weight_at = [&](const int* tab, int t) -> float* {
    return weights + (static_cast<int64_t>(tab[t / page_size]) * Hkv + hk) * page_size +
           t % page_size;
  };

  if (len <= budget) {
    for (int i = tid; i < budget; i += kEvictThreads) kept[i] = i < len ? i : -1;
  } else {
    // The candidates are tokens [0, n); `want` of them stay. Radix selection from the top
    // digit finds the want-th largest key; equal keys are taken from the lowest token.
    const int n = len - recent;
    uint32_t want = budget - recent, prefix = 0;
    for (int shift = 24; shift >= 0 && want; shift -= 8) {
      for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int t = tid; t < n; t += kEvictThreads) {
        const uint32_t key = order_key(*weight_at(src_table, t));
        if (shift == 24 || (key >> (shift + 8)) == prefix)
          atomicAdd(&hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t before = 0;
        int digit = 255;
        while (digit > 0 && before + hist[digit] < want) before += hist[digit--];
        s_digit = digit;
        s_before = before;
      }
      __syncthreads();
      prefix = prefix << 8 | s_digit;
      want -= s_before;   // of the keys that start with prefix
      __syncthreads();
    }
    const bool any = budget > recent;
    uint32_t placed = 0, equal_seen = 0;
    for (int t0 = 0; t0 < n; t0 += kEvictThreads) {
      const int t = t0 + tid;
      const uint32_t key = t < n ? order_key(*weight_at(src_table, t)) : 0u;
      const uint32_t is_equal = any && t < n && key == prefix;
      uint32_t equal_total, keep_total;
      const uint32_t rank = equal_seen + block_prefix(is_equal, scratch, &equal_total);
      const uint32_t keep = any && t < n && (key > prefix || (is_equal && rank < want));
      const uint32_t at = placed + block_prefix(keep, scratch, &keep_total);
      if (keep) kept[at] = t;
      equal_seen += equal_total;
      placed += keep_total;
    }
    for (int i = tid; i < recent; i += kEvictThreads) kept[budget - recent + i] = n + i;
  }
  __syncthreads();

  // The kept rows in order, a round of kEvictThreads tokens at a time: a round's reads come
  // before its writes, and a later round's sources lie behind every earlier destination.
  for (int i0 = 0; i0 < new_len; i0 += kEvictThreads) {
    const int i = i0 + tid;
    const int chunks = d / 8;
    int64_t src = 0, dst = 0;
    float w = 0.f;
    if (i < new_len) {
      const int t = kept[i];
      src = ((static_cast<int64_t>(src_table[t / page_size]) * page_size + t % page_size) * Hkv +
             hk) * chunks;
      dst = ((static_cast<int64_t>(dst_table[i / page_size]) * page_size + i % page_size) * Hkv +
             hk) * chunks;
      w = *weight_at(src_table, t);
    }
    for (int c = 0; c < chunks; ++c) {
      uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
      if (i < new_len) {
        kv = k_pages[src + c];
        vv = v_pages[src + c];
      }
      __syncthreads();
      if (i < new_len) {
        k_pages[dst + c] = kv;
        v_pages[dst + c] = vv;
      }
    }
    __syncthreads();
    if (i < new_len) *weight_at(dst_table, i) = w;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  fa_paged_append_kernel<<<static_cast<unsigned>(static_cast<int64_t>(c.B) * p.N), 128, 0,
                           stream>>>(
      static_cast<const uint4*>(p.k), static_cast<const uint4*>(p.v), p.w,
      static_cast<uint4*>(c.k_pages), static_cast<uint4*>(c.v_pages), c.weights, c.block_table,
      c.seqlens, p.new_lens, p.N, c.Hkv, c.d, c.page_size, c.num_pages, c.max_pages);
  return cudaGetLastError();
}

size_t paged_decode_workspace(int, int, int, int, int, int, bool) { return 16; }

cudaError_t launch_paged_decode(const DecodeParams& p, cudaStream_t stream) {
  if (p.c.d == 64)
    return p.fp16 ? decode_impl<64, true>(p, stream) : decode_impl<64, false>(p, stream);
  return p.fp16 ? decode_impl<128, true>(p, stream) : decode_impl<128, false>(p, stream);
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  fa_paged_evict_kernel<<<c.B * c.Hkv, kEvictThreads, 0, stream>>>(
      static_cast<uint4*>(c.k_pages), static_cast<uint4*>(c.v_pages), c.weights, c.block_table,
      c.seqlens, p.out_table, p.kept, p.new_seqlens, c.Hkv, c.d, c.page_size, c.num_pages,
      c.max_pages, p.out_pages, p.budget, p.recent);
  return cudaGetLastError();
}

cudaError_t read_and_clear_paged_error(int* value) {
  int bits = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&bits, g_paged_error, sizeof(int));
  if (err != cudaSuccess) return err;
  *value = bits & 1 ? kErrTimeout : bits & kPageError ? kErrPage : 0;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(int));
}

}  // namespace fa
