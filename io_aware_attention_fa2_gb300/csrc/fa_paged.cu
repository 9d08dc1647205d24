// fa_paged.cu -- the paged key-value cache: append and evict (include/fa.h has the layouts and
// the rules for bad block-table entries and lengths).
#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;

constexpr int kErrTimeout = -8, kErrPage = -13;   // FA_ERR_TIMEOUT, FA_ERR_PAGE

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
  cudaError_t err = read_and_clear_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_decode_error(&bits);
  *value = bits & kTimeoutBit ? kErrTimeout : bits & kPageBit ? kErrPage : 0;
  return err;
}

}  // namespace fa
