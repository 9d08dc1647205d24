// fa_paged_tree.cu -- attention of drafted tokens over a paged key-value cache: each sees its
// sequence's context, its ancestors in the draft's tree and itself (include/fa.h).
//
// A block for each (sequence, drafted token, query head): its four warps take every fourth token
// with a running maximum, sum and O of their own, joined at the end.
#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 128, kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float2 widen(uint32_t v);
template <>
__device__ __forceinline__ float2 widen<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) fa_paged_tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr int kPairs = D / 64;   // pairs of columns of a lane: 64 x + 2 lane, + 1
  __shared__ uint32_t s_seen[kMaxDraft / 32];
  __shared__ int s_depth;
  __shared__ short s_up[kMaxDraft];     // token -> its depth, for ancestors
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ __align__(16) float s_o[kWarps][D];   // (accessed as float2)
  const int h = blockIdx.x % p.Hq, i = blockIdx.x / p.Hq % p.T, b = blockIdx.x / p.Hq / p.T;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const PagedCache& c = p.c;
  wait_prerequisites();
  launch_dependents();
  const Draft dr = draft_of(c.seqlens, p.new_lens, b, p.T, c.max_pages * c.page_size);
  const int64_t row = static_cast<int64_t>(blockIdx.x);
  E* const o = static_cast<E*>(p.o) + row * D;
  float* const lse = p.lse + (static_cast<int64_t>(b) * p.Hq + h) * p.T + i;
  if (dr.count < 0 && threadIdx.x == 0) record_page_error();
  if (threadIdx.x < kMaxDraft / 32) s_seen[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x == 0 && i < dr.count) {
    int n = 0;
    for (int at = i; at >= 0; ++n) {
      s_seen[at / 32] |= 1u << (at % 32);
      s_up[at] = static_cast<short>(n);
      int up = at - 1;
      if (p.parents) {
        up = p.parents[static_cast<int64_t>(b) * p.T + at];
        if (up < -1 || up >= at) {
          record_page_error();
          up = -1;
        }
      }
      at = up;
    }
    s_depth = n - 1;
  }
  __syncthreads();
  const E* const q = static_cast<const E*>(p.q) + row * D;
  float2 qv[kPairs], acc[kPairs];
#pragma unroll
  for (int x = 0; x < kPairs; ++x) {
    qv[x] = widen<E>(*reinterpret_cast<const uint32_t*>(q + 64 * x + 2 * lane));
    acc[x] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  const int last = i < dr.count ? dr.base + i : -1;
  const int first =
      i < dr.count && p.window_left >= 0 ? max(0, dr.base + s_depth - p.window_left) : 0;
  for (int t = min(first, dr.base) + warp; t <= last; t += kWarps) {
    if (t < dr.base) {
      if (t < first) continue;
    } else {
      const int j = t - dr.base;
      if (!(s_seen[j / 32] >> (j % 32) & 1)) continue;
      if (p.window_left >= 0 && s_up[j] > p.window_left) continue;
    }
    const int page = c.block_table[static_cast<int64_t>(b) * c.max_pages + t / c.page_size];
    if (page < 0 || page >= c.num_pages) {
      record_page_error();
      continue;
    }
    const int64_t at =
        ((static_cast<int64_t>(page) * c.page_size + t % c.page_size) * c.Hkv + h / (p.Hq / c.Hkv)) * D;
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < kPairs; ++x) {
      const float2 k = widen<E>(*reinterpret_cast<const uint32_t*>(
          static_cast<const E*>(c.k_pages) + at + 64 * x + 2 * lane));
      s += qv[x].x * k.x + qv[x].y * k.y;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float n = fmaxf(m, s), u = n == -INFINITY ? 0.f : n;
    const float f = exp2f(m - u), e = exp2f(s - u);
    m = n;
    l = l * f + e;
#pragma unroll
    for (int x = 0; x < kPairs; ++x) {
      const float2 v = widen<E>(*reinterpret_cast<const uint32_t*>(
          static_cast<const E*>(c.v_pages) + at + 64 * x + 2 * lane));
      acc[x].x = acc[x].x * f + e * v.x;
      acc[x].y = acc[x].y * f + e * v.y;
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < kPairs; ++x)
    *reinterpret_cast<float2*>(&s_o[warp][64 * x + 2 * lane]) = acc[x];
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float u = m == -INFINITY ? 0.f : m;
  float sum = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = exp2f(s_m[w] - u);
    sum += s_l[w] * f[w];
  }
  for (int x = threadIdx.x; x < D; x += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_o[w][x] * f[w];
    put(o + x, sum == 0.f ? 0.f : v / sum);
  }
  if (threadIdx.x == 0) *lse = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

}  // namespace

size_t paged_tree_workspace(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_paged_tree(const TreeParams& p, cudaStream_t stream) {
  const int64_t grid = static_cast<int64_t>(p.c.B) * p.T * p.Hq;
  if (p.c.d == 64)
    return p.fp16 ? launch_paged(fa_paged_tree_kernel<__half, 64>, grid, kThreads, 0, stream, 0, p)
                  : launch_paged(fa_paged_tree_kernel<__nv_bfloat16, 64>, grid, kThreads, 0, stream, 0, p);
  return p.fp16 ? launch_paged(fa_paged_tree_kernel<__half, 128>, grid, kThreads, 0, stream, 0, p)
                : launch_paged(fa_paged_tree_kernel<__nv_bfloat16, 128>, grid, kThreads, 0, stream, 0, p);
}

cudaError_t read_and_clear_tree_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
