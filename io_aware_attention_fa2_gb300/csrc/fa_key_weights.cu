// fa_key_weights.cu -- the attention weight that every key of a prompt received:
//   w[b, hk, j] = sum_{h of hk} sum_{i sees j} exp(scale <q_i, k_j> - LSE[b, h, i]).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "ptx_sm103.cuh"

namespace fa {

__device__ int g_key_weights_error = 0;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <bool FP16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if constexpr (FP16) {
    return __half2float(__ushort_as_half(x));
  } else {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
}

// One warp per key: lane t holds components t, t + 32, ... of the key; the queries that see it
// are walked in order.
template <int D, bool FP16>
__global__ void __launch_bounds__(256)
    fa_key_weights_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k,
                          const float* __restrict__ lse, float* __restrict__ w, int B, int Hq,
                          int Hkv, int N, int causal, int left, int right,
                          const int* __restrict__ seqlens, float scale_log2) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(B) * Hkv * N) return;
  const int lane = threadIdx.x % 32;
  const int j = static_cast<int>(row % N);
  const int hk = static_cast<int>(row / N % Hkv), b = static_cast<int>(row / N / Hkv);
  const int len = seqlens ? min(max(seqlens[b], 0), N) : N;
  float kr[D / 32];
  for (int e = 0; e < D / 32; ++e)
    kr[e] = to_float<FP16>(k[((static_cast<int64_t>(b) * N + j) * Hkv + hk) * D + lane + 32 * e]);
  int lo = 0, hi = j < len ? len : 0;   // queries that see key j
  if (causal) lo = max(lo, j);
  if (left >= 0) hi = min(hi, j + left + 1);
  if (right >= 0) lo = max(lo, j - right);
  float sum = 0.f;
  for (int g = 0; g < Hq / Hkv; ++g) {
    const int h = hk * (Hq / Hkv) + g;
    for (int i = lo; i < hi; ++i) {
      const uint16_t* qr = q + ((static_cast<int64_t>(b) * N + i) * Hq + h) * D;
      float s = 0.f;
      for (int e = 0; e < D / 32; ++e) s = fmaf(kr[e], to_float<FP16>(qr[lane + 32 * e]), s);
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float l = lse[(static_cast<int64_t>(b) * Hq + h) * N + i];
      if (l != -INFINITY) sum += exp2f(s * scale_log2 - l * kLog2e);
    }
  }
  if (lane == 0) w[row] = sum;
}

template <int D, bool FP16>
cudaError_t launch_impl(const KeyWeightsParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.N;
  fa_key_weights_kernel<D, FP16><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(
      static_cast<const uint16_t*>(p.q), static_cast<const uint16_t*>(p.k), p.lse, p.w, p.B,
      p.Hq, p.Hkv, p.N, p.causal, p.window_left, p.window_right, p.seqlens_k, p.scale_log2);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  if (p.d == 64)
    return p.fp16 ? launch_impl<64, true>(p, stream) : launch_impl<64, false>(p, stream);
  return p.fp16 ? launch_impl<128, true>(p, stream) : launch_impl<128, false>(p, stream);
}

cudaError_t read_and_clear_key_weights_error(int* value) {
  cudaError_t err = cudaMemcpyFromSymbol(value, g_key_weights_error, sizeof(int));
  if (err != cudaSuccess) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_key_weights_error, &zero, sizeof(int));
}

}  // namespace fa
