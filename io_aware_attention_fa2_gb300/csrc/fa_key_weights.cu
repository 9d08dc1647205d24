// fa_key_weights.cu -- the attention weight that every key of a prompt received:
//   w[b, hk, j] = sum_{h of hk} sum_{i sees j} exp(scale <q_i, k_j> - LSE[b, h, i]).
//
// The forward's S and its softmax statistics again, without P V: 2 d operations and one
// exponential for every visible (query, key) pair, and no tensor larger than the inputs. It is
// bound by the tensor pipe and the exponentials (at d = 128 a 128 x 128 tile is 4.2 MFLOP and
// 16384 exponentials).
//
// Keys are the rows: S^T = K Q^T puts one key in each TMEM lane, so that the sum over queries is
// a sum inside a thread, and the query's LSE is a value that all lanes share (a broadcast read
// from shared memory). One CTA takes 256 keys (two tiles, A and B) of one (batch, query head),
// keeps them in shared memory and walks the tiles of 256 queries that see them:
//   warp 0       TMA producer: K_A, K_B once, then the Q tiles through a ring
//   warp 1       TMEM allocator and MMA issuer (one thread): S_A and S_B in turn, 256 columns
//                each
//   warps 2..9   S_A: p = 2^(scale_log2 S - LSE log2 e), summed per key, four warps for each 128
//                queries of the tile; warps 10..17 the same for S_B. Nothing synchronises them
//                but the S buffers: every warp keeps its own copy of the LSEs that it needs.
// One half of the warps sums S_A while S_B is computed, and the other way round. Measured on B=1
// H=16 N=16384 d=128 causal: 390 us alone (1411 TFLOP/s, 74 % of the measured dense bf16 peak),
// 413-417 among other calls, at the power limit (d=64: 363). Of the 390 the products alone take
// 309 and the sums alone 375: the exponentials (32 a cycle and
// SM, 55 % busy) and the shared-memory reads of the LSEs share an issue queue, and four warps a
// scheduler do not fill their latencies. Slower: all sixteen warps on S_A, then on S_B (421 us);
// eight warps with twice the columns (427); 32-column loads of S one ahead of the sums (439);
// 16x256b loads of S, which need half of the LSE reads (468); products with 128 queries, whose
// operands are 8 KB of shared memory for 64 cycles of work (494). The same: CTAs that take
// further units off the hardware's launch queue instead of ending (395).
//
// Sums: 32 bits, 64 queries at a time in four chains, the tiles' sums added with Kahan's
// compensation: a key of a long prompt is the sum of many thousand terms. With shared key heads
// each query head writes its own sums (fp32 workspace) and a second kernel adds them in the order
// of the heads, so that the result does not depend on which CTA ends first.
#include <algorithm>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kQueries = 256;                               // queries of a tile
constexpr int kThreads = 64 + 512;
constexpr int kCols = 64;                                   // columns of S in registers
constexpr uint32_t kBoxBytes = BOX_ROWS * BOX_COLS * 2;     // 16 KiB
constexpr uint64_t kWaitLimitNs = 1000000000ull;            // 1 s per wait
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 2 : 4;          // depth of the Q ring
  static constexpr uint32_t kKTile = (D / BOX_COLS) * kBoxBytes;
  static constexpr uint32_t kQTile = 2 * kKTile;            // 64 columns of 256 queries, twice
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kQ = 2 * kKTile;
  static constexpr uint32_t kLse = kQ + kStages * kQTile;   // [warp][buffer][128] floats
  static constexpr uint32_t kSums = kLse + 16 * 2 * 128 * 4;   // [half][256] floats
  static constexpr uint32_t kBars = kSums + 2 * 256 * 4;
  static constexpr uint32_t kDynamic = kBars + 16 * 8 + 1024;
};

enum : int {
  BAR_K_FULL = 0,
  BAR_S_FULL = 1,                         // + tile
  BAR_S_EMPTY = BAR_S_FULL + 2,           // + tile (one arrival a warp)
  BAR_MMA_DONE = BAR_S_EMPTY + 2,
  BAR_Q_FULL = BAR_MMA_DONE + 1,          // + stage
  BAR_Q_EMPTY = BAR_Q_FULL + 4,           // + stage
  BAR_COUNT = BAR_Q_EMPTY + 4
};
static_assert(BAR_COUNT <= 16, "barrier slots");

__device__ __forceinline__ void record_timeout(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_error, kTimeoutBit);
}

// The queries that see key j: [lo(j), hi(j)), both nondecreasing in j.
struct QueryMask {
  int len, causal, left, right;
  __device__ __forceinline__ int lo(int j) const {
    int a = causal ? j : 0;
    if (right >= 0) a = max(a, j - right);
    return a;
  }
  __device__ __forceinline__ int hi(int j) const {
    return left >= 0 ? min(len, j + left + 1) : len;
  }
  // Query tiles [t0, t1) that see a key of the tile starting at k0; t1 <= t0 when none does.
  __device__ __forceinline__ void tile_range(int k0, int& t0, int& t1) const {
    const int a = lo(k0), z = k0 < len ? hi(min(k0 + BLOCK_N, len) - 1) : 0;
    t0 = z <= a ? 0 : a / kQueries;
    t1 = z <= a ? 0 : (z + kQueries - 1) / kQueries;
  }
};

// Bits [lo, hi) of 64.
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 64);
  hi = min(max(hi, 0), 64);
  if (hi <= lo) return 0;
  return (hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((1ull << lo) - 1);
}

// Sum over 64 queries of 2^(scale_log2 s + nl), of those with a bit in `visible` alone when
// MASKED.
template <bool MASKED>
__device__ __forceinline__ float tile_sum(const uint32_t (&sr)[2][32], const float* nl,
                                          float scale_log2, uint64_t visible) {
  float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < kCols / 4; ++c) {
    const float4 n4 = *reinterpret_cast<const float4*>(nl + 4 * c);
    const uint32_t(&s)[32] = sr[c / 8];
    const int o = 4 * (c % 8);
    float e[4];
    ptx::fma2(e[0], e[1], __uint_as_float(s[o]), __uint_as_float(s[o + 1]), scale_log2,
              scale_log2, n4.x, n4.y);
    ptx::fma2(e[2], e[3], __uint_as_float(s[o + 2]), __uint_as_float(s[o + 3]), scale_log2,
              scale_log2, n4.z, n4.w);
    if constexpr (MASKED) {
      const uint32_t bits = static_cast<uint32_t>(visible >> (c < 8 ? 0 : 32)) >> (4 * (c % 8));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!(bits & (1u << k))) e[k] = -INFINITY;
    }
    ptx::add2(t[0], t[1], t[0], t[1], ptx::exp2_approx(e[0]), ptx::exp2_approx(e[1]));
    ptx::add2(t[2], t[3], t[2], t[3], ptx::exp2_approx(e[2]), ptx::exp2_approx(e[3]));
  }
  return (t[0] + t[1]) + (t[2] + t[3]);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const float* lse, float* out, int Hq, int G, int N, int causal, int left,
                          int right, const int* seqlens, float scale_log2, int heads_per_group) {
  using L = Smem<D>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = base + L::kK, sQ = base + L::kQ;
  uint8_t* const gen = smem_raw + (base - ptx::smem_addr(smem_raw));
  auto bar = [&](int i) { return base + L::kBars + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  wait_prerequisites();
  launch_dependents();
  // Unit from a 1-D grid: heads in groups whose Q stays in L2, in a group key block by key
  // block, the first (seen by the most queries when causal) first.
  const int num_kblk = (N + 2 * BLOCK_N - 1) / (2 * BLOCK_N);
  const int num_bh = gridDim.x / num_kblk;
  const int group_units = heads_per_group * num_kblk;
  const int grp = static_cast<int>(blockIdx.x) / group_units;
  const int rem = static_cast<int>(blockIdx.x) % group_units;
  const int g_size = min(heads_per_group, num_bh - grp * heads_per_group);
  const int bh = grp * heads_per_group + rem % g_size;
  const int kblk = rem / g_size;
  const int b = bh / Hq, h = bh % Hq;
  QueryMask mask;
  mask.len = seqlens ? min(max(seqlens[b], 0), N) : N;
  mask.causal = causal;
  mask.left = left;
  mask.right = right;
  // query tiles of key tiles A and B, and their union [u0, u1), which the producer streams
  int a0, a1, b0, b1;
  mask.tile_range(2 * kblk * BLOCK_N, a0, a1);
  mask.tile_range((2 * kblk + 1) * BLOCK_N, b0, b1);
  const bool a_any = a1 > a0, b_any = b1 > b0, any_work = a_any || b_any;
  const int u0 = a_any ? (b_any ? min(a0, b0) : a0) : b0;
  const int u1 = max(a1, b1);

  // Q tile u0 + n into its stage of the ring
  auto load_q = [&](int n) {
    const int s = n % kStages;
    ptx::mbar_arrive_expect_tx(bar(BAR_Q_FULL + s), L::kQTile);
    for (int c = 0; c < D / BOX_COLS; ++c)
      for (int r = 0; r < 2; ++r)
        ptx::tma_load_4d(sQ + s * L::kQTile + (2 * c + r) * kBoxBytes, &tm_q, bar(BAR_Q_FULL + s),
                         c * BOX_COLS, h, (u0 + n) * kQueries + r * BOX_ROWS, b);
  };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    ptx::mbar_init(bar(BAR_K_FULL), 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(BAR_Q_FULL + s), 1);
      ptx::mbar_init(bar(BAR_Q_EMPTY + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(bar(BAR_S_FULL + x), 1);
      ptx::mbar_init(bar(BAR_S_EMPTY + x), 8);
    }
    ptx::mbar_init(bar(BAR_MMA_DONE), 1);
    ptx::fence_barrier_init();
    // K and the first Q tiles are on their way before the other warps and TMEM are ready (B=1 H=8
    // N=500 d=64: 10.2 -> 9.7 us)
    if (any_work) {
      ptx::mbar_arrive_expect_tx(bar(BAR_K_FULL), 2 * L::kKTile);
      for (int x = 0; x < 2; ++x)
        for (int c = 0; c < D / BOX_COLS; ++c)
          ptx::tma_load_4d(sK + x * L::kKTile + c * kBoxBytes, &tm_k, bar(BAR_K_FULL),
                           c * BOX_COLS, h / G, (2 * kblk + x) * BLOCK_N, b);
      for (int n = 0; n < min(kStages, u1 - u0); ++n) load_q(n);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&tmem_base_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = tmem_base_slot;
  volatile int* abort_p = &abort_flag;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0 && any_work) {
      int issued = min(kStages, u1 - u0);
      for (int n = issued; n < u1 - u0; ++n) {
        if (!ptx::wait_bounded(bar(BAR_Q_EMPTY + n % kStages), ((n / kStages) & 1) ^ 1, abort_p,
                               kWaitLimitNs)) {
          record_timeout(abort_p);
          break;
        }
        load_q(n);
        issued = n + 1;
      }
      // Leave no copy in flight (on the normal path these phases completed long ago).
      ptx::wait_bounded(bar(BAR_K_FULL), 0, abort_p, kWaitLimitNs);
      for (int n = max(0, issued - kStages); n < issued; ++n)
        ptx::wait_bounded(bar(BAR_Q_FULL + n % kStages), (n / kStages) & 1, abort_p,
                          kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_f16(FP16, BLOCK_N, kQueries, false);
      auto wait = [&](int slot, uint32_t parity) {
        return ptx::wait_bounded(bar(slot), parity, abort_p, kWaitLimitNs);
      };
      bool ok = !any_work || wait(BAR_K_FULL, 0);
      for (int i = u0; ok && i < u1; ++i) {
        const int n = i - u0, s = n % kStages;
        if (!wait(BAR_Q_FULL + s, (n / kStages) & 1)) { ok = false; break; }
        const ptx::SmemDesc q_desc = ptx::smem_desc_sw128_split(sQ + s * L::kQTile, 16, 1024);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int x0 = x ? b0 : a0, x1 = x ? b1 : a1;
          if (i < x0 || i >= x1) continue;
          if (!wait(BAR_S_EMPTY + x, ((i - x0) & 1) ^ 1)) { ok = false; break; }
          ptx::tc_fence_after_sync();
          const ptx::SmemDesc k_desc = ptx::smem_desc_sw128_split(sK + x * L::kKTile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_f16_ss(tmem + x * kQueries, k_desc.at((kk / 4) * kBoxBytes + (kk % 4) * 32),
                            q_desc.at((kk / 4) * 2 * kBoxBytes + (kk % 4) * 32), idesc, kk > 0);
          ptx::mma_commit(bar(BAR_S_FULL + x));
        }
        ptx::mma_commit(bar(BAR_Q_EMPTY + s));
      }
      if (!ok) record_timeout(abort_p);
      // Every MMA this thread issued has completed before TMEM can be released.
      ptx::mma_commit(bar(BAR_MMA_DONE));
      wait(BAR_MMA_DONE, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ sums over queries
    const int cw = warp - 2, x = cw / 8, half = cw / 4 % 2;   // key tile; 128 of the queries
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;               // TMEM lane = key of the tile
    const int k0 = (2 * kblk + x) * BLOCK_N, key = k0 + row;
    const int x0 = x ? b0 : a0, x1 = x ? b1 : a1;
    const uint32_t tS =
        tmem + (static_cast<uint32_t>(quarter * 32) << 16) + x * kQueries + half * 128;
    float* const my_lse = reinterpret_cast<float*>(gen + L::kLse) + cw * 2 * 128;
    const float* lse_row = lse + static_cast<int64_t>(bh) * N;
    // LSE of query q as it is loaded (one tile ahead), and as it is used: negated, in log2 units,
    // -inf where the query adds nothing
    auto load_lse = [&](int q) { return q < mask.len ? lse_row[q] : -INFINITY; };
    auto minus_log2 = [](float v) { return v == -INFINITY ? v : -v * kLog2e; };
    float total = 0.f, comp = 0.f;
    int q0 = x0 * kQueries + half * 128;               // first of the warp's queries of tile i
    // Queries [q_lo, q_hi) see this key; queries inside [full_lo, full_hi) are seen by every key
    // of the tile, those outside [any_lo, any_hi) by none. (Keys at or past len are left out at
    // the end.)
    const int q_lo = mask.lo(key), q_hi = mask.hi(key);
    const int full_lo = mask.lo(k0 + BLOCK_N - 1), full_hi = mask.hi(k0);
    const int any_lo = mask.lo(k0), any_hi = mask.hi(k0 + BLOCK_N - 1);
    float next[4] = {0.f, 0.f, 0.f, 0.f};
    if (x1 > x0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = load_lse(q0 + 32 * e + lane);
    }
    bool ok = true;
    for (int i = x0; i < x1; ++i, q0 += kQueries) {
      float* const nl = my_lse + (i & 1) * 128;
#pragma unroll
      for (int e = 0; e < 4; ++e) nl[32 * e + lane] = minus_log2(next[e]);
      if (i + 1 < x1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) next[e] = load_lse(q0 + kQueries + 32 * e + lane);
      }
      __syncwarp();
      if (!ptx::wait_bounded_warp(bar(BAR_S_FULL + x), (i - x0) & 1, abort_p, kWaitLimitNs)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after_sync();
      float tile = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t sr[2][32];
        ptx::tmem_ld_32x32b_x32(tS + 64 * hf, sr[0]);
        ptx::tmem_ld_32x32b_x32(tS + 64 * hf + 32, sr[1]);
        ptx::tmem_wait_ld();
        if (hf == 1) {
          ptx::tc_fence_before_sync();
          if (lane == 0) ptx::mbar_arrive(bar(BAR_S_EMPTY + x));
        }
        ptx::reg_fence(sr[0]);
        ptx::reg_fence(sr[1]);
        const int q = q0 + 64 * hf;
        if (q >= full_lo && q + 64 <= full_hi)
          tile += tile_sum<false>(sr, nl + 64 * hf, scale_log2, 0);
        else if (q < any_hi && q + 64 > any_lo)
          tile += tile_sum<true>(sr, nl + 64 * hf, scale_log2, bit_range(q_lo - q, q_hi - q));
      }
      const float y = tile - comp;
      const float sum = total + y;
      comp = (sum - total) - y;
      total = sum;
    }
    if (!ok) record_timeout(abort_p);
    // the two halves' sums of each key
    float* const sums = reinterpret_cast<float*>(gen + L::kSums);
    sums[half * 256 + x * 128 + row] = total;
    ptx::named_barrier_sync(1, 512);
    const int at = threadIdx.x - 64, okey = 2 * kblk * BLOCK_N + at;
    if (at < 256 && okey < N)
      out[static_cast<int64_t>(bh) * N + okey] = okey < mask.len ? sums[at] + sums[256 + at] : 0.f;
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// w[b, hk, j] = sum over the G query heads, in their order, of part[b, hk * G + g, j].
__global__ void __launch_bounds__(256)
    fa_key_weights_sum_kernel(const float* part, float* w, int G, int N, int64_t count) {
  wait_prerequisites();
  launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= count) return;
  const int64_t head = at / N, j = at % N;
  float sum = 0.f;
  for (int g = 0; g < G; ++g) sum += part[(head * G + g) * N + j];
  w[at] = sum;
}

template <int D, bool FP16>
cudaError_t launch_impl(const KeyWeightsParams& p, cudaStream_t stream) {
  auto kernel = fa_key_weights_kernel<D, FP16>;
  const int smem = static_cast<int>(Smem<D>::kDynamic);
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const int64_t bh = static_cast<int64_t>(p.B) * p.Hq;
  const int64_t num_kblk = (p.N + 2 * BLOCK_N - 1) / (2 * BLOCK_N);
  const int G = p.Hq / p.Hkv;
  // Heads per dispatch group: their Q within 32 MiB, a quarter of L2, as in the forward.
  const int64_t q_bytes = 2ll * p.N * D;
  const int heads_per_group =
      static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(bh, (32ll << 20) / q_bytes)));
  err = launch_chained(kernel, bh * num_kblk, kThreads, smem, stream, 0, p.tm_q, p.tm_k, p.lse,
                       G > 1 ? p.part : p.w, p.Hq, G, p.N, p.causal, p.window_left, p.window_right,
                       p.seqlens_k, p.scale_log2, heads_per_group);
  if (err != cudaSuccess || G == 1) return err;
  const int64_t count = static_cast<int64_t>(p.B) * p.Hkv * p.N;
  return launch_chained(fa_key_weights_sum_kernel, (count + 255) / 256, 256, 0, stream, 0, p.part,
                        p.w, G, p.N, count);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  if (p.d == 64)
    return p.fp16 ? launch_impl<64, true>(p, stream) : launch_impl<64, false>(p, stream);
  return p.fp16 ? launch_impl<128, true>(p, stream) : launch_impl<128, false>(p, stream);
}

cudaError_t read_and_clear_key_weights_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
