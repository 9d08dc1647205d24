// fa_paged_decode.cu -- attention of one new token per sequence over a paged key-value cache.
//
//   s_j = scale <q, k_j>,  O = sum_j e^{s_j - LSE} v_j,  LSE = ln sum_j e^{s_j}
//
// over the visible tokens of each sequence, and with a cache that keeps weights
// weights[j] += sum over the query heads of the key head of e^{s_j - LSE}.
//
// What bounds it: K and V are read once, 4 d bytes a token and key head, against 4 G d
// operations for the G query heads that share it. On the FP32 pipe that is slower than HBM from
// G = 4 on, so both products run on the tensor cores: mma.sync m16n8k16 with the (up to 16) query
// heads of a key head as its 16 rows. The 16-row tile is the smallest there is; tcgen05 takes
// 64 or 128 rows, of which a key head's queries would fill a few, and the products are far from
// being the bound (the kernel waits on HBM).
//
// Work split. The tokens of a (sequence, key head, block of 16 query heads) -- a unit -- are cut
// into tiles of 64, and the tiles of all units, in order, into one equal run for each CTA (two
// CTAs on each SM), whatever the lengths are: a long sequence alone fills the GPU and a batch of
// unequal ones is balanced without the host knowing the lengths. A run that covers a whole unit
// writes O and LSE; one that covers a part leaves the part's running maximum, sum and
// unnormalised O (fp32) in the workspace, and a second kernel joins the parts of a unit in a
// fixed order. Each CTA recomputes where its run starts from seqlens.
//
// Measured (calls one after the other over three caches): B=16 GQA 4 lengths to 16K, pages of 16:
// 102-106 us, 6.1-6.3 TB/s, 90-93 % of the measured copy rate; B=4 GQA 8 to 64K: 54-56 us (77-80 %:
// 5 are the first loads' latency, 4 the join); B=8 GQA 4 to 32K with weights: 124-128 us (79-81 %;
// keeping the scores, most of which go through HBM, costs 8 us, adding the weights 11). The second
// product with P's rest costs nothing measurable, nor does keeping infinities out of it; two
// stages instead of three cost 2 % at B=16, one CTA of six stages on each SM 12 %.
//
// One CTA: warp 4 loads (TMA boxes of up to 64 rows of a page, all d columns of one head, into a
// ring of three tiles of K and V, 128-byte swizzle); warps 0..3 each take 16 tokens of every tile
// with a running maximum, sum and O of their own, so that nothing but the ring synchronises
// them until the run's end, when the four are joined through shared memory.
//
// P is kept as two 16-bit values, the rounded one and the rounded rest, for two products with V
// into one fp32 accumulator: O then carries the rounding of the output alone. fp16 ends at 2^-24,
// so there P is taken 2^15 times as large (at most 2^15 against a largest number of 65504) until
// a run's end: what is lost are probabilities below 2^-40 of the largest, not 2^-25, which many
// tokens behind a heavy one would miss.
//
// Weights need the final LSE: the scaled scores are kept (fp32, 4 G bytes a token against the
// 4 d of K and V) and the second kernel adds exp2(score - maximum) / sum over the group's heads.
// Short caches (the smallest calls, where latency counts) take one launch and no workspace: a
// cluster of up to eight CTAs has one unit, up to four tiles each, all of them on their way at
// once, and the parts are joined through distributed shared memory (choose_short has the rule).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;
namespace cg = cooperative_groups;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kTile = 64;                      // tokens of a tile
constexpr int kStagesLong = 3;                 // ring of tiles
constexpr int kShortTiles = 4;                 // tiles of a CTA of a short unit, one stage each
constexpr int kWarps = 4;                      // consumer warps, 16 tokens of a tile each
constexpr int kThreads = 32 * (kWarps + 1);    // and the producer warp
constexpr int kRows = 16;                      // query heads of a unit, at most
constexpr int kSms = 152;                      // of a GB300; on another count only speed differs
constexpr int kMaxCtas = 2 * kSms;             // two CTAs on each SM
constexpr int kMaxCluster = 8;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// P, its sums and the unnormalised O are 2^kPShift as large within a run.
template <bool FP16>
constexpr float kPShift = FP16 ? 15.f : 0.f;
template <bool FP16>
constexpr float kPUnshift = FP16 ? 1.f / 32768.f : 1.f;

template <int D, bool SHORT>
struct Smem {
  static constexpr int kStages = SHORT ? kShortTiles : kStagesLong;
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kStages * kTileBytes;
  // one half of the rows (8) and 64 columns of each warp's O at a time; rows padded by 32 bytes
  static constexpr int kJoinCols = 64, kJoinPitch = kJoinCols + 8;
  static constexpr uint32_t kJoin = 2 * kStages * kTileBytes;
  static constexpr uint32_t kStats = kJoin + kWarps * 8 * kJoinPitch * 4;   // m, l [warp][row]
  static constexpr uint32_t kMask = kStats + 2 * kWarps * kRows * 4;        // uint64 per stage
  static constexpr uint32_t kBars = kMask + kStages * 8;                    // full, empty
  // short units: this CTA's part (O, maxima and sums) and its scores
  static constexpr uint32_t kPart = (kBars + 2 * kStages * 8 + 15) / 16 * 16;   // [16][D] floats
  static constexpr uint32_t kPartMl = kPart + kRows * D * 4;                    // [16] float2
  static constexpr int kScorePitch = kShortTiles * kTile + 8;                   // floats
  static constexpr uint32_t kScores = kPartMl + kRows * 8;
  static constexpr uint32_t kEnd = SHORT ? kScores + kRows * kScorePitch * 4 : kPart;
  static constexpr uint32_t kDynamic = kEnd + 1024;   // slack for 1 KiB alignment
};

struct Args {
  const void* q;
  const int* table;
  const int* seqlens;
  void* o;
  float* lse;
  float* weights;
  float* part_o;      // [2 * CTAs][part_rows][D]: CTA c's first run at slot 2c, its last at 2c + 1
  float2* part_ml;    // [2 * CTAs][part_rows]: maximum (log2 units) and sum of the part
  int2* units;        // [B * Hkv * blocks]: slot of the unit's first part, number of parts (0: the
                      // unit was one run's, and is written)
  float2* stats;      // [B * Hq]: maximum and 1 / sum of a head that one run covered, when the
                      // cache keeps weights
  float* scores;      // [B * Hq][capacity], log2 units, when the cache keeps weights
  int B, Hq, Hkv, G, blocks;   // blocks of 16 query heads for each key head
  int part_rows;               // query heads of a unit, at most: min(G, 16)
  int page_size, num_pages, max_pages, capacity, box_rows;
  int window_left;
  float scale_log2;
};

// Tiles of sequence b: [first, first + count), at least one (an empty sequence's unit is
// written by the run that holds its empty tile).
struct Tiles {
  int lo, hi, first, count;
};
template <bool RECORD>
__device__ __forceinline__ Tiles tiles_of(const Args& a, int b) {
  const Visible v = visible_tokens<RECORD>(a.seqlens, b, a.capacity, a.window_left);
  const int first = v.lo / kTile;
  return {v.lo, v.hi, first, max(1, (v.hi - 1) / kTile + 1 - first)};
}

// Tiles of a unit summed over all sequences, by one warp.
__device__ __forceinline__ int64_t count_tiles(const Args& a) {
  int64_t x = 0;
  for (int b = threadIdx.x % 32; b < a.B; b += 32) x += tiles_of<false>(a, b).count;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// CTAs that get a run: every one of them at least a tile, so that no part of a unit is empty.
__device__ __forceinline__ int running(int64_t total, int ctas) {
  return static_cast<int>(min(total, static_cast<int64_t>(ctas)));
}
// First tile of CTA c's run, of `total` tiles over `ctas` running CTAs: floor(total * c / ctas).
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int ctas) {
  return total / ctas * c + total % ctas * c / ctas;
}

// 1 / sum of a row's probabilities: 0 for a row without any, NaN for a NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
// LSE in natural units from the maximum (log2 units) and the sum.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// A run as its segments: consecutive tiles of one unit.
struct Segment {
  int b, unit, tile, count;   // unit of the sequence, first tile of it, tiles
  bool whole;
};
struct Walk {
  int64_t left;    // tiles of the run that are left
  int64_t at;      // tile within sequence b's units
  int b;
};
template <bool RECORD>
__device__ __forceinline__ Segment next_segment(const Args& a, Walk& w, Tiles& t) {
  t = tiles_of<RECORD>(a, w.b);
  Segment s;
  s.b = w.b;
  s.unit = static_cast<int>(w.at / t.count);
  s.tile = static_cast<int>(w.at % t.count);
  s.count = static_cast<int>(min(static_cast<int64_t>(t.count - s.tile), w.left));
  s.whole = s.count == t.count;
  w.left -= s.count;
  w.at += s.count;
  if (w.at == static_cast<int64_t>(t.count) * a.Hkv * a.blocks) {
    w.at = 0;
    ++w.b;
  }
  return s;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b: a 16 x 16 (rows = query heads), b 16 x 8, fp32 accumulators.
template <bool FP16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (FP16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// (x, y) rounded to 16 bits each, and what the rounding left, rounded too.
template <bool FP16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
}
// Two 16-bit values with infinities (and NaN) replaced by the type's largest number of their sign.
template <bool FP16>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  uint32_t r;
  if constexpr (FP16)
    asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7bff7bffu));
  else
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7f7f7f7fu));
  return r;
}
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

// SHORT: a cluster of CTAs has one unit, each CTA an equal share of its tiles. Otherwise: runs
// over all units.
template <int D, bool FP16, bool WEIGHTS, bool SHORT>
__global__ void __launch_bounds__(kThreads, SHORT ? 1 : 2)
    fa_paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Args a) {
  using L = Smem<D, SHORT>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_flag, s_seq;
  __shared__ int64_t s_at, s_left, s_start, s_total;
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gen = smem_raw + (base - ptx::smem_addr(smem_raw));
  auto full = [&](int s) { return base + L::kBars + 8u * s; };
  auto empty = [&](int s) { return base + L::kBars + 8u * (kStages + s); };
  uint64_t* const masks = reinterpret_cast<uint64_t*>(gen + L::kMask);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;

  if (threadIdx.x == 32 * kWarps) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), kWarps);
    }
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  wait_prerequisites();
  launch_dependents();
  // where this CTA's run starts: the sequence, and the tile within it
  if (!SHORT && warp == 0) {
    const int64_t total = count_tiles(a) * a.Hkv * a.blocks;
    const int ctas = running(total, gridDim.x);
    const int64_t start = run_start(total, cta, ctas);
    // the last sequence whose first tile is at or before `start`
    int64_t before = 0, at = start;
    int seq = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t n =
          b < a.B ? static_cast<int64_t>(tiles_of<false>(a, b).count) * a.Hkv * a.blocks : 0;
      int64_t inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      const int64_t first = before + inc - n;
      const unsigned here = __ballot_sync(0xffffffffu, n > 0 && first <= start &&
                                                           start < before + inc);
      if (here) {
        const int src = __ffs(here) - 1;
        seq = b0 + src;
        at = start - __shfl_sync(0xffffffffu, first, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      s_seq = seq;
      s_at = at;
      s_left = cta < ctas ? run_start(total, cta + 1, ctas) - start : 0;
      s_start = start;
      s_total = total;
    }
  }
  __syncthreads();
  Walk walk{};
  if constexpr (!SHORT) walk = Walk{s_left, s_at, s_seq};
  const int rank = SHORT ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int ranks = SHORT ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
  // the segments of this CTA, one after the other: a short unit's share, or those of the run
  auto more = [&](int done) { return SHORT ? done == 0 : walk.left > 0; };
  auto next = [&](auto record, Tiles& t) {
    if constexpr (SHORT) {
      const int unit = cta / ranks, units = a.Hkv * a.blocks;
      Segment s;
      s.b = unit / units;
      s.unit = unit % units;
      t = tiles_of<decltype(record)::value>(a, s.b);
      s.tile = t.count * rank / ranks;
      s.count = t.count * (rank + 1) / ranks - s.tile;
      s.whole = false;
      return s;
    } else {
      return next_segment<decltype(record)::value>(a, walk, t);
    }
  };
  volatile int* abort_p = &abort_flag;
  auto give_up = [&] {
    *abort_p = 1;
    atomicOr(&g_error, kTimeoutBit);
  };

  if (warp == kWarps) {
    // ------------------------------------------------------------------ producer
    const int br = a.box_rows, boxes = kTile / br;
    const uint32_t box_bytes = static_cast<uint32_t>(br) * D * 2;
    int n = 0;   // tiles loaded so far: tile n goes through stage n % kStages
    bool ok = true;
    for (int done = 0; ok && more(done); ++done) {
      Tiles t;
      const Segment sg = next(std::true_type{}, t);
      const int hk = sg.unit / a.blocks;
      const int row0 = (t.first + sg.tile) * kTile;      // first token of the segment
      const int total_boxes = sg.count * boxes;
      const int* tab = a.table + static_cast<int64_t>(sg.b) * a.max_pages;
      // Box j holds tokens row0 + j * br ..; lane x keeps the table entries of boxes x,
      // 32 + x, ... one batch of 32 ahead of the loads.
      auto needed = [&](int j) {
        const int r = row0 + j * br;
        return j < total_boxes && r < t.hi && r + br > t.lo;
      };
      auto entry = [&](int j) { return needed(j) ? tab[(row0 + j * br) / a.page_size] : -1; };
      int cur = entry(lane), nxt = entry(32 + lane);
      for (int i = 0; i < sg.count; ++i, ++n) {
        const int j0 = i * boxes;
        if (i > 0 && j0 % 32 == 0) {
          cur = nxt;
          nxt = entry(j0 + 32 + lane);
        }
        const int s = n % kStages;
        if (!ptx::wait_bounded_warp(empty(s), ((n / kStages) & 1) ^ 1, abort_p, kWaitLimitNs)) {
          ok = false;
          break;
        }
        // lane x < boxes loads box x of this tile
        const int page = __shfl_sync(0xffffffffu, cur, (j0 + lane) % 32);
        const bool need = lane < boxes && needed(j0 + lane);
        const bool load = need && page >= 0 && page < a.num_pages;
        if (need && !load) record_page_error();
        const int r = row0 + (j0 + lane) * br;          // first token of this lane's box
        // visible tokens of the box, as bits of the tile's 64
        uint64_t m = 0;
        if (load) {
          const int x0 = max(t.lo - r, 0), x1 = min(t.hi - r, br);
          m = (x1 >= 64 ? ~0ull : (1ull << x1) - 1) & ~((1ull << x0) - 1);
          m <<= lane * br & 63;
        }
        const unsigned loads = __ballot_sync(0xffffffffu, load);
        uint32_t m_lo = static_cast<uint32_t>(m), m_hi = static_cast<uint32_t>(m >> 32);
        m_lo = __reduce_or_sync(0xffffffffu, m_lo);
        m_hi = __reduce_or_sync(0xffffffffu, m_hi);
        if (lane == 0) {
          masks[s] = static_cast<uint64_t>(m_hi) << 32 | m_lo;
          ptx::mbar_arrive_expect_tx(full(s), 2 * box_bytes * __popc(loads));
        }
        __syncwarp();
        if (load) {
          const uint32_t dst = base + s * L::kTileBytes + lane * box_bytes;
          const int row = r % a.page_size;
          tma_load_5d(dst + L::kK, &tm_k, full(s), 0, hk, row, 0, page);
          tma_load_5d(dst + L::kV, &tm_v, full(s), 0, hk, row, 0, page);
        }
      }
    }
    if (!ok && lane == 0) give_up();
    // Leave no copy in flight (on the normal path these phases completed long ago).
    for (int x = max(0, n - kStages); x < n; ++x)
      ptx::wait_bounded(full(x % kStages), (x / kStages) & 1, abort_p, kWaitLimitNs);
    if constexpr (SHORT) {   // the consumers' two meetings of the cluster
      __syncwarp();
      cg::this_cluster().sync();
      cg::this_cluster().sync();
    }
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int r0 = lane / 4, c0 = 2 * (lane % 4);   // this lane's rows r0, r0 + 8; columns c0, +1
  float* const join = reinterpret_cast<float*>(gen + L::kJoin);
  float* const sm_m = reinterpret_cast<float*>(gen + L::kStats);
  float* const sm_l = sm_m + kWarps * kRows;
  // this warp's 16 tokens of a tile: box and row within it
  const int br = a.box_rows;
  const uint32_t my_rows =
      (16 * warp / br) * static_cast<uint32_t>(br) * D * 2 + (16 * warp % br) * 128u;
  const uint32_t half_bytes = static_cast<uint32_t>(br) * 128;   // 64 columns of a box
  const int mi = lane / 8, l7 = lane % 8;          // ldmatrix: matrix and row of this lane
  float* const scores = reinterpret_cast<float*>(gen + L::kScores);   // SHORT: [16][kScorePitch]
  int n = 0, runs = 0;
  bool ok = true;
  for (; more(runs); ++runs) {
    Tiles t;
    const Segment sg = next(std::false_type{}, t);
    const int hk = sg.unit / a.blocks, h0 = (sg.unit % a.blocks) * kRows;
    const int rows = min(kRows, a.G - h0);
    const int64_t head0 = static_cast<int64_t>(sg.b) * a.Hq + hk * a.G + h0;   // row 0's (b, h)
    uint32_t qf[D / 16][4];
    {
      const uint16_t* q0 = static_cast<const uint16_t*>(a.q) + (head0 + r0) * D + c0;
      const uint16_t* q1 = q0 + 8 * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        auto ld = [](const uint16_t* p, bool in) {
          return in ? *reinterpret_cast<const uint32_t*>(p) : 0u;
        };
        qf[kk][0] = ld(q0 + kk * 16, r0 < rows);
        qf[kk][1] = ld(q1 + kk * 16, r0 + 8 < rows);
        qf[kk][2] = ld(q0 + kk * 16 + 8, r0 < rows);
        qf[kk][3] = ld(q1 + kk * 16 + 8, r0 + 8 < rows);
      }
    }
    float acc[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) acc[x][y] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int i = 0; i < sg.count; ++i, ++n) {
      const int s = n % kStages;
      // after a wait has run out the loop goes on without data, so that every warp reaches the
      // barriers below
      if (ok && !ptx::wait_bounded_warp(full(s), (n / kStages) & 1, abort_p, kWaitLimitNs)) {
        ok = false;
        if (lane == 0) give_up();
      }
      if (!ok) continue;
      const uint32_t mask = static_cast<uint32_t>(masks[s] >> (16 * warp)) & 0xffffu;
      if (mask) {
        const uint32_t kt = base + L::kK + s * L::kTileBytes + my_rows;
        const uint32_t vt = base + L::kV + s * L::kTileBytes + my_rows;
        // S = Q K^T for 16 tokens: two 8-token columns, two accumulator chains each
        float sc[2][2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) sc[0][x][y] = sc[1][x][y] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t kf[4];
          const int chunk = (kk % 4) * 2 + (mi & 1);
          ldsm_x4(kt + (kk / 4) * half_bytes + ((mi >> 1) * 8 + l7) * 128 + ((chunk ^ l7) << 4),
                  kf);
          mma<FP16>(sc[kk & 1][0], qf[kk], kf[0], kf[1]);
          mma<FP16>(sc[kk & 1][1], qf[kk], kf[2], kf[3]);
        }
        float sv[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) sv[x][y] = (sc[0][x][y] + sc[1][x][y]) * a.scale_log2;
        if (mask != 0xffffu) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (!(mask >> (8 * x + c0 + (y & 1)) & 1)) sv[x][y] = -INFINITY;
        }
        if constexpr (WEIGHTS && SHORT) {
          float* const at = scores + r0 * L::kScorePitch + i * kTile + 16 * warp + c0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            *reinterpret_cast<float2*>(at + 8 * x) = make_float2(sv[x][0], sv[x][1]);
            *reinterpret_cast<float2*>(at + 8 * L::kScorePitch + 8 * x) =
                make_float2(sv[x][2], sv[x][3]);
          }
        } else if constexpr (WEIGHTS) {
          const int token = (t.first + sg.tile + i) * kTile + 16 * warp + c0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (r0 < rows)
              *reinterpret_cast<float2*>(a.scores + (head0 + r0) * a.capacity + token + 8 * x) =
                  make_float2(sv[x][0], sv[x][1]);
            if (r0 + 8 < rows)
              *reinterpret_cast<float2*>(a.scores + (head0 + r0 + 8) * a.capacity + token +
                                         8 * x) = make_float2(sv[x][2], sv[x][3]);
          }
        }
        float x0 = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1]));
        float x1 = fmaxf(fmaxf(sv[0][2], sv[0][3]), fmaxf(sv[1][2], sv[1][3]));
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
        }
        if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
          const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
          const float f0 = ptx::exp2_approx(m0 - (n0 == -INFINITY ? 0.f : n0));
          const float f1 = ptx::exp2_approx(m1 - (n1 == -INFINITY ? 0.f : n1));
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            acc[x][0] *= f0;
            acc[x][1] *= f0;
            acc[x][2] *= f1;
            acc[x][3] *= f1;
          }
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        // (the shift comes after the difference: next to a large maximum it would be rounded)
        auto prob = [](float s, float u) { return ptx::exp2_approx((s - u) + kPShift<FP16>); };
        float p[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          p[x][0] = prob(sv[x][0], u0);
          p[x][1] = prob(sv[x][1], u0);
          p[x][2] = prob(sv[x][2], u1);
          p[x][3] = prob(sv[x][3], u1);
        }
        l0 += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        l1 += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
        uint32_t ph[4], pl[4];
        split2<FP16>(p[0][0], p[0][1], ph[0], pl[0]);
        split2<FP16>(p[0][2], p[0][3], ph[1], pl[1]);
        split2<FP16>(p[1][0], p[1][1], ph[2], pl[2]);
        split2<FP16>(p[1][2], p[1][3], ph[3], pl[3]);
        // rows of V that are not visible may hold anything, NaN included: they count as zeros
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (mask != 0xffffu) {
          keep0 = (mask >> c0 & 1 ? 0xffffu : 0u) | (mask >> (c0 + 1) & 1 ? 0xffff0000u : 0u);
          keep1 = (mask >> (8 + c0) & 1 ? 0xffffu : 0u) |
                  (mask >> (9 + c0) & 1 ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t vf[4];
          const int chunk = (x % 4) * 2 + (mi >> 1);
          ldsm_x4_trans(
              vt + (x / 4) * half_bytes + ((mi & 1) * 8 + l7) * 128 + ((chunk ^ l7) << 4), vf);
          vf[0] &= keep0;
          vf[1] &= keep1;
          vf[2] &= keep0;
          vf[3] &= keep1;
          mma<FP16>(acc[2 * x], ph, vf[0], vf[1]);
          mma<FP16>(acc[2 * x + 1], ph, vf[2], vf[3]);
          // the rest may be zero or negative: an infinite value counts in the first product alone
#pragma unroll
          for (int y = 0; y < 4; ++y) vf[y] = finite2<FP16>(vf[y]);
          mma<FP16>(acc[2 * x], pl, vf[0], vf[1]);
          mma<FP16>(acc[2 * x + 1], pl, vf[2], vf[3]);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty(s));
    }

    // ---- join the four warps
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (lane % 4 == 0) {
      sm_m[warp * kRows + r0] = m0;
      sm_m[warp * kRows + r0 + 8] = m1;
      sm_l[warp * kRows + r0] = l0 * kPUnshift<FP16>;
      sm_l[warp * kRows + r0 + 8] = l1 * kPUnshift<FP16>;
    }
    ptx::named_barrier_sync(1, 32 * kWarps);
    auto row_stats = [&](int r, float& m, float& l) {
      m = -INFINITY;
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w * kRows + r]);
      l = 0.f;
      const float u = m == -INFINITY ? 0.f : m;
      for (int w = 0; w < kWarps; ++w)
        l += sm_l[w * kRows + r] * ptx::exp2_approx(sm_m[w * kRows + r] - u);
    };
    const int64_t slot = 2ll * cta + (runs > 0);
    float* const part = reinterpret_cast<float*>(gen + L::kPart);
    float2* const part_ml = reinterpret_cast<float2*>(gen + L::kPartMl);
    if (!SHORT && sg.tile == 0 && threadIdx.x == 0) {
      // this run holds the unit's first tile; its last is in the last run that starts before
      // the unit's end: the largest c with floor(total * c / ctas) < end
      const int ctas = running(s_total, gridDim.x);
      const int64_t end = s_start + n - sg.count + t.count;
      const int last = static_cast<int>((end * ctas - 1) / s_total);
      a.units[static_cast<int64_t>(sg.b) * a.Hkv * a.blocks + sg.unit] =
          make_int2(static_cast<int>(slot), sg.whole ? 0 : last - cta + 1);
    }
    if (threadIdx.x < kRows) {
      float m, l;
      row_stats(threadIdx.x, m, l);
      if constexpr (SHORT) {
        part_ml[threadIdx.x] = make_float2(m, l);
      } else if (static_cast<int>(threadIdx.x) >= rows) {
        // a row without a query head
      } else if (!sg.whole) {
        a.part_ml[slot * a.part_rows + threadIdx.x] = make_float2(m, l);
      } else {
        a.lse[head0 + threadIdx.x] = lse_of(m, l);
        if constexpr (WEIGHTS) a.stats[head0 + threadIdx.x] = make_float2(m, inverse(l));
      }
    }
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      if (rh * 8 >= rows) break;
      float m, l;
      row_stats(r0 + 8 * rh, m, l);
      const float f =
          ptx::exp2_approx((rh ? m1 : m0) - (m == -INFINITY ? 0.f : m)) * kPUnshift<FP16>;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<float2*>(join + (warp * 8 + r0) * L::kJoinPitch + 8 * x + c0) =
              make_float2(acc[ch * 8 + x][2 * rh] * f, acc[ch * 8 + x][2 * rh + 1] * f);
        ptx::named_barrier_sync(1, 32 * kWarps);
        // thread t: row t / 16 of the eight, four columns
        const int r = threadIdx.x / 16, c = threadIdx.x % 16 * 4, row = rh * 8 + r;
        if (row < rows) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v =
                *reinterpret_cast<const float4*>(join + (w * 8 + r) * L::kJoinPitch + c);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
          if constexpr (SHORT) {
            *reinterpret_cast<float4*>(part + row * D + ch * 64 + c) = sum;
          } else if (!sg.whole) {
            *reinterpret_cast<float4*>(a.part_o + (slot * a.part_rows + row) * D + ch * 64 + c) = sum;
          } else {
            float mr, lr;
            row_stats(row, mr, lr);
            const float inv = inverse(lr);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (head0 + row) * D + ch * 64 +
                                      c) = make_uint2(pack2<FP16>(sum.x * inv, sum.y * inv),
                                                      pack2<FP16>(sum.z * inv, sum.w * inv));
          }
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
      }
    }
    if constexpr (SHORT) {
      const cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();   // every CTA's part is in its shared memory
      const int tid = threadIdx.x;
      // four columns of a row a thread, the rows shared out over the cluster
      for (int at = rank * 32 * kWarps + tid; at < rows * (D / 4); at += ranks * 32 * kWarps) {
        const int row = at / (D / 4), x = at % (D / 4);
        float m = -INFINITY, l = 0.f;
        float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r >= ranks) break;
          const float2 ml = *cluster.map_shared_rank(part_ml + row, r);
          const float4 v =
              *reinterpret_cast<const float4*>(cluster.map_shared_rank(part + row * D + 4 * x, r));
          const float top = fmaxf(m, ml.x), u = top == -INFINITY ? 0.f : top;
          const float f = ptx::exp2_approx(m - u), g = ptx::exp2_approx(ml.x - u);
          m = top;
          l = l * f + ml.y * g;
          acc4.x = acc4.x * f + v.x * g;
          acc4.y = acc4.y * f + v.y * g;
          acc4.z = acc4.z * f + v.z * g;
          acc4.w = acc4.w * f + v.w * g;
        }
        const float inv = inverse(l);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (head0 + row) * D + 4 * x) =
            make_uint2(pack2<FP16>(acc4.x * inv, acc4.y * inv),
                       pack2<FP16>(acc4.z * inv, acc4.w * inv));
        if (x == 0) a.lse[head0 + row] = lse_of(m, l);
      }
      if constexpr (WEIGHTS) {
        // maximum and 1 / sum of every row (where the warps' statistics were), then the tokens of
        // this CTA's tiles: the bits of a tile's mask are its visible tokens in good pages
        float2* const stat = reinterpret_cast<float2*>(gen + L::kStats);
        if (tid < rows) {
          float m = -INFINITY, l = 0.f;
          for (int r = 0; r < ranks; ++r) m = fmaxf(m, cluster.map_shared_rank(part_ml + tid, r)->x);
          const float u = m == -INFINITY ? 0.f : m;
          for (int r = 0; r < ranks; ++r) {
            const float2 ml = *cluster.map_shared_rank(part_ml + tid, r);
            l += ml.y * ptx::exp2_approx(ml.x - u);
          }
          stat[tid] = make_float2(u, inverse(l));
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
        for (int at = tid; ok && at < sg.count * kTile; at += 32 * kWarps) {
          if (!(masks[at / kTile] >> (at % kTile) & 1)) continue;
          float sum = 0.f;
          for (int row = 0; row < rows; ++row)
            sum += ptx::exp2_approx(scores[row * L::kScorePitch + at] - stat[row].x) * stat[row].y;
          const int token = (t.first + sg.tile) * kTile + at;
          const int64_t page =
              a.table[static_cast<int64_t>(sg.b) * a.max_pages + token / a.page_size];
          ptx::red_add_f32(a.weights + (page * a.Hkv + hk) * a.page_size + token % a.page_size,
                           sum);
        }
      }
      cluster.sync();   // no CTA leaves while another reads its part
    }
  }
}

// After the runs, in one launch: blocks [0, B * Hq) join the parts of a query head whose unit
// more than one run covers; with weights, the blocks behind them add the probabilities to the
// weights, 1024 tokens of a (sequence, key head) each. These need every head's final maximum and
// sum, and join those (not O) themselves instead of waiting for the others.
constexpr int kFinishThreads = 256;

// Maximum (log2 units) and sum of row `row` of a unit of `info` parts, by one warp (every lane
// gets them). The part in the first run's slot is followed by those of the next CTAs, each in
// its CTA's first slot.
__device__ __forceinline__ int part_slot(int2 info, int p) {
  return p == 0 ? info.x : 2 * (info.x / 2 + p);
}
__device__ __forceinline__ float2 join_stats(const Args& a, int2 info, int row) {
  const int lane = threadIdx.x % 32;
  float m = -INFINITY, l = 0.f;
  for (int p = lane; p < info.y; p += 32)
    m = fmaxf(m, a.part_ml[static_cast<int64_t>(part_slot(info, p)) * a.part_rows + row].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float u = m == -INFINITY ? 0.f : m;
  for (int p = lane; p < info.y; p += 32) {
    const float2 ml = a.part_ml[static_cast<int64_t>(part_slot(info, p)) * a.part_rows + row];
    l += ml.y * ptx::exp2_approx(ml.x - u);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  return make_float2(m, l);
}
__device__ __forceinline__ int2 unit_info(const Args& a, int b, int h) {
  const int unit = h / a.G * a.blocks + h % a.G / kRows;
  return a.units[static_cast<int64_t>(b) * a.Hkv * a.blocks + unit];
}

// O and LSE of a head from its parts. A thread has four columns of every kSets-th part and a
// running maximum of its own, so that statistics and O of the parts are loaded together.
template <int D, bool FP16>
__device__ __forceinline__ void join_head(const Args& a, int64_t head) {
  constexpr int kLanes = D / 4, kSets = kFinishThreads / kLanes;
  __shared__ float4 s_acc[kSets][kLanes];
  __shared__ float2 s_ml[kSets];
  const int b = static_cast<int>(head / a.Hq), h = static_cast<int>(head % a.Hq);
  const int row = h % a.G % kRows;
  const int2 info = unit_info(a, b, h);
  if (info.y == 0) return;   // one run covered the unit: written already
  const int set = threadIdx.x / kLanes, x = threadIdx.x % kLanes;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int p = set; p < info.y; p += kSets) {
    const int64_t at = static_cast<int64_t>(part_slot(info, p)) * a.part_rows + row;
    const float2 ml = a.part_ml[at];
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * D + 4 * x);
    const float n = fmaxf(m, ml.x), u = n == -INFINITY ? 0.f : n;
    const float f = ptx::exp2_approx(m - u), g = ptx::exp2_approx(ml.x - u);
    m = n;
    l = l * f + ml.y * g;
    acc.x = acc.x * f + v.x * g;
    acc.y = acc.y * f + v.y * g;
    acc.z = acc.z * f + v.z * g;
    acc.w = acc.w * f + v.w * g;
  }
  s_acc[set][x] = acc;
  if (x == 0) s_ml[set] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  m = -INFINITY;
#pragma unroll
  for (int y = 0; y < kSets; ++y) m = fmaxf(m, s_ml[y].x);
  const float u = m == -INFINITY ? 0.f : m;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int y = 0; y < kSets; ++y) {
    const float f = ptx::exp2_approx(s_ml[y].x - u);
    const float4 v = s_acc[y][x];
    l += s_ml[y].y * f;
    acc.x += v.x * f;
    acc.y += v.y * f;
    acc.z += v.z * f;
    acc.w += v.w * f;
  }
  const float inv = inverse(l);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + head * D + 4 * x) = make_uint2(
      pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
  if (x == 0) a.lse[head] = lse_of(m, l);
}

// weights[page, hk, row] += sum over the group's heads of 2^(score - maximum) / sum. Four
// tokens a thread (one 16-byte load of each head's scores). Every weight gets one addition from
// each sequence that holds its page, as an atomic so that sequences may share pages; where none
// does the result has one order only.
__device__ __forceinline__ void add_weights(const Args& a, int64_t unit, int chunk) {
  constexpr int kHeads = 64;
  __shared__ float2 s_stat[kHeads];   // maximum and 1 / sum
  const int b = static_cast<int>(unit / a.Hkv), hk = static_cast<int>(unit % a.Hkv);
  const Visible v = visible_tokens<false>(a.seqlens, b, a.capacity, a.window_left);
  const int first = (v.lo / 4 + chunk * kFinishThreads) * 4;
  if (first >= v.hi) return;
  const int t0 = first + static_cast<int>(threadIdx.x) * 4;
  const int page = t0 < v.hi ? a.table[static_cast<int64_t>(b) * a.max_pages + t0 / a.page_size]
                             : -1;
  const bool in = page >= 0 && page < a.num_pages;   // a bad page was recorded by the runs
  const int64_t head0 = static_cast<int64_t>(b) * a.Hq + hk * a.G;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int g0 = 0; g0 < a.G; g0 += kHeads) {
    const int heads = min(kHeads, a.G - g0);
    for (int g = threadIdx.x / 32; g < heads; g += kFinishThreads / 32) {
      const int h = hk * a.G + g0 + g;
      const int2 info = unit_info(a, b, h);
      float2 st;
      if (info.y == 0) {
        st = a.stats[static_cast<int64_t>(b) * a.Hq + h];
      } else {
        st = join_stats(a, info, (g0 + g) % kRows);
        st.y = inverse(st.y);
      }
      if (threadIdx.x % 32 == 0) s_stat[g] = make_float2(st.x == -INFINITY ? 0.f : st.x, st.y);
    }
    __syncthreads();
    if (in) {
#pragma unroll 4
      for (int g = 0; g < heads; ++g) {
        const float4 s =
            *reinterpret_cast<const float4*>(a.scores + (head0 + g0 + g) * a.capacity + t0);
        const float2 st = s_stat[g];
        sum.x += ptx::exp2_approx(s.x - st.x) * st.y;
        sum.y += ptx::exp2_approx(s.y - st.x) * st.y;
        sum.z += ptx::exp2_approx(s.z - st.x) * st.y;
        sum.w += ptx::exp2_approx(s.w - st.x) * st.y;
      }
    }
    __syncthreads();
  }
  if (!in) return;
  float* w = a.weights + (static_cast<int64_t>(page) * a.Hkv + hk) * a.page_size +
             t0 % a.page_size;
  if (t0 >= v.lo && t0 + 4 <= v.hi) {
    ptx::red_add_v4(w, sum.x, sum.y, sum.z, sum.w);
  } else {
    const float each[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + i >= v.lo && t0 + i < v.hi) ptx::red_add_f32(w + i, each[i]);
  }
}

template <int D, bool FP16, bool WEIGHTS>
__global__ void __launch_bounds__(kFinishThreads)
    fa_paged_finish_kernel(const __grid_constant__ Args a, int64_t heads, int chunks) {
  wait_prerequisites();
  launch_dependents();
  const int64_t at = blockIdx.x;
  if (at < heads)
    join_head<D, FP16>(a, at);
  else if constexpr (WEIGHTS)
    add_weights(a, (at - heads) / chunks, static_cast<int>((at - heads) % chunks));
}

// k_pages or v_pages as a 5-D TMA map: 64 columns, head, row of the page, 64-column half, page.
// A box is box_rows rows of one page and head with all their columns, half by half.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode_pages(CUtensorMap* map, void* pages, const PagedCache& c, int box_rows, bool fp16) {
  const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(encode_tiled_entry());
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.Hkv) * c.d * 2;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(c.Hkv),
                              static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.d / 64),
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(c.d) * 2, row, 128, row * c.page_size};
  const cuuint32_t box[5] = {64, 1, static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(c.d / 64), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            pages, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs for a call: two on each SM, or one for each tile where there are fewer.
int64_t grid_size(int B, int Hq, int Hkv, int64_t capacity) {
  const int64_t blocks = (Hq / Hkv + kRows - 1) / kRows;
  const int64_t tiles = B * Hkv * blocks * ((capacity + kTile - 1) / kTile);
  return std::min<int64_t>(kMaxCtas, tiles);
}

// Clusters of `ctas` CTAs of a short call that run at once. A CTA's shared memory leaves room for
// one on each SM at d = 128, two at d = 64; a cluster has to lie within one of the groups of SMs
// that the GPU is made of, so that the larger ones leave SMs over (as the runtime's occupancy
// query counts them on a GB300).
int resident_clusters(int ctas, int d) {
  const bool small = d == 64;
  switch (ctas) {
    case 8: return small ? 36 : 15;
    case 4: return small ? 74 : 36;
    case 2: return small ? 152 : 76;
    default: return small ? 304 : 152;
  }
}

// The smallest calls: 0, or the CTAs of a cluster that has one unit. Where every unit fits in a
// cluster of CTAs with up to kShortTiles tiles each, and all of them run at once, one launch
// without a workspace is faster than runs and their join: B=1 Hkv=8 d=64 with 1001 tokens 8.3 us
// instead of 10.3 a replay of a graph, 19 us instead of 26 a call from Python, which has no
// workspace to allocate. Units of one CTA may take a second turn, each turn a single round trip to
// memory: 240 units of 250 tokens (d=64, 4 heads on a key head) 6.4 us instead of 11.3 a replay,
// 560 units 12.5 instead of 16.7; at d=128 296 units 12.3 instead of 13.5, but a third and a
// fourth turn of 560 units of 100 tokens cost 18.0 instead of 15.6. Clusters get no second turn:
// 16 units of 2000 tokens, d=128, take 21.0 us in two turns of clusters of eight and 18.9 as runs
// (15 units in one turn 14.9), 37 units of 1000 tokens 21.0 in clusters of four and 18.9 as runs.
// With weights the query heads of a key head have to be one unit, so that every weight gets one
// addition.
int choose_short(int B, int Hq, int Hkv, int d, int64_t tiles, bool with_weights) {
  const int64_t blocks = (Hq / Hkv + kRows - 1) / kRows, units = B * Hkv * blocks;
  if (with_weights && blocks > 1) return 0;
  for (int ctas = kMaxCluster; ctas >= 2; ctas /= 2)
    if (units <= resident_clusters(ctas, d) && ctas / 2 < tiles)
      return tiles <= ctas * kShortTiles ? ctas : 0;
  return units <= 2 * resident_clusters(1, d) && tiles <= kShortTiles ? 1 : 0;
}

// Workspace: the parts' O, their maxima and sums, the units' parts, then (with weights)
// statistics and scores.
struct Layout {
  size_t part_ml, units, stats, scores, end;
};
Layout layout(int B, int Hq, int Hkv, int d, int64_t capacity, bool with_weights) {
  const size_t slots = 2 * static_cast<size_t>(grid_size(B, Hq, Hkv, capacity));
  Layout l;
  const size_t rows = std::min(Hq / Hkv, kRows);
  l.part_ml = slots * rows * d * 4;
  l.units = l.part_ml + slots * rows * 8;
  const size_t blocks = (Hq / Hkv + kRows - 1) / kRows;
  l.stats = l.units + static_cast<size_t>(B) * Hkv * blocks * 8;
  const size_t heads = static_cast<size_t>(B) * Hq;
  l.scores = (l.stats + (with_weights ? heads * 8 : 0) + 15) / 16 * 16;
  l.end = l.scores + (with_weights ? heads * capacity * 4 : 0);
  return l;
}

template <int D, bool FP16, bool WEIGHTS>
cudaError_t launch_impl(const DecodeParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  Args a;
  a.q = p.q;
  a.table = c.block_table;
  a.seqlens = c.seqlens;
  a.o = p.o;
  a.lse = p.lse;
  a.weights = c.weights;
  a.capacity = c.max_pages * c.page_size;
  const Layout l = layout(c.B, p.Hq, c.Hkv, D, a.capacity, WEIGHTS);
  char* ws = static_cast<char*>(p.workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  a.units = reinterpret_cast<int2*>(ws + l.units);
  a.stats = reinterpret_cast<float2*>(ws + l.stats);
  a.scores = reinterpret_cast<float*>(ws + l.scores);
  a.B = c.B;
  a.Hq = p.Hq;
  a.Hkv = c.Hkv;
  a.G = p.Hq / c.Hkv;
  a.blocks = (a.G + kRows - 1) / kRows;
  a.part_rows = std::min(a.G, kRows);
  a.page_size = c.page_size;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.box_rows = std::min(c.page_size, kTile);
  a.window_left = p.window_left;
  a.scale_log2 = p.scale_log2;
  CUtensorMap tm_k, tm_v;
  if (!encode_pages(&tm_k, c.k_pages, c, a.box_rows, FP16) ||
      !encode_pages(&tm_v, c.v_pages, c, a.box_rows, FP16))
    return cudaErrorInvalidValue;
  // tiles of a unit, at most: a window's tokens span two more tiles than its length fills
  int64_t tiles = (static_cast<int64_t>(a.capacity) + kTile - 1) / kTile;
  if (a.window_left >= 0) tiles = std::min<int64_t>(tiles, a.window_left / kTile + 2);
  if (const int cluster = choose_short(c.B, p.Hq, c.Hkv, D, tiles, WEIGHTS)) {
    auto kernel = fa_paged_decode_kernel<D, FP16, WEIGHTS, true>;
    const int smem = static_cast<int>(Smem<D, true>::kDynamic);
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    return launch_chained(kernel, static_cast<int64_t>(c.B) * c.Hkv * a.blocks * cluster, kThreads,
                          smem, stream, cluster, tm_k, tm_v, a);
  }
  auto kernel = fa_paged_decode_kernel<D, FP16, WEIGHTS, false>;
  const int smem = static_cast<int>(Smem<D, false>::kDynamic);
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const int ctas = static_cast<int>(grid_size(c.B, p.Hq, c.Hkv, a.capacity));
  err = launch_chained(kernel, ctas, kThreads, smem, stream, 0, tm_k, tm_v, a);
  if (err != cudaSuccess) return err;
  // units of one tile are never split: no head to join
  const int64_t heads = a.capacity > kTile ? static_cast<int64_t>(c.B) * p.Hq : 0;
  int64_t blocks = heads;
  int chunks = 1;
  if (WEIGHTS) {
    // a window's tokens span at most window_left + 1, from a multiple of 4
    int64_t span = a.capacity;
    if (a.window_left >= 0) span = std::min<int64_t>(span, static_cast<int64_t>(a.window_left) + 4);
    chunks = static_cast<int>((span + 4 * kFinishThreads - 1) / (4 * kFinishThreads));
    blocks += static_cast<int64_t>(c.B) * c.Hkv * chunks;
  }
  if (blocks == 0) return cudaSuccess;
  return launch_chained(fa_paged_finish_kernel<D, FP16, WEIGHTS>, blocks, kFinishThreads, 0, stream,
                        0, a, heads, chunks);
}

template <int D, bool FP16>
cudaError_t launch_weights(const DecodeParams& p, cudaStream_t stream) {
  return p.c.weights ? launch_impl<D, FP16, true>(p, stream)
                     : launch_impl<D, FP16, false>(p, stream);
}

}  // namespace

size_t paged_decode_workspace(int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                              bool with_weights) {
  const int64_t capacity = static_cast<int64_t>(max_pages) * page_size;
  if (choose_short(B, Hq, Hkv, d, (capacity + kTile - 1) / kTile, with_weights)) return 0;
  return layout(B, Hq, Hkv, d, capacity, with_weights).end;
}

cudaError_t launch_paged_decode(const DecodeParams& p, cudaStream_t stream) {
  if (p.c.d == 64)
    return p.fp16 ? launch_weights<64, true>(p, stream) : launch_weights<64, false>(p, stream);
  return p.fp16 ? launch_weights<128, true>(p, stream) : launch_weights<128, false>(p, stream);
}

cudaError_t read_and_clear_decode_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
