// fa_paged_tree.cu -- attention of drafted tokens over a paged key-value cache: each sees its
// sequence's context, its ancestors in the draft's tree and itself (include/fa.h).
//
//   s_ij = scale <q_i, k_j>,  O_i = sum_j e^{s_ij - LSE_i} v_j,  LSE_i = ln sum_j e^{s_ij}
//
// What bounds it: K and V are read once, 4 d bytes a token and key head, for 4 d operations of
// each row -- a drafted token and one of the G query heads that share the key head. Up to about
// 250 rows HBM is the bound, from there the tensor cores; both products run on tcgen05 with 128 rows
// to a tile, whatever their number, so that a tile of K and V costs the same time for 2 rows as for
// 128 and less than its way from HBM.
//
// Rows of a (sequence, key head) are taken in the order (token, query head), in blocks of 128 (one
// row tile) or 256 (two). A block over its keys is a unit. The keys are cut into tiles of 128
// tokens, and the tiles of all units, in order, into one equal run for each CTA (one on each SM),
// whatever the lengths are. A run that covers a whole unit writes O and LSE; one that covers a part
// leaves the part's maximum, sum and unnormalised O (fp32) in the workspace, and a second kernel
// joins the parts of a unit in a fixed order.
//
// One CTA:
//   warp 0       TMA producer: K and V tiles into two rings, box by box of a page's rows
//   warp 1       TMEM allocator and MMA issuer (one thread)
//   warps 4..11  two softmax groups, A and B, a row to a thread: S from TMEM, P back over it,
//                O rescaled in TMEM when the maximum has grown; Q into shared memory at a unit's
//                start, O out of TMEM at its end
// Two row tiles: A has the first 128 rows, B the others; both see every tile. One row tile: A takes
// the even tiles of a run's part of a unit and B the odd ones, each with a maximum, sum and O of its
// own, joined at the end; so there, too, one group's softmax runs beside the other's products.
//
// Masks. Tiles of the context that no window cuts need none. In the others a thread builds the
// 128 bits of its row: a range of the context, and the ancestors by walking up the tree. Keys that
// some row of the tile does not see have P = 0 there, but 0 times a NaN or an infinity would not
// be 0: in such tiles group A (the tile's group) first replaces what is not finite in V by 0, and
// rows of tokens that do not exist or were not loaded as well; where it found any, the unit's end
// adds them to the rows that do see them.
//
// P is rounded to the type once for the product with V, a rounding of the same size as the
// output's. fp16 ends at 2^-24, so there P is taken 2^11 times as large, and up to 2^4 more until
// a grown maximum moves the offset: what is lost are probabilities below 2^-36 of the largest.
#include <algorithm>
#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;

constexpr int kTile = 128;                     // tokens of a tile, and rows of a row tile
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = 128 + kSoftmaxThreads;
constexpr int kSms = 152;                      // of a GB300; on another count only speed differs
constexpr uint32_t kHalfBytes = kTile * 64 * 2;   // 128 rows of 64 columns
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kInfoSlots = 8;                  // more than the tiles between a load and its softmax

// The offset of a row's exponents is its maximum less kShift, and moves when the maximum has
// grown by more than kLag (log2 units).
template <bool FP16>
constexpr float kShift = FP16 ? 11.f : 0.f;
template <bool FP16>
constexpr float kLag = FP16 ? 4.f : 8.f;

template <int D, int QT>
struct Smem {
  static constexpr int kStages = QT == 2 && D == 128 ? 2 : 3;
  static constexpr uint32_t kTileBytes = (D / 64) * kHalfBytes;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + QT * kTileBytes;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  static constexpr uint32_t kInfo = kV + kStages * kTileBytes;      // uint4: the tile's loaded keys
  static constexpr uint32_t kBars = kInfo + kInfoSlots * 16;
  static constexpr uint32_t kEnd = kBars + 32 * 8;
  static constexpr uint32_t kDynamic = kEnd + 1024;   // slack for 1 KiB alignment
};
static_assert(Smem<128, 1>::kDynamic + 1300 <= 232448, "with the static shared memory");

struct Args {
  const void* q;
  const int* table;
  const int* seqlens;
  const int* parents;
  const int* new_lens;
  const void* v_pages;
  void* o;
  float* lse;
  float* part_o;      // [2 * CTAs][part_rows][D]: CTA c's first run at slot 2c, its last at 2c + 1
  float2* part_ml;    // [2 * CTAs][part_rows]: offset (log2 units) and sum of the part
  int2* units;        // [B * Hkv * blocks]: slot of the unit's first part, number of parts (0: the
                      // unit was one run's, and is written)
  int B, T, Hq, Hkv, G, blocks;   // blocks of rows for each key head
  int part_rows;                  // rows of a unit, at most
  int page_shift, num_pages, max_pages, box_rows, window_left;
  float scale_log2;
};

// A block of rows: tokens [i0, i1) (i1 <= i0: only rows of the padding) and tiles
// [first, first + count), at least one.
struct Unit {
  int i0, i1, first, count;
};
template <int ROWS>
__device__ __forceinline__ Unit unit_of(const Args& a, Draft dr, int rb) {
  Unit u;
  u.i0 = rb * ROWS / a.G;
  u.i1 = min(dr.count, ((rb + 1) * ROWS + a.G - 1) / a.G);
  u.first = 0;
  u.count = 1;
  if (u.i1 > u.i0) {
    // the first key of the row that stands first (a tree's tokens may all be next to the context)
    const int lo = a.window_left < 0 ? 0
                   : max(0, dr.base + (a.parents ? 0 : u.i0) - a.window_left);
    u.first = lo / kTile;
    u.count = (dr.base + u.i1 - 1) / kTile + 1 - u.first;
  }
  return u;
}
__device__ __forceinline__ Draft draft(const Args& a, int b) {
  return draft_of(a.seqlens, a.new_lens, b, a.T, a.max_pages << a.page_shift);
}
// Tiles of all row blocks of a key head of sequence b.
template <int ROWS>
__device__ __forceinline__ int64_t head_tiles(const Args& a, int b) {
  const Draft dr = draft(a, b);
  int64_t n = 0;
  for (int rb = 0; rb < a.blocks; ++rb) n += unit_of<ROWS>(a, dr, rb).count;
  return n;
}

// A run as its segments: consecutive tiles of one unit.
struct Segment {
  Draft dr;
  Unit u;
  int b, hk, rb, tile, count;   // first tile within the unit's, tiles
  bool whole, empty;
};
struct Walk {
  int64_t left;    // tiles of the run that are left
  int b, hk, rb;
  int tile;        // within the unit
};
template <int ROWS>
__device__ __forceinline__ Segment next_segment(const Args& a, Walk& w) {
  Segment s;
  s.dr = draft(a, w.b);
  s.u = unit_of<ROWS>(a, s.dr, w.rb);
  s.b = w.b;
  s.hk = w.hk;
  s.rb = w.rb;
  s.tile = w.tile;
  s.count = static_cast<int>(min(static_cast<int64_t>(s.u.count - w.tile), w.left));
  s.whole = s.count == s.u.count;
  s.empty = s.u.i1 <= s.u.i0;
  w.left -= s.count;
  w.tile += s.count;
  if (w.tile == s.u.count) {
    w.tile = 0;
    if (++w.rb == a.blocks) {
      w.rb = 0;
      if (++w.hk == a.Hkv) {
        w.hk = 0;
        ++w.b;
      }
    }
  }
  return s;
}

// Barrier slots.
constexpr int kMaxStages = 3;
enum : int {
  BAR_K_FULL = 0,                          // + stage
  BAR_K_EMPTY = BAR_K_FULL + kMaxStages,   // + stage
  BAR_V_FULL = BAR_K_EMPTY + kMaxStages,   // + stage
  BAR_V_EMPTY = BAR_V_FULL + kMaxStages,   // + stage
  BAR_INFO = BAR_V_EMPTY + kMaxStages,     // + slot: the tile's loaded keys are in kInfo
  BAR_S_FULL = BAR_INFO + kInfoSlots,      // + group: S computed
  BAR_P_FULL = BAR_S_FULL + 2,             // + group: P in TMEM, O rescaled, V cleaned (128)
  BAR_O_DONE = BAR_P_FULL + 2,             // + group: P V computed
  BAR_Q_FULL = BAR_O_DONE + 2,             // Q of the segment in shared memory (256)
  BAR_O_FREE = BAR_Q_FULL + 1,             // O of the segment out of TMEM (256)
  BAR_MMA_DONE = BAR_O_FREE + 1,
  BAR_COUNT = BAR_MMA_DONE + 1
};
static_assert(BAR_COUNT <= 32, "barrier slots");

// Bits [lo, hi) of 32, for any lo and hi.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1;
  return below_hi & ~below_lo;
}

// Parent of drafted token i of sequence b, -1 for the context and (recorded) for what is no
// earlier token.
__device__ __forceinline__ int parent_of(const Args& a, int b, int i) {
  const int up = a.parents[static_cast<int64_t>(b) * a.T + i];
  if (up >= -1 && up < i) return up;
  record_page_error();
  return -1;
}

// A row's token: what it sees.
struct Row {
  int b, i;        // i < 0: no token
  int lo;          // its first key of the context (window)
};
// Keys k0 .. k0 + 127 that the row sees, as bits.
__device__ __forceinline__ void visible_bits(const Args& a, const Row& r, int base, int k0,
                                             uint32_t (&vis)[4]) {
  const int hi = a.parents ? base : base + r.i + 1;   // a chain's keys are a range, too
#pragma unroll
  for (int w = 0; w < 4; ++w)
    vis[w] = r.i < 0 ? 0u : bit_range(r.lo - k0 - 32 * w, hi - k0 - 32 * w);
  if (a.parents && r.i >= 0 && k0 + kTile > base) {
    int steps = 0;
    for (int at = r.i; at >= 0 && base + at >= k0; at = parent_of(a, r.b, at), ++steps) {
      if (a.window_left >= 0 && steps > a.window_left) break;
      const int t = base + at - k0;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (t >> 5 == w) vis[w] |= 1u << (t & 31);
    }
  }
}

// Halves of v that are infinite or NaN, as ones.
template <bool FP16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t v) {
  constexpr uint32_t kExp = FP16 ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpeq2(v & kExp, kExp);
}

template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (FP16)
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// The rare end of a segment in whose masked tiles V was not finite: those values, which the
// products have taken as 0, added to the thread's row (fp32 part or output, columns [c0, c0 + cols))
// for the keys that it sees.
template <bool FP16>
__device__ __noinline__ void add_not_finite(const Args& a, const Row& rw, int base, int hk, int d,
                                            int first_key, int tiles, int full_lo, int full_hi,
                                            int c0, int cols, float* part, uint16_t* out) {
  const int* const tab = a.table + static_cast<int64_t>(rw.b) * a.max_pages;
  for (int j = 0; j < tiles; ++j) {
    const int k0 = first_key + j * kTile;
    bool masked = k0 < full_lo || k0 + kTile > full_hi;
    for (int t = k0; t < k0 + kTile && !masked; t += a.box_rows) {   // all within [0, full_hi)
      const int page = tab[t >> a.page_shift];
      masked = page < 0 || page >= a.num_pages;
    }
    if (!masked) continue;
    uint32_t vis[4];
    visible_bits(a, rw, base, k0, vis);
    for (int t = 0; t < kTile; ++t) {
      const uint32_t word = t < 64 ? (t < 32 ? vis[0] : vis[1]) : (t < 96 ? vis[2] : vis[3]);
      if (!(word >> (t % 32) & 1)) continue;
      const int page = tab[(k0 + t) >> a.page_shift];
      if (page < 0 || page >= a.num_pages) continue;
      const int64_t at = (static_cast<int64_t>(page) << a.page_shift) +
                         ((k0 + t) & ((1 << a.page_shift) - 1));
      const uint32_t* const src = reinterpret_cast<const uint32_t*>(
          static_cast<const uint16_t*>(a.v_pages) + (at * a.Hkv + hk) * d + c0);
      for (int c = 0; c < cols; c += 2) {
        const uint32_t w = src[c / 2];
        if (!not_finite2<FP16>(w)) continue;
        const float2 f = unpack2<FP16>(w);
        const float fx = isfinite(f.x) ? 0.f : f.x, fy = isfinite(f.y) ? 0.f : f.y;
        if (part) {
          part[c0 + c] += fx;
          part[c0 + c + 1] += fy;
        } else {
          uint32_t* const to = reinterpret_cast<uint32_t*>(out + c0 + c);
          const float2 o = unpack2<FP16>(*to);
          *to = pack2<FP16>(o.x + fx, o.y + fy);
        }
      }
    }
  }
}

template <int D, bool FP16, int QT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_tree_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Args a) {
  using L = Smem<D, QT>;
  constexpr int kStages = L::kStages, kRows = QT * kTile;
  constexpr uint32_t kTmemO = 2 * kTile, kTmemCols = 512;   // S_A, S_B, O_A, O_B
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag, s_not_finite;    // segment (+ 1) whose masked tiles had such values
  __shared__ float2 s_ml[kTile];              // one row tile: a group's offsets and sums
  __shared__ int64_t s_left, s_start, s_total;
  __shared__ int s_at[4];
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gen = smem_raw + (base - ptx::smem_addr(smem_raw));
  auto bar = [&](int i) { return base + L::kBars + 8u * static_cast<uint32_t>(i); };
  uint4* const info = reinterpret_cast<uint4*>(gen + L::kInfo);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    s_not_finite = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(BAR_K_FULL + s), 1);
      ptx::mbar_init(bar(BAR_K_EMPTY + s), 1);
      ptx::mbar_init(bar(BAR_V_FULL + s), 1);
      ptx::mbar_init(bar(BAR_V_EMPTY + s), 1);
    }
    for (int s = 0; s < kInfoSlots; ++s) ptx::mbar_init(bar(BAR_INFO + s), 1);
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(bar(BAR_S_FULL + x), 1);
      ptx::mbar_init(bar(BAR_P_FULL + x), 128);
      ptx::mbar_init(bar(BAR_O_DONE + x), 1);
    }
    ptx::mbar_init(bar(BAR_Q_FULL), kSoftmaxThreads);
    ptx::mbar_init(bar(BAR_O_FREE), kSoftmaxThreads);
    ptx::mbar_init(bar(BAR_MMA_DONE), 1);
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&tmem_base_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  wait_prerequisites();
  launch_dependents();
  // where this CTA's run starts
  if (warp == 2) {
    int64_t total = 0;
    for (int b = lane; b < a.B; b += 32) total += head_tiles<kRows>(a, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    total *= a.Hkv;
    const int ctas = running(total, gridDim.x);
    const int64_t start = run_start(total, cta, ctas);
    // the sequence that holds tile `start`
    int64_t before = 0, at = start;
    int seq = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t n = b < a.B ? head_tiles<kRows>(a, b) * a.Hkv : 0;
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
      const int64_t per_head = head_tiles<kRows>(a, seq);
      const Draft dr = draft(a, seq);
      const int hk = static_cast<int>(at / per_head);
      at %= per_head;
      int rb = 0;
      for (; rb < a.blocks - 1; ++rb) {
        const int n = unit_of<kRows>(a, dr, rb).count;
        if (at < n) break;
        at -= n;
      }
      s_at[0] = seq;
      s_at[1] = hk;
      s_at[2] = rb;
      s_at[3] = static_cast<int>(at);
      s_left = cta < ctas ? run_start(total, cta + 1, ctas) - start : 0;
      s_start = start;
      s_total = total;
    }
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = tmem_base_slot;
  Walk walk{s_left, s_at[0], s_at[1], s_at[2], s_at[3]};
  volatile int* abort_p = &abort_flag;
  auto give_up = [&] {
    *abort_p = 1;
    atomicOr(&g_error, kTimeoutBit);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    const int br = a.box_rows, boxes = kTile / br;
    const uint32_t box_bytes = static_cast<uint32_t>(br) * 128;   // 64 columns of its rows
    int n = 0, k_issued = 0, v_issued = 0;   // tiles so far: tile n goes through stage n % kStages
    bool ok = true;
    while (ok && walk.left > 0) {
      const Segment sg = next_segment<kRows>(a, walk);
      if (sg.dr.count < 0 && lane == 0) record_page_error();
      if (sg.empty) continue;
      const int row0 = (sg.u.first + sg.tile) * kTile;   // first token of the segment
      const int lo = a.window_left < 0 ? 0 : max(0, sg.dr.base - a.window_left);
      const int hi = sg.dr.base + sg.u.i1;
      const int total_boxes = sg.count * boxes;
      const int* tab = a.table + static_cast<int64_t>(sg.b) * a.max_pages;
      // Box j holds tokens row0 + j * br ..; lane x keeps the table entries of boxes x, 32 + x,
      // ... one batch of 32 ahead of the loads.
      auto needed = [&](int j) {
        const int r = row0 + j * br;
        return j < total_boxes && r < hi && r + br > lo;
      };
      auto entry = [&](int j) { return needed(j) ? tab[(row0 + j * br) >> a.page_shift] : -1; };
      int cur = entry(lane), nxt = entry(32 + lane);
      for (int i = 0; i < sg.count; ++i, ++n) {
        const int j0 = i * boxes;
        if (i > 0 && j0 % 32 == 0) {
          cur = nxt;
          nxt = entry(j0 + 32 + lane);
        }
        const int s = n % kStages;
        const uint32_t ph = (n / kStages) & 1;
        if (!ptx::wait_bounded_warp(bar(BAR_K_EMPTY + s), ph ^ 1, abort_p, kWaitLimitNs)) {
          ok = false;
          break;
        }
        // lane x < boxes loads box x of this tile
        const int page = __shfl_sync(0xffffffffu, cur, (j0 + lane) % 32);
        const bool need = lane < boxes && needed(j0 + lane);
        const bool load = need && page >= 0 && page < a.num_pages;
        if (need && !load) record_page_error();
        const int r = row0 + (j0 + lane) * br;   // first token of this lane's box
        const unsigned loads = __ballot_sync(0xffffffffu, load);
        const int end = load ? lane * br + min(hi - r, br) : 0;
        uint32_t m[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          m[w] = __reduce_or_sync(0xffffffffu,
                                  load ? bit_range(lane * br - 32 * w, end - 32 * w) : 0u);
        const uint32_t bytes = (D / 64) * box_bytes * __popc(loads);
        if (lane == 0) {
          info[n % kInfoSlots] = make_uint4(m[0], m[1], m[2], m[3]);
          ptx::mbar_arrive(bar(BAR_INFO + n % kInfoSlots));
          ptx::mbar_arrive_expect_tx(bar(BAR_K_FULL + s), bytes);
        }
        __syncwarp();
        const uint32_t dst = base + s * L::kTileBytes + lane * box_bytes;
        const int row = r & ((1 << a.page_shift) - 1);
        if (load)
          for (int c = 0; c < D / 64; ++c)
            tma_load_5d(dst + L::kK + c * kHalfBytes, &tm_k, bar(BAR_K_FULL + s), 0, sg.hk, row, c,
                        page);
        k_issued = n + 1;
        if (!ptx::wait_bounded_warp(bar(BAR_V_EMPTY + s), ph ^ 1, abort_p, kWaitLimitNs)) {
          ok = false;
          break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar(BAR_V_FULL + s), bytes);
        __syncwarp();
        if (load)
          for (int c = 0; c < D / 64; ++c)
            tma_load_5d(dst + L::kV + c * kHalfBytes, &tm_v, bar(BAR_V_FULL + s), 0, sg.hk, row, c,
                        page);
        v_issued = n + 1;
      }
    }
    if (!ok && lane == 0) give_up();
    // Leave no copy in flight (on the normal path these phases completed long ago).
    for (int x = max(0, k_issued - kStages); x < k_issued; ++x)
      ptx::wait_bounded(bar(BAR_K_FULL + x % kStages), (x / kStages) & 1, abort_p, kWaitLimitNs);
    for (int x = max(0, v_issued - kStages); x < v_issued; ++x)
      ptx::wait_bounded(bar(BAR_V_FULL + x % kStages), (x / kStages) & 1, abort_p, kWaitLimitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = ptx::idesc_f16(FP16, kTile, kTile, false);
      constexpr uint32_t idesc_pv = ptx::idesc_f16(FP16, kTile, D, true);
      auto wait = [&](int slot, uint32_t parity) {
        return ptx::wait_bounded(bar(slot), parity & 1, abort_p, kWaitLimitNs);
      };
      auto wait_k = [&](int n) { return wait(BAR_K_FULL + n % kStages, n / kStages); };
      auto wait_v = [&](int n) { return wait(BAR_V_FULL + n % kStages, n / kStages); };
      // S_x = Q K_n^T
      auto issue_s = [&](int x, int n) {
        ptx::tc_fence_after_sync();
        const ptx::SmemDesc q_desc = ptx::smem_desc_sw128_split(
            base + L::kQ + (QT == 2 ? x : 0) * L::kTileBytes, 16, 1024);
        const ptx::SmemDesc k_desc =
            ptx::smem_desc_sw128_split(base + L::kK + (n % kStages) * L::kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * kHalfBytes + (kk % 4) * 32;
          ptx::mma_f16_ss(tmem + x * kTile, q_desc.at(off), k_desc.at(off), idesc_qk, kk > 0);
        }
        ptx::mma_commit(bar(BAR_S_FULL + x));
      };
      // O_x (+)= P_x V_n, P_x from TMEM
      auto issue_pv = [&](int x, int n, bool first) {
        ptx::tc_fence_after_sync();
        const ptx::SmemDesc v_desc = ptx::smem_desc_sw128_split(
            base + L::kV + (n % kStages) * L::kTileBytes, kHalfBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          ptx::mma_f16_ts(tmem + kTmemO + x * D, tmem + x * kTile + kk * 8,
                          v_desc.at(kk * 16 * 128), idesc_pv, (!first || kk > 0) ? 1u : 0u);
        ptx::mma_commit(bar(BAR_O_DONE + x));
      };
      int n0 = 0, segs = 0, done[2] = {0, 0};   // tiles, segments, and tiles of each group so far
      bool ok = true;
      while (ok && walk.left > 0) {
        const Segment sg = next_segment<kRows>(a, walk);
        if (sg.empty) continue;
        const int count = sg.count;
        const bool b_any = QT == 1 || (sg.dr.count * a.G - sg.rb * kRows) > kTile;
        ok = wait(BAR_Q_FULL, segs) && wait_k(n0);
        if (!ok) break;
        issue_s(0, n0);
        if constexpr (QT == 2) {
          if (b_any) issue_s(1, n0);
          ptx::mma_commit(bar(BAR_K_EMPTY + n0 % kStages));
        } else {
          ptx::mma_commit(bar(BAR_K_EMPTY + n0 % kStages));
          if (count > 1) {
            if (!wait_k(n0 + 1)) { ok = false; break; }
            issue_s(1, n0 + 1);
            ptx::mma_commit(bar(BAR_K_EMPTY + (n0 + 1) % kStages));
          }
        }
        for (int j = 0; j < count; ++j) {
          const int n = n0 + j;
          if (!wait_v(n)) { ok = false; break; }
          // O of the segment before has to be out of TMEM
          if (j == 0 && segs > 0 && !wait(BAR_O_FREE, segs - 1)) { ok = false; break; }
          if constexpr (QT == 2) {
            const bool next = j + 1 < count;
            if (!wait(BAR_P_FULL + 0, done[0]++)) { ok = false; break; }
            issue_pv(0, n, j == 0);
            if (next && !wait_k(n + 1)) { ok = false; break; }
            if (next) issue_s(0, n + 1);
            if (b_any) {
              if (!wait(BAR_P_FULL + 1, done[1]++)) { ok = false; break; }
              issue_pv(1, n, j == 0);
            }
            ptx::mma_commit(bar(BAR_V_EMPTY + n % kStages));
            if (next) {
              if (b_any) issue_s(1, n + 1);
              ptx::mma_commit(bar(BAR_K_EMPTY + (n + 1) % kStages));
            }
          } else {
            const int x = j & 1;
            if (!wait(BAR_P_FULL + x, done[x]++)) { ok = false; break; }
            issue_pv(x, n, j < 2);
            ptx::mma_commit(bar(BAR_V_EMPTY + n % kStages));
            if (j + 2 < count) {
              if (!wait_k(n + 2)) { ok = false; break; }
              issue_s(x, n + 2);
              ptx::mma_commit(bar(BAR_K_EMPTY + (n + 2) % kStages));
            }
          }
        }
        n0 += count;
        ++segs;
      }
      if (!ok) give_up();
      // Every MMA this thread issued has completed before TMEM can be released.
      ptx::mma_commit(bar(BAR_MMA_DONE));
      wait(BAR_MMA_DONE, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax groups
    const int x = (warp - 4) / 4;                  // group: 0 = A, 1 = B
    const int quarter = warp & 3;                  // TMEM lanes [32q, 32q+32)
    const int row = quarter * 32 + lane;           // row within the row tile
    const int tid = threadIdx.x - 128, gtid = tid % 128;   // within the groups, within the group
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * kTile;
    const uint32_t tO = tmem + lane_off + kTmemO;  // O_A; O_B is D columns on
    const bool scale_pos = a.scale_log2 > 0.f;
    const float scale = a.scale_log2;
    int n0 = 0, segs = 0, done = 0;   // tiles, segments with tiles, and this group's tiles so far
    int64_t before = 0;               // tiles of the run before the segment, empty units' among them
    bool ok = true;
    // after a wait has run out the loop goes on without data, so that every warp reaches the
    // barriers below
    auto wait = [&](int slot, uint32_t parity) {
      if (ok && !ptx::wait_bounded_warp(bar(slot), parity & 1, abort_p, kWaitLimitNs)) {
        ok = false;
        if (lane == 0) give_up();
      }
      return ok;
    };
    while (walk.left > 0) {
      const Segment sg = next_segment<kRows>(a, walk);
      const int r0 = sg.rb * kRows;                              // first row of the unit
      const int rows = min(kRows, a.T * a.G - r0);               // padding's rows among them
      const int live = min(rows, sg.dr.count * a.G - r0);        // and without them
      const int my = (QT == 2 ? x * kTile : 0) + row;            // this thread's row of the unit
      const int token = (r0 + my) / a.G, head = sg.hk * a.G + (r0 + my) % a.G;
      const int64_t out_row = (static_cast<int64_t>(sg.b) * a.T + token) * a.Hq + head;
      float* const lse = a.lse + (static_cast<int64_t>(sg.b) * a.Hq + head) * a.T + token;
      const int64_t slot = 2ll * cta + (before > 0);
      if (sg.tile == 0 && tid == 0) {
        // this run holds the unit's first tile; its last is in the last run that starts before
        // the unit's end: the largest c with floor(total * c / ctas) < end
        const int ctas = running(s_total, gridDim.x);
        const int64_t end = s_start + before + sg.u.count;
        const int last = static_cast<int>((end * ctas - 1) / s_total);
        a.units[(static_cast<int64_t>(sg.b) * a.Hkv + sg.hk) * a.blocks + sg.rb] =
            make_int2(static_cast<int>(slot), sg.whole ? 0 : last - cta + 1);
      }
      before += sg.count;
      if (sg.tile == 0 && my >= live && my < rows && (QT == 2 || x == 0)) {   // padding
        uint4* const dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out_row * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
        *lse = -INFINITY;
      }
      if (sg.empty) continue;

      // ---- Q: no S of the segment before is still to be computed (its last one has been read)
      {
        constexpr int kChunks = D / 8, kLoaders = QT == 2 ? 128 : kSoftmaxThreads;
        constexpr int kEach = kTile * kChunks / kLoaders;
        const int t = QT == 2 ? gtid : tid, first = QT == 2 ? x * kTile : 0;
        const uint32_t dst = base + L::kQ + (QT == 2 ? x : 0) * L::kTileBytes;
        uint4 v[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const int r = (u * kLoaders + t) / kChunks, c = (u * kLoaders + t) % kChunks;
          if (first + r < live) {
            const int tok = (r0 + first + r) / a.G, h = sg.hk * a.G + (r0 + first + r) % a.G;
            v[u] = *reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(a.q) +
                ((static_cast<int64_t>(sg.b) * a.T + tok) * a.Hq + h) * D + c * 8);
          } else {
            v[u] = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const int r = (u * kLoaders + t) / kChunks, c = (u * kLoaders + t) % kChunks;
          ptx::st_shared_v4(dst + (c / 8) * kHalfBytes + r * 128 + (((c % 8) ^ (r & 7)) << 4), v[u].x,
                            v[u].y, v[u].z, v[u].w);
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(bar(BAR_Q_FULL));
      }

      Row rw{sg.b, my < live ? token : -1, 0};
      if (a.window_left >= 0 && rw.i >= 0) {
        int depth = rw.i;
        if (a.parents) {
          depth = 0;
          for (int at = parent_of(a, sg.b, rw.i); at >= 0; at = parent_of(a, sg.b, at)) ++depth;
        }
        rw.lo = max(0, sg.dr.base + depth - a.window_left);
      }
      // every row sees all keys of a tile within [full_lo, full_hi)
      const int full_lo = a.window_left < 0 ? 0 : sg.dr.base + sg.u.i1 - 1 - a.window_left;
      const int full_hi = a.parents ? sg.dr.base : sg.dr.base + sg.u.i0 + 1;
      const int first_key = (sg.u.first + sg.tile) * kTile;
      const bool active = (QT == 2 ? x * kTile : 0) + quarter * 32 < live;   // rows of this warp
      const int j_first = QT == 2 ? 0 : x, j_step = QT == 2 ? 1 : 2;
      const int j_end = QT == 2 && x == 1 && live <= kTile ? 0 : sg.count;
      float m = -INFINITY, l = 0.f;   // offset of the exponents (log2 units), sum

      for (int j = j_first; j < j_end; j += j_step, ++done) {
        const int n = n0 + j, k0 = first_key + j * kTile;
        wait(BAR_INFO + n % kInfoSlots, n / kInfoSlots);
        // (the product of the tile before is done, too: it was issued before this S)
        if (!wait(BAR_S_FULL + x, done) || (j > j_first && !wait(BAR_O_DONE + x, done - 1)))
          continue;
        const uint4 loaded = info[n % kInfoSlots];
        const bool masked = (loaded.x & loaded.y & loaded.z & loaded.w) != 0xffffffffu ||
                            k0 < full_lo || k0 + kTile > full_hi;
        ptx::tc_fence_after_sync();
        if (active) {
          uint32_t sr[kTile / 32][32];
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c) ptx::tmem_ld_32x32b_x32(tS + c * 32, sr[c]);
          ptx::tmem_wait_ld();
          float s[kTile];
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c) {
            ptx::reg_fence(sr[c]);
#pragma unroll
            for (int t = 0; t < 32; ++t) s[c * 32 + t] = __uint_as_float(sr[c][t]);
          }
          if (!scale_pos) {
            // scale first, so that the maximum below is the maximum of the scaled scores
#pragma unroll
            for (int t = 0; t < kTile; t += 2)
              ptx::mul2(s[t], s[t + 1], s[t], s[t + 1], scale, scale);
          }
          if (masked) {
            uint32_t vis[4];
            visible_bits(a, rw, sg.dr.base, k0, vis);
            vis[0] &= loaded.x;
            vis[1] &= loaded.y;
            vis[2] &= loaded.z;
            vis[3] &= loaded.w;
            __syncwarp();
#pragma unroll
            for (int t = 0; t < kTile; ++t)
              if (!(vis[t / 32] >> (t % 32) & 1)) s[t] = -INFINITY;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int t = 0; t < kTile; t += 8) {
            mx[0] = ptx::max3(mx[0], s[t + 0], s[t + 1]);
            mx[1] = ptx::max3(mx[1], s[t + 2], s[t + 3]);
            mx[2] = ptx::max3(mx[2], s[t + 4], s[t + 5]);
            mx[3] = ptx::max3(mx[3], s[t + 6], s[t + 7]);
          }
          const float mt = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
          const float m_tile = (scale_pos ? mt * scale : mt) - kShift<FP16>;
          float alpha = 1.f;
          const bool rescale = __any_sync(0xffffffffu, m_tile > m + kLag<FP16>);
          if (rescale) {
            // every row of this warp to its running maximum; l now, O below
            const float m_new = fmaxf(m, m_tile);
            alpha = ptx::exp2_approx(m - (m_new == -INFINITY ? 0.f : m_new));
            l *= alpha;
            m = m_new;
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          // P = 2^(scaled score - offset) over the first 64 columns of S, two keys to a column
          float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c) {
            uint32_t pr[16];
#pragma unroll
            for (int t = 0; t < 16; ++t) {
              float e0, e1;
              if (scale_pos)
                ptx::fma2(e0, e1, s[32 * c + 2 * t], s[32 * c + 2 * t + 1], scale, scale, -m_use,
                          -m_use);
              else
                ptx::add2(e0, e1, s[32 * c + 2 * t], s[32 * c + 2 * t + 1], -m_use, -m_use);
              const float p0 = ptx::exp2_approx(e0), p1 = ptx::exp2_approx(e1);
              ptx::add2(rs0, rs1, rs0, rs1, p0, p1);
              pr[t] = pack2<FP16>(p0, p1);
            }
            ptx::tmem_st_32x32b_x16(tS + c * 16, pr);
          }
          l += rs0 + rs1;
          if (rescale && j > j_first) {
            // the product before has completed: it was issued before this S
            uint32_t orr[D / 32][32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              ptx::tmem_ld_32x32b_x32(tO + x * D + c * 32, orr[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              ptx::reg_fence(orr[c]);
#pragma unroll
              for (int t = 0; t < 32; t += 2) {
                float a0 = __uint_as_float(orr[c][t]), a1 = __uint_as_float(orr[c][t + 1]);
                ptx::mul2(a0, a1, a0, a1, alpha, alpha);
                orr[c][t] = __float_as_uint(a0);
                orr[c][t + 1] = __float_as_uint(a1);
              }
              ptx::tmem_st_32x32b_x32(tO + x * D + c * 32, orr[c]);
            }
          }
          ptx::tmem_wait_st();
        }
        if (masked && (QT == 1 || x == 0) && wait(BAR_V_FULL + n % kStages, n / kStages)) {
          // V: zeros for the rows of no token, and for what is not finite
          constexpr int kChunks = D / 8;
          const uint32_t vt = L::kV + (n % kStages) * L::kTileBytes;
          bool found = false;
#pragma unroll 4
          for (int u = gtid; u < kTile * kChunks; u += 128) {
            const int r = u / kChunks, c = u % kChunks;
            const uint32_t bits = r < 64 ? (r < 32 ? loaded.x : loaded.y)
                                         : (r < 96 ? loaded.z : loaded.w);
            uint4* const at = reinterpret_cast<uint4*>(
                gen + vt + (c / 8) * kHalfBytes + r * 128 + (((c % 8) ^ (r & 7)) << 4));
            if (!(bits >> (r % 32) & 1)) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint4 v = *at;
            const uint32_t bx = not_finite2<FP16>(v.x), by = not_finite2<FP16>(v.y),
                           bz = not_finite2<FP16>(v.z), bw = not_finite2<FP16>(v.w);
            if (bx | by | bz | bw) {
              found = true;
              *at = make_uint4(v.x & ~bx, v.y & ~by, v.z & ~bz, v.w & ~bw);
            }
          }
          if (found) s_not_finite = segs + 1;
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before_sync();
        ptx::mbar_arrive(bar(BAR_P_FULL + x));
      }

      // ---- the segment's end
      if (j_end > j_first) wait(BAR_O_DONE + x, done - 1);
      // one row tile: the groups exchange their offsets and sums, A's first, then B's in its place
      if (QT == 1 && x == 0) s_ml[row] = make_float2(m, l);
      ptx::tc_fence_before_sync();
      ptx::named_barrier_sync(1, kSoftmaxThreads);
      ptx::tc_fence_after_sync();
      float2 other = make_float2(-INFINITY, 0.f);
      if constexpr (QT == 1) {
        if (x == 1) {
          other = s_ml[row];
          s_ml[row] = make_float2(m, l);
        }
        ptx::named_barrier_sync(1, kSoftmaxThreads);
        if (x == 0) other = s_ml[row];
      }
      constexpr int kCols = QT == 2 ? D : D / 2;   // columns of this thread's row: [c_first, ..)
      const int c_first = QT == 2 ? 0 : x * kCols;
      const bool two = QT == 1 && sg.count > 1;    // both groups have an O
      float fa = 1.f, fb = 0.f;
      if (QT == 1) {
        const float2 mine = make_float2(m, l), ml_a = x == 0 ? mine : other,
                     ml_b = x == 0 ? other : mine;
        m = fmaxf(ml_a.x, ml_b.x);
        const float u = m == -INFINITY ? 0.f : m;
        fa = ptx::exp2_approx(ml_a.x - u);
        fb = ptx::exp2_approx(ml_b.x - u);
        l = ml_a.y * fa + ml_b.y * fb;
      }
      const float inv = inverse(l);
      if (ok && (QT == 1 ? active : j_end > 0 && active)) {
#pragma unroll 1
        for (int c = 0; c < kCols / 32; ++c) {
          const int col = c_first + c * 32;
          uint32_t oa[32], ob[32];
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(tO + (QT == 2 ? x * D : 0) + col, oa);
          if (two) ptx::tmem_ld_32x32b_x32(tO + D + col, ob);
          ptx::tmem_wait_ld();
          ptx::reg_fence(oa);
          if (two) ptx::reg_fence(ob);
          float v[32];
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            v[t] = __uint_as_float(oa[t]);
            if (QT == 1) v[t] = v[t] * fa + (two ? __uint_as_float(ob[t]) * fb : 0.f);
          }
          if (my < live) {
            if (sg.whole) {
              uint4* const dst =
                  reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out_row * D + col);
#pragma unroll
              for (int t = 0; t < 4; ++t)
                dst[t] = make_uint4(pack2<FP16>(v[8 * t] * inv, v[8 * t + 1] * inv),
                                    pack2<FP16>(v[8 * t + 2] * inv, v[8 * t + 3] * inv),
                                    pack2<FP16>(v[8 * t + 4] * inv, v[8 * t + 5] * inv),
                                    pack2<FP16>(v[8 * t + 6] * inv, v[8 * t + 7] * inv));
            } else {
              float4* const dst =
                  reinterpret_cast<float4*>(a.part_o + (slot * a.part_rows + my) * D + col);
#pragma unroll
              for (int t = 0; t < 8; ++t)
                dst[t] = make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
            }
          }
        }
        if (s_not_finite == segs + 1 && rw.i >= 0)
          add_not_finite<FP16>(
              a, rw, sg.dr.base, sg.hk, D, first_key, sg.count, full_lo, full_hi, c_first, kCols,
              sg.whole ? nullptr : a.part_o + (slot * a.part_rows + my) * D,
              sg.whole ? static_cast<uint16_t*>(a.o) + out_row * D : nullptr);
        if (my < live && (QT == 2 || x == 0)) {
          if (sg.whole)
            *lse = lse_of(m, l);
          else
            a.part_ml[slot * a.part_rows + my] = make_float2(m, l);
        }
      }
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(bar(BAR_O_FREE));
      n0 += sg.count;
      ++segs;
    }
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// The parts of a unit that more than one run covers, joined: a warp for each row, D / 32 columns
// a lane. The part in the first run's slot is followed by those of the next CTAs, each in its
// CTA's first slot.
constexpr int kJoinThreads = 256;

template <int D, bool FP16, int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    fa_paged_tree_join_kernel(const __grid_constant__ Args a) {
  constexpr int E = D / 32;
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  wait_prerequisites();
  launch_dependents();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + threadIdx.x / 32;
  if (id >= static_cast<int64_t>(a.B) * a.T * a.Hq) return;
  const int lane = threadIdx.x % 32;
  const int h = static_cast<int>(id % a.Hq), i = static_cast<int>(id / a.Hq % a.T);
  const int b = static_cast<int>(id / a.Hq / a.T);
  const int r = i * a.G + h % a.G, my = r % ROWS;
  const int2 u =
      a.units[(static_cast<int64_t>(b) * a.Hkv + h / a.G) * a.blocks + r / ROWS];
  if (u.y == 0 || i >= draft(a, b).count) return;   // one run's, and written; padding
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int p = 0; p < u.y; ++p) {
    const int64_t slot = p == 0 ? u.x : 2 * (u.x / 2 + p);
    const int64_t at = slot * a.part_rows + my;
    const float2 ml = a.part_ml[at];
    const Vec v = *reinterpret_cast<const Vec*>(a.part_o + at * D + lane * E);
    const float* const f = reinterpret_cast<const float*>(&v);
    const float n = fmaxf(m, ml.x), top = n == -INFINITY ? 0.f : n;
    const float old = ptx::exp2_approx(m - top), now = ptx::exp2_approx(ml.x - top);
    m = n;
    l = l * old + ml.y * now;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * old + f[e] * now;
  }
  const float inv = inverse(l);
  uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + id * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<FP16>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.T + i] = lse_of(m, l);
}

// Row tiles of a unit, and with it its rows: two where a key head has more than 128 rows.
int row_tiles(int T, int Hq, int Hkv) { return static_cast<int64_t>(T) * (Hq / Hkv) > kTile ? 2 : 1; }

// Workspace: the parts' O, their offsets and sums, the units' parts.
struct Layout {
  int64_t ctas, blocks, part_rows;
  size_t part_ml, units, end;
};
Layout layout(int B, int T, int Hq, int Hkv, int d, int64_t capacity) {
  Layout l;
  const int64_t rows = static_cast<int64_t>(T) * (Hq / Hkv), unit = row_tiles(T, Hq, Hkv) * kTile;
  l.blocks = (rows + unit - 1) / unit;
  l.part_rows = std::min(rows, unit);
  l.ctas = std::min<int64_t>(kSms, B * Hkv * l.blocks * ((capacity + kTile - 1) / kTile));
  l.part_ml = static_cast<size_t>(2 * l.ctas * l.part_rows * d) * 4;
  l.units = l.part_ml + static_cast<size_t>(2 * l.ctas * l.part_rows) * 8;
  l.end = l.units + static_cast<size_t>(B * Hkv * l.blocks) * 8;
  return l;
}

template <int D, bool FP16, int QT>
cudaError_t launch_impl(const TreeParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  const int64_t capacity = static_cast<int64_t>(c.max_pages) * c.page_size;
  const Layout l = layout(c.B, p.T, p.Hq, c.Hkv, D, capacity);
  char* const ws = static_cast<char*>(p.workspace);
  Args a;
  a.q = p.q;
  a.table = c.block_table;
  a.seqlens = c.seqlens;
  a.parents = p.parents;
  a.new_lens = p.new_lens;
  a.v_pages = c.v_pages;
  a.o = p.o;
  a.lse = p.lse;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  a.units = reinterpret_cast<int2*>(ws + l.units);
  a.B = c.B;
  a.T = p.T;
  a.Hq = p.Hq;
  a.Hkv = c.Hkv;
  a.G = p.Hq / c.Hkv;
  a.blocks = static_cast<int>(l.blocks);
  a.part_rows = static_cast<int>(l.part_rows);
  a.page_shift = 0;
  while (1 << a.page_shift < c.page_size) ++a.page_shift;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.box_rows = std::min(c.page_size, kTile);
  a.window_left = p.window_left;
  a.scale_log2 = p.scale_log2;
  CUtensorMap tm_k, tm_v;
  if (!encode_pages(&tm_k, c.k_pages, c, a.box_rows, 1, FP16) ||
      !encode_pages(&tm_v, c.v_pages, c, a.box_rows, 1, FP16))
    return cudaErrorInvalidValue;
  auto kernel = fa_paged_tree_kernel<D, FP16, QT>;
  const int smem = static_cast<int>(Smem<D, QT>::kDynamic);
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  err = launch_paged(kernel, l.ctas, kThreads, smem, stream, 0, tm_k, tm_v, a);
  // units of one tile are never split: nothing to join
  if (err != cudaSuccess || capacity <= kTile) return err;
  const int64_t rows = static_cast<int64_t>(c.B) * p.T * p.Hq;
  return launch_paged(fa_paged_tree_join_kernel<D, FP16, QT * kTile>,
                      (rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32), kJoinThreads, 0, stream, 0,
                      a);
}

template <int D, bool FP16>
cudaError_t launch_rows(const TreeParams& p, cudaStream_t stream) {
  return row_tiles(p.T, p.Hq, p.c.Hkv) == 1 ? launch_impl<D, FP16, 1>(p, stream)
                                            : launch_impl<D, FP16, 2>(p, stream);
}

}  // namespace

size_t paged_tree_workspace(int B, int T, int Hq, int Hkv, int d, int page_size, int max_pages) {
  return layout(B, T, Hq, Hkv, d, static_cast<int64_t>(max_pages) * page_size).end;
}

cudaError_t launch_paged_tree(const TreeParams& p, cudaStream_t stream) {
  if (p.c.d == 64)
    return p.fp16 ? launch_rows<64, true>(p, stream) : launch_rows<64, false>(p, stream);
  return p.fp16 ? launch_rows<128, true>(p, stream) : launch_rows<128, false>(p, stream);
}

cudaError_t read_and_clear_tree_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
