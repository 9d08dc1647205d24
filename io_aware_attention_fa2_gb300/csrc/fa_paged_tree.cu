// fa_paged_tree.cu -- attention of drafted tokens over a paged key-value cache: each sees its
// sequence's context, its ancestors in the draft's tree and itself (include/fa.h).
//
//   s_ij = scale <q_i, k_j>,  O_i = sum_j e^{s_ij - LSE_i} v_j,  LSE_i = ln sum_j e^{s_ij}
//
// What bounds it: K and V are read once, 4 d bytes a token and key head, for 4 d operations of
// each row -- a drafted token and one of the G query heads that share the key head. Up to about
// 250 rows HBM is the bound, from there the tensor cores; both products run on tcgen05 with 128 rows
// to a tile, whatever their number: a tile of 128 keys takes 1100 cycles of the tensor pipe (d = 128)
// for 2 rows as for 128, less than the 2800 that its 64 KiB take from HBM.
//
// Rows of a (sequence, key head) are taken in the order (token, query head), in blocks of 128 (one
// row tile) or 256 (two, where there are more than 128 rows). A block over its keys is a unit. The
// keys are cut into tiles of 128 tokens, and the tiles of all units, in order, into one equal run
// for each CTA (one on each SM), whatever the lengths are; a unit's start and end count as some
// tiles more. A run that covers a whole unit writes O and LSE; one that covers a part leaves the
// part's offset, sum and unnormalised O (fp32) in the workspace, and a second kernel joins the
// parts of a unit in a fixed order. Short caches take one launch and no workspace: a cluster of up to
// eight CTAs has one unit, and the parts are joined through distributed shared memory.
//
// One CTA:
//   warp 0, 2    TMA producers of K and V: boxes of a page's rows into two rings
//   warp 1       TMEM allocator and MMA issuer
//   warp 3       scheduler: the run's segments (a unit's part) from lengths that only the device
//                knows, four of them ahead
//   warps 4..19  softmax: S from TMEM, P back over it, O rescaled in TMEM when the maximum has
//                grown; Q into shared memory at a segment's start, O out of TMEM at its end
// Eight softmax warps have a stream, A or B. A thread has half a row, 64 keys of a tile, and
// exchanges the row's maximum with the thread that has the others. Two row tiles: A has the first
// 128 rows, B the others, and both see every tile. One row tile: A takes the even tiles of a
// segment and B the odd ones, each with an offset, sums and O of its own, joined at the end; so
// there, too, one stream's softmax runs beside the other's products.
//
// Measured on the device (replays): B=8 Hkv=8 of 4 query heads d=128 bf16, 64 drafted tokens (256
// rows) over up to 32K: 140-142 us, 1210-1230 TFLOP/s, 4.8-4.9 TB/s; B=16, 16 drafted tokens (64 rows)
// over up to 16K, pages of 16: 116-118 us, 5.5-5.6 TB/s (82-83 % of the measured copy rate); B=4 Hkv=4
// of 8, up to 5 tokens over up to 64K: 65-66 us, 4.4-4.5 TB/s. With one row tile HBM is busy at 97 % of the copy rate from the
// first load to the last; before it are 3 us (lengths, table: dependent reads, and cold instructions),
// behind it 4 for the last part and 4 for the join. In the steady state a tile takes 1800 to 2600
// cycles (one row tile; HBM) or 3200 (two; 2180 of them the tensor pipe's), and the step from one
// unit to the next some 6000 or 14000 that nothing overlaps.
//
// Measured slower (the B=16 case where no other is named): eight softmax warps with a whole row each,
// which spilled registers, and one producer for K and V, 151 us, when this form took 135; segments
// worked out by every role for itself and S kept in registers between its maximum and P, 135 when
// 129; products issued behind a branch on one lane, where operands move to uniform registers one
// by one (85 cycles an instruction instead of 30), 180 us for the B=8 case when 150; equal runs
// without the units' cost, 74 us for the B=4 case when 69; parts as rows of D columns, where 32
// threads with a row each write 16 bytes to 32 lines, 117.0 us instead of 115.4, B=8 142.1 instead of
// 139.8; a third stage of K or of V for two row tiles in the place that O passes through on its way
// out, 146 us for the B=8 case when 143.
//
// Masks. Tiles of the context that no window cuts need none. In the others a thread builds the 64
// bits of its keys: a range of the context, and the ancestors by walking up the tree. Keys that some
// row of the tile does not see have P = 0 there, but 0 times a NaN or an infinity would not be 0: in
// such tiles stream A (the tile's stream) first replaces what is not finite in V by 0, and rows of
// tokens that do not exist or were not loaded as well; where it found any, the segment's end adds
// them to the rows that do see them.
//
// P is rounded to the type once for the product with V, a rounding of the same size as the output's
// (relative error 0.0019 to 0.0023 for both, bf16, instead of 0.0016 for the output's alone, at which
// the decoding kernel stays, which keeps two numbers for P). fp16 ends at 2^-24, so there P is taken
// 2^11 times as large, and up to 2^4 more until a grown maximum moves the offset: what is lost are
// probabilities below 2^-36 of the largest.
#include <cooperative_groups.h>
#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;
namespace cg = cooperative_groups;

constexpr int kTile = 128;                     // tokens of a tile, and rows of a row tile
constexpr int kSoftmaxThreads = 512;
constexpr int kThreads = 128 + kSoftmaxThreads;
constexpr int kSms = 152;                      // of a GB300; on another count only speed differs
constexpr uint32_t kHalfBytes = kTile * 64 * 2;   // 128 rows of 64 columns
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kMaxStages = 6;
// A slot is written again with the tile kInfoSlots on, for which a K stage has to be free: the
// softmax of the tile kMaxStages + 2 before it is over by then.
constexpr int kInfoSlots = kMaxStages + 2;

// P = 2^((s - m) scale + kShift): m is the row's maximum of the products s as they are, and moves
// when that has grown by more than kLag (log2 units). The difference comes first, and is 0 for the
// maximum itself: scaled, a large maximum would be rounded by more than the type holds beside the
// shift (from 2^24 on by 1 and more). The packed addition that this takes costs nothing measurable
// (B=8 140.1 and 140.3 us).
template <bool FP16>
constexpr float kShift = FP16 ? 11.f : 0.f;
template <bool FP16>
constexpr float kLag = FP16 ? 4.f : 8.f;

struct Args {
  const void* q;
  const int* table;
  const int* seqlens;
  const int* parents;
  const int* new_lens;
  const void* v_pages;
  void* o;
  float* lse;
  float* part_o;      // [2 * CTAs][D / 4][part_rows][4]: CTA c's first run at slot 2c, its last at
                      // 2c + 1; four columns of all rows together, as 32 threads with a row each
                      // write them
  float2* part_ml;    // [2 * CTAs][part_rows]: offset (a product, not scaled) and sum of the part
  int2* units;        // [B * Hkv * blocks]: slot of the unit's first part, number of parts (0: the
                      // unit was one run's, and is written)
  int B, T, Hq, Hkv, G, blocks;   // blocks of rows for each key head
  uint32_t g_magic;               // ceil(2^32 / G), or 0: see token_of
  int part_rows;                  // rows of a unit, at most
  int page_shift, num_pages, max_pages, box_rows, window_left;
  int unit_cost;                  // of a unit's start and end, in tiles
  float scale_log2;
};

// Drafted token of row r, r / G: by the product's upper half, which is exact while r * G < 2^32
// (r < T * G, so for G up to 2047); g_magic is 0 for G = 1 and for more.
__device__ __forceinline__ int token_of(const Args& a, int r) {
  if (a.g_magic) return static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.g_magic));
  return a.G == 1 ? r : r / a.G;
}

// Factor of a difference of products in an exponent (log2 units). Q takes the scale's sign, and a
// scale of 0, so that it is positive.
__device__ __forceinline__ float factor_of(const Args& a) {
  return a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
}
// LSE in natural units of a row from its offset and its sum.
template <bool FP16>
__device__ __forceinline__ float lse_at(float m, float l, float scale) {
  return l == 0.f ? -INFINITY : fmaf(m, scale, log2f(l) - kShift<FP16>) * kLn2;
}

// A block of rows: tokens [i0, i1) (i1 <= i0: only rows of the padding) and tiles
// [first, first + count), at least one.
struct Unit {
  int i0, i1, first, count;
};
template <int ROWS>
__device__ __forceinline__ Unit unit_of(const Args& a, Draft dr, int rb) {
  Unit u;
  u.i0 = token_of(a, rb * ROWS);
  u.i1 = min(dr.count, token_of(a, min((rb + 1) * ROWS, a.T * a.G) - 1) + 1);
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
// What a unit costs in a run, in tiles: its tiles and, for its start and end, unit_cost.
__device__ __forceinline__ int cost_of(const Args& a, const Unit& u) {
  return u.i1 > u.i0 ? u.count + a.unit_cost : 1;
}
// That of all row blocks of a key head.
template <int ROWS>
__device__ __forceinline__ int head_cost(const Args& a, Draft dr) {
  int n = 0;
#pragma unroll 1
  for (int rb = 0; rb < a.blocks; ++rb) n += cost_of(a, unit_of<ROWS>(a, dr, rb));
  return n;
}
// Equal runs of a cost of `total` (within 31 bits) for `ctas` CTAs.
struct Runs {
  int each, more;   // the first `more` of them are longer by one
  __device__ __forceinline__ Runs(int total, int ctas) : each(total / ctas), more(total - each * ctas) {}
  __device__ __forceinline__ int start(int c) const { return each * c + min(c, more); }
};

// A part of a run: consecutive tiles of one unit.
struct Segment {
  int b, hk, base;          // sequence, key head, length of the context
  int r0, live;             // the unit's first row, and its rows that are not padding
  int rows;                 // rows with the padding's, which this segment writes; or 0
  int first_key, count;     // of the segment; its tiles (0: there is no further segment)
  int lo, hi;               // keys that some row sees are within [lo, hi)
  int full_lo, full_hi;     // every row sees all keys of a tile within these
  int whole;                // the segment is the unit
  int slot;                 // of its part otherwise
};

// Barrier slots.
constexpr int kSegments = 4;               // segments that are known ahead
constexpr int kConsumers = 3 + kSoftmaxThreads / 32;   // warps that read them
enum : int {
  BAR_K_FULL = 0,                          // + stage
  BAR_K_EMPTY = BAR_K_FULL + kMaxStages,   // + stage
  BAR_V_FULL = BAR_K_EMPTY + kMaxStages,   // + stage
  BAR_V_EMPTY = BAR_V_FULL + kMaxStages,   // + stage
  BAR_INFO = BAR_V_EMPTY + kMaxStages,     // + slot: the tile's loaded keys and masks are known
  BAR_SEG_FULL = BAR_INFO + kInfoSlots,    // + slot: a segment is there
  BAR_SEG_EMPTY = BAR_SEG_FULL + kSegments,   // + slot: and was read by all
  BAR_S_FULL = BAR_SEG_EMPTY + kSegments,  // + stream: S computed
  BAR_P_FULL = BAR_S_FULL + 2,             // + stream: P in TMEM, O rescaled, V cleaned (256)
  BAR_O_DONE = BAR_P_FULL + 2,             // + stream: the segment's last P V computed
  BAR_Q_FULL = BAR_O_DONE + 2,             // Q of the segment in shared memory (512)
  BAR_O_FREE = BAR_Q_FULL + 1,             // O of the segment out of TMEM (512)
  BAR_MMA_DONE = BAR_O_FREE + 1,
  BAR_COUNT = BAR_MMA_DONE + 1
};

// What is in shared memory besides Q and the rings.
struct Misc {
  uint64_t bars[BAR_COUNT];
  uint4 loaded[kInfoSlots];     // bits of a tile's keys that exist and were loaded
  int masked[kInfoSlots];       // some row does not see all of a tile's keys
  float red[2][2][kTile];       // [stream][half][row]: exchange of maxima and sums
  Segment seg[kSegments];
  uint32_t tmem_base;
  int abort;
  int go;                       // the softmax warps have another segment
  int not_finite[2];            // by segments in turns: the segment (+ 1) in whose masked tiles V
                                // had such values
};

template <int D, int QT>
struct Smem {
  static constexpr uint32_t kTileBytes = (D / 64) * kHalfBytes;
  static constexpr int kStages = D == 128 ? (QT == 1 ? 3 : 2) : (QT == 1 ? 6 : 5);
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + QT * kTileBytes;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  // two row tiles: for each softmax warp 32 rows of kChunk columns of O on their way out
  static constexpr int kChunk = 16;
  static constexpr uint32_t kOut = kV + kStages * kTileBytes;
  static constexpr uint32_t kMisc = kOut + (QT == 2 ? kSoftmaxThreads * kChunk * 2 : 0);
  static constexpr uint32_t kDynamic = kMisc + sizeof(Misc);
};
static_assert(Smem<128, 1>::kDynamic <= 232448 && Smem<128, 2>::kDynamic <= 232448 &&
                  Smem<64, 1>::kDynamic <= 232448 && Smem<64, 2>::kDynamic <= 232448,
              "shared memory");

// Bits [lo, hi) of 32, for any lo and hi.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1;
  return below_hi & ~below_lo;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Parent of drafted token i of sequence b, -1 for the context and (recorded) for what is no
// earlier token.
__device__ __forceinline__ int parent_of(const Args& a, int b, int i) {
  const int up = a.parents[static_cast<int64_t>(b) * a.T + i];
  if (up >= -1 && up < i) return up;
  record_page_error();
  return -1;
}

// Keys k0 .. k0 + 63 that drafted token i of sequence b sees, as bits.
__device__ __forceinline__ uint2 visible_bits(const Args& a, int b, int base, int i, int k0) {
  int lo = 0;
  if (a.window_left >= 0) {
    int depth = i;
    if (a.parents) {
      depth = 0;
#pragma unroll 1
      for (int at = parent_of(a, b, i); at >= 0; at = parent_of(a, b, at)) ++depth;
    }
    lo = base + depth - a.window_left - k0;
  }
  const int hi = (a.parents ? base : base + i + 1) - k0;   // a chain's keys are a range, too
  uint32_t v0 = bit_range(lo, hi), v1 = bit_range(lo - 32, hi - 32);
  if (a.parents && k0 + 64 > base) {
    int steps = a.window_left >= 0 ? a.window_left : kMaxDraft;   // ancestors within the window
#pragma unroll 1
    for (int at = i; at >= 0 && base + at >= k0; at = parent_of(a, b, at)) {
      if (steps-- < 0) break;
      const int t = base + at - k0;
      const uint32_t bit = 1u << (t & 31);
      if (t < 32)
        v0 |= bit;
      else if (t < 64)
        v1 |= bit;
    }
  }
  return make_uint2(v0, v1);
}

// One lane of a converged warp: nonzero in it.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}
// ptx::mma_f16_ss, mma_f16_ts and mma_commit, by the lanes whose `one` is not zero.
__device__ __forceinline__ void mma_ss_if(uint32_t one, uint32_t d_tmem, uint64_t a_desc,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t one, uint32_t d_tmem, uint32_t a_tmem,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
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

// V of a masked tile, by the 256 threads of a stream: zeros for the rows of no token, and for what
// is not finite (then true).
template <int D, bool FP16>
__device__ __noinline__ bool clean_values(uint8_t* tile, uint4 loaded, int t) {
  // thread t has the piece t % kChunks of every kStep-th row, at one place of the swizzle
  constexpr int kChunks = D / 8, kStep = 256 / kChunks, kEach = kTile / kStep;
  const int r0 = t / kChunks, c = t % kChunks;
  uint4* const at = reinterpret_cast<uint4*>(tile + (c / 8) * kHalfBytes + r0 * 128 +
                                             (((c % 8) ^ (r0 & 7)) << 4));
  uint4 v[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) v[u] = at[u * kStep * 8];
  bool found = false;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const uint32_t words[4] = {loaded.x, loaded.y, loaded.z, loaded.w};
    if (!(words[u * kStep / 32] >> ((u * kStep + r0) % 32) & 1)) {
      at[u * kStep * 8] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint32_t x = not_finite2<FP16>(v[u].x), y = not_finite2<FP16>(v[u].y),
                   z = not_finite2<FP16>(v[u].z), w = not_finite2<FP16>(v[u].w);
    if (x | y | z | w) {
      found = true;
      at[u * kStep * 8] = make_uint4(v[u].x & ~x, v[u].y & ~y, v[u].z & ~z, v[u].w & ~w);
    }
  }
  return found;
}

// The rare end of a segment in whose masked tiles V was not finite: those values, which the
// products have taken as 0, added to the row of token i (its part, `step` floats from four columns
// to the next four, or its output; columns [c0, c0 + cols)) for the keys that it sees.
template <bool FP16>
__device__ __noinline__ void add_not_finite(const Args& a, const Segment& sg, int i, int d, int c0,
                                            int cols, float* part, int step, uint16_t* out) {
  const int* const tab = a.table + static_cast<int64_t>(sg.b) * a.max_pages;
  for (int j = 0; j < sg.count; ++j) {
    const int k0 = sg.first_key + j * kTile;
    bool masked = k0 < sg.full_lo || k0 + kTile > sg.full_hi;
    for (int t = k0; t < k0 + kTile && !masked; t += a.box_rows) {   // all within [0, full_hi)
      const int page = tab[t >> a.page_shift];
      masked = page < 0 || page >= a.num_pages;
    }
    if (!masked) continue;
    const uint2 first = visible_bits(a, sg.b, sg.base, i, k0);
    const uint2 second = visible_bits(a, sg.b, sg.base, i, k0 + 64);
    const uint4 vis = make_uint4(first.x, first.y, second.x, second.y);
    for (int t = 0; t < kTile; ++t) {
      const uint32_t word = t < 64 ? (t < 32 ? vis.x : vis.y) : (t < 96 ? vis.z : vis.w);
      if (!(word >> (t % 32) & 1)) continue;
      const int page = tab[(k0 + t) >> a.page_shift];
      if (page < 0 || page >= a.num_pages) continue;
      const int64_t at = (static_cast<int64_t>(page) << a.page_shift) +
                         ((k0 + t) & ((1 << a.page_shift) - 1));
      const uint32_t* const src = reinterpret_cast<const uint32_t*>(
          static_cast<const uint16_t*>(a.v_pages) + (at * a.Hkv + sg.hk) * d + c0);
      for (int c = 0; c < cols; c += 2) {
        const uint32_t w = src[c / 2];
        if (!not_finite2<FP16>(w)) continue;
        const float2 f = unpack2<FP16>(w);
        const float fx = isfinite(f.x) ? 0.f : f.x, fy = isfinite(f.y) ? 0.f : f.y;
        if (part) {
          float* const to = part + (c0 + c) / 4 * step + (c0 + c) % 4;
          to[0] += fx;
          to[1] += fy;
        } else {
          uint32_t* const to = reinterpret_cast<uint32_t*>(out + c0 + c);
          const float2 o = unpack2<FP16>(*to);
          *to = pack2<FP16>(o.x + fx, o.y + fy);
        }
      }
    }
  }
}

// SHORT: a cluster of CTAs has one unit, each CTA an equal share of its tiles, and the parts are
// joined through distributed shared memory. Otherwise: runs over all units.
template <int D, bool FP16, int QT, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_tree_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Args a) {
  using L = Smem<D, QT>;
  constexpr int kStages = L::kStages, kRows = QT * kTile;
  constexpr uint32_t kTmemO = 2 * kTile, kTmemCols = 512;   // S_A, S_B, O_A, O_B
  // (there is no room for a base that is not aligned)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  if (base != ptx::smem_addr(smem_raw)) {
    atomicOr(&g_error, kTimeoutBit);
    return;
  }
  Misc& ms = *reinterpret_cast<Misc*>(smem_raw + L::kMisc);
  const uint32_t bars = base + L::kMisc + static_cast<uint32_t>(offsetof(Misc, bars));
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    ms.abort = 0;
    ms.not_finite[0] = ms.not_finite[1] = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(BAR_K_FULL + s), 1);
      ptx::mbar_init(bar(BAR_K_EMPTY + s), 1);
      ptx::mbar_init(bar(BAR_V_FULL + s), 1);
      ptx::mbar_init(bar(BAR_V_EMPTY + s), 1);
    }
    for (int s = 0; s < kInfoSlots; ++s) ptx::mbar_init(bar(BAR_INFO + s), 1);
    for (int s = 0; s < kSegments; ++s) {
      ptx::mbar_init(bar(BAR_SEG_FULL + s), 1);
      ptx::mbar_init(bar(BAR_SEG_EMPTY + s), kConsumers);
    }
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(bar(BAR_S_FULL + x), 1);
      ptx::mbar_init(bar(BAR_P_FULL + x), kSoftmaxThreads / 2);
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
    ptx::tmem_alloc(ptx::smem_addr(&ms.tmem_base), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  wait_prerequisites();
  launch_dependents();
  // (an allocation of all 512 columns starts at address 0, which the products use as a constant)
  const uint32_t tmem = 0;
  volatile int* abort_p = &ms.abort;
  auto give_up = [&] {
    *abort_p = 1;
    atomicOr(&g_error, kTimeoutBit);
  };
  // SHORT: this CTA's part, where K and V were
  float* const short_part = reinterpret_cast<float*>(smem_raw + L::kK);                 // [D / 4][128][4]
  float2* const short_ml = reinterpret_cast<float2*>(smem_raw + L::kK + kTile * D * 4);   // [128]
  static_assert(!SHORT || L::kK + kTile * (D * 4 + 8) <= L::kMisc, "the part's place");
  // Segment s of the run for the warps that read them; false when a wait has run out. What is in front
  // of it may be all lengths of the batch, or units of nothing but padding: 41 ns a sequence.
  const uint64_t segment_limit = kWaitLimitNs + static_cast<uint64_t>(a.B) * 200;
  auto segment = [&](int s) {
    return ptx::wait_bounded(bar(BAR_SEG_FULL + s % kSegments), (s / kSegments) & 1, abort_p,
                             segment_limit);
  };
  auto segment_read = [&](int s) { ptx::mbar_arrive(bar(BAR_SEG_EMPTY + s % kSegments)); };

  if (warp == 3) {
    // ------------------------------------------------------------------ scheduler
    int segs = 0;
    bool ok = true;
    // a segment in front may take as long as the run's tiles do (some 2 us each)
    uint64_t limit = kWaitLimitNs;
    auto publish = [&](int b, int hk, Draft dr, const Unit& u, int r0, int live, int tile, int count,
                       int slot) {
      const int s = segs % kSegments;
      ok = ptx::wait_bounded_warp(bar(BAR_SEG_EMPTY + s), ((segs / kSegments) & 1) ^ 1, abort_p,
                                  limit);
      if (ok && lane == 0) {
        Segment& g = ms.seg[s];
        g.b = b;
        g.hk = hk;
        g.base = dr.base;
        g.r0 = r0;
        g.live = live;
        g.rows = tile == 0 ? min(kRows, a.T * a.G - r0) : 0;
        g.first_key = (u.first + tile) * kTile;
        g.count = count;
        g.lo = a.window_left < 0 ? 0 : max(0, dr.base - a.window_left);
        g.hi = dr.base + u.i1;
        g.full_lo = a.window_left < 0 ? 0 : dr.base + u.i1 - 1 - a.window_left;
        g.full_hi = a.parents ? dr.base : dr.base + u.i0 + 1;
        g.whole = !SHORT && count == u.count;
        g.slot = slot;
        ptx::mbar_arrive(bar(BAR_SEG_FULL + s));
      }
      ++segs;
    };
    // a unit of padding alone: `rows` rows from r0 (12000 cycles for 256 of them, by one warp)
    auto clear = [&](int b, int hk, int r0, int rows) {
      constexpr int kChunks = D / 8, kStep = 32 / kChunks;
      const int c = lane % kChunks, step_t = token_of(a, kStep), step_h = kStep - step_t * a.G;
      int token = token_of(a, r0 + lane / kChunks), h = r0 + lane / kChunks - token * a.G;
#pragma unroll 4
      for (int r = lane / kChunks; r < rows; r += kStep) {
        const int head = hk * a.G + h;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) +
                                 ((static_cast<int64_t>(b) * a.T + token) * a.Hq + head) * D)[c] =
            make_uint4(0, 0, 0, 0);
        if (c == 0) a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.T + token] = -INFINITY;
        token += step_t;
        h += step_h;
        if (h >= a.G) {
          h -= a.G;
          ++token;
        }
      }
    };
    if constexpr (SHORT) {
      const int rank = static_cast<int>(cg::this_cluster().block_rank());
      const int ranks = static_cast<int>(cg::this_cluster().num_blocks());
      const int b = cta / ranks / a.Hkv, hk = cta / ranks % a.Hkv;
      const Draft dr = draft(a, b);
      const Unit u = unit_of<kRows>(a, dr, 0);
      const int tile = u.count * rank / ranks, count = u.count * (rank + 1) / ranks - tile;
      const int live = dr.count * a.G;
      if (dr.count < 0 && lane == 0) record_page_error();
      if (u.i1 > u.i0 && count > 0) publish(b, hk, dr, u, 0, live, tile, count, 0);
    } else {
    // Where this CTA's run starts: the cost of the sequences summed up to it. The first 32
    // sequences' stays in registers.
    const Draft dr0 = lane < a.B ? draft(a, lane) : Draft{0, -1};
    const int mine = lane < a.B ? head_cost<kRows>(a, dr0) : 0;
    int total = mine;
#pragma unroll 1
    for (int b = 32 + lane; b < a.B; b += 32) total += head_cost<kRows>(a, draft(a, b));
    total = __reduce_add_sync(0xffffffffu, total) * a.Hkv;
    const int ctas = min(total, static_cast<int>(gridDim.x));   // each gets at least one
    const Runs runs(total, ctas);
    const int start = runs.start(cta);
    int left = cta < ctas ? runs.start(cta + 1) - start : 0;
    limit += static_cast<uint64_t>(left) * 20000;
    int b = 0, at = 0, per_head = 1;
#pragma unroll 1
    for (int b0 = 0, before = 0; b0 < a.B; b0 += 32) {
      const int head = b0 == 0 ? mine : b0 + lane < a.B ? head_cost<kRows>(a, draft(a, b0 + lane)) : 0;
      int inc = head * a.Hkv;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      const unsigned here = __ballot_sync(0xffffffffu, start < before + inc);
      if (here) {   // the first sequence that ends behind it
        const int src = __ffs(here) - 1;
        b = b0 + src;
        per_head = __shfl_sync(0xffffffffu, head, src);
        at = start - before - __shfl_sync(0xffffffffu, inc, src) + per_head * a.Hkv;
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    int hk = at / per_head, rb = 0, taken = 0;
    int pos = at % per_head;   // within the unit's cost, once rb is known
    bool found = false, first = true;
#pragma unroll 1
    while (left > 0) {
      Draft dr;   // (every lane is here)
      if (b < 32) {
        dr.base = __shfl_sync(0xffffffffu, dr0.base, b);
        dr.count = __shfl_sync(0xffffffffu, dr0.count, b);
      } else {
        dr = draft(a, b);
      }
      const Unit u = unit_of<kRows>(a, dr, rb);
      const int cost = cost_of(a, u), before = cost - u.count;
      if (!found && pos >= cost && rb + 1 < a.blocks) {
        pos -= cost;
        ++rb;
        continue;
      }
      found = true;
      // the run's share of the unit's cost, and the tiles in it, which stand at its end
      const int share = min(cost - pos, left);
      const int tile = max(pos - before, 0), count = max(pos + share - before, 0) - tile;
      const int r0 = rb * kRows, rows = min(kRows, a.T * a.G - r0);
      const int live = min(rows, dr.count * a.G - r0);
      const int slot = 2 * cta + (first ? 0 : 1);
      if (dr.count < 0 && lane == 0) record_page_error();
      if (u.i1 > u.i0 && count > 0) {
        publish(b, hk, dr, u, r0, live, tile, count, slot);
        if (!ok) break;
        first = false;
      }
      if (tile == 0 && count > 0) {
        if (a.units && lane == 0) {
          // This run holds the unit's first tile; its last is in the last run that starts before
          // the unit's end.
          const int end = start + taken - pos + cost;
          int last = cta;
          if (count < u.count) {
            last = static_cast<int>(static_cast<float>(end) / static_cast<float>(total) * ctas);
            last = min(max(last, cta), ctas - 1);
            while (runs.start(last) >= end) --last;
            while (last + 1 < ctas && runs.start(last + 1) < end) ++last;
          }
          a.units[(static_cast<int64_t>(b) * a.Hkv + hk) * a.blocks + rb] =
              make_int2(slot, count == u.count ? 0 : last - cta + 1);
        }
        if (u.i1 <= u.i0 && !a.units) clear(b, hk, r0, rows);   // (else the join does)
      }
      left -= share;
      taken += share;
      pos += share;
      if (pos == cost) {
        pos = 0;
        if (++rb == a.blocks) {
          rb = 0;
          if (++hk == a.Hkv) {
            hk = 0;
            ++b;
          }
        }
      }
    }
    }
    if (ok) {   // the end
      const int s = segs % kSegments;
      ok = ptx::wait_bounded_warp(bar(BAR_SEG_EMPTY + s), ((segs / kSegments) & 1) ^ 1, abort_p,
                                  limit);
      if (ok && lane == 0) {
        ms.seg[s].count = 0;
        ptx::mbar_arrive(bar(BAR_SEG_FULL + s));
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------------ producers of K and V
    const bool is_v = warp == 2;
    const CUtensorMap* const map = is_v ? &tm_v : &tm_k;
    const uint32_t ring = base + (is_v ? L::kV : L::kK);
    const int full = is_v ? BAR_V_FULL : BAR_K_FULL, empty = is_v ? BAR_V_EMPTY : BAR_K_EMPTY;
    const int br = a.box_rows, boxes = kTile / br;
    const uint32_t box_bytes = static_cast<uint32_t>(br) * 128;   // 64 columns of its rows
    int n = 0;   // tiles so far: tile n goes through stage n % kStages
    bool ok = true;
#pragma unroll 1
    for (int segs = 0; ok; ++segs) {
      ok = __all_sync(0xffffffffu, segment(segs));
      const Segment& sg = ms.seg[segs % kSegments];
      const int count = ok ? sg.count : 0;
      if (count == 0) break;
      const int row0 = sg.first_key, hk = sg.hk, lo = sg.lo, hi = sg.hi;
      const int total_boxes = count * boxes;
      const int* tab = a.table + static_cast<int64_t>(sg.b) * a.max_pages;
      // Box j holds tokens row0 + j * br ..; lane x keeps the table entries of boxes x, 32 + x,
      // ... one batch of 32 ahead of the loads.
      auto needed = [&](int j) {
        const int r = row0 + j * br;
        return j < total_boxes && r < hi && r + br > lo;
      };
      auto entry = [&](int j) { return needed(j) ? tab[(row0 + j * br) >> a.page_shift] : -1; };
      int cur = entry(lane), nxt = entry(32 + lane);
      if (!is_v && segs > 0) {
        // its Q, which is read when the segment before ends, in some 5 us (146 -> 143 us for the
        // B=8 case; fetched earlier, by the scheduler, it left L2 again)
#pragma unroll 1
        for (int r = lane; r < sg.live; r += 32) {
          const int token = token_of(a, sg.r0 + r);
          const int64_t at = (static_cast<int64_t>(sg.b) * a.T + token) * a.Hq + hk * a.G + sg.r0 + r -
                             token * a.G;
          for (int c = 0; c < D; c += 64) prefetch_l2(static_cast<const uint16_t*>(a.q) + at * D + c);
        }
      }
#pragma unroll 1
      for (int i = 0; i < count; ++i, ++n) {
        const int j0 = i * boxes;
        if (i > 0 && j0 % 32 == 0) {
          cur = nxt;
          nxt = entry(j0 + 32 + lane);
        }
        const int s = n % kStages;
        // lane x < boxes loads box x of this tile
        const int page = __shfl_sync(0xffffffffu, cur, (j0 + lane) % 32);
        const bool need = lane < boxes && needed(j0 + lane);
        const bool load = need && page >= 0 && page < a.num_pages;
        const int r = row0 + (j0 + lane) * br;   // first token of this lane's box
        const unsigned loads = __ballot_sync(0xffffffffu, load);
        if (!ptx::wait_bounded_warp(bar(empty + s), ((n / kStages) & 1) ^ 1, abort_p,
                                    kWaitLimitNs)) {
          ok = false;
          break;
        }
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar(full + s), (D / 64) * box_bytes * __popc(loads));
        __syncwarp();
        const uint32_t dst = ring + s * L::kTileBytes + lane * box_bytes;
        if (load)
          for (int c = 0; c < D / 64; ++c)
            tma_load_5d(dst + c * kHalfBytes, map, bar(full + s), 0, hk,
                        r & ((1 << a.page_shift) - 1), c, page);
        __syncwarp();
        if (!is_v) {
          // what the softmax has to know of the tile
          if (need && !load) record_page_error();
          const int end = load ? lane * br + min(hi - r, br) : 0;
          uint32_t m[4];
#pragma unroll
          for (int w = 0; w < 4; ++w)
            m[w] = __reduce_or_sync(0xffffffffu,
                                    load ? bit_range(lane * br - 32 * w, end - 32 * w) : 0u);
          if (lane == 0) {
            const int k0 = row0 + i * kTile;
            ms.loaded[n % kInfoSlots] = make_uint4(m[0], m[1], m[2], m[3]);
            ms.masked[n % kInfoSlots] = (m[0] & m[1] & m[2] & m[3]) != 0xffffffffu ||
                                        k0 < sg.full_lo || k0 + kTile > sg.full_hi;
            ptx::mbar_arrive(bar(BAR_INFO + n % kInfoSlots));
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) segment_read(segs);
    }
    if (!ok && lane == 0) give_up();
    // Leave no copy in flight (on the normal path these phases completed long ago).
    for (int x = max(0, n - kStages); x < n; ++x)
      ptx::wait_bounded(bar(full + x % kStages), (x / kStages) & 1, abort_p, kWaitLimitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop without a branch on the lane, and one lane's instructions count:
    // descriptors, addresses and counters are then the same for all lanes as the compiler sees it.
    constexpr uint32_t idesc_qk = ptx::idesc_f16(FP16, kTile, kTile, false);
    constexpr uint32_t idesc_pv = ptx::idesc_f16(FP16, kTile, D, true);
    const uint32_t one = elect_one();
    auto wait = [&](int slot, uint32_t parity) {
      return ptx::wait_bounded_warp(bar(slot), parity & 1, abort_p, kWaitLimitNs);
    };
    // (stage and phase of the next K, and of the next V)
    int ks = 0, vs = 0;
    uint32_t kp = 0, vp = 0;
    auto commit = [&](int slot) { commit_if(one, bar(slot)); };
    // S_x = Q K^T of the K stage
    auto issue_s = [&](int x) {
      ptx::tc_fence_after_sync();
      const ptx::SmemDesc q_desc = ptx::smem_desc_sw128_split(
          base + L::kQ + (QT == 2 ? x : 0) * L::kTileBytes, 16, 1024);
      const ptx::SmemDesc k_desc =
          ptx::smem_desc_sw128_split(base + L::kK + ks * L::kTileBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * kHalfBytes + (kk % 4) * 32;
        mma_ss_if(one, x * kTile, q_desc.at(off), k_desc.at(off), idesc_qk, kk > 0);
      }
      commit(BAR_S_FULL + x);
    };
    // O_x (+)= P_x V of the V stage, P_x from TMEM: keys 0 .. 63 in the first 32 columns of S_x, the
    // others in those from 64 on
    auto issue_pv = [&](int x, bool first, bool last) {
      ptx::tc_fence_after_sync();
      const ptx::SmemDesc v_desc =
          ptx::smem_desc_sw128_split(base + L::kV + vs * L::kTileBytes, kHalfBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts_if(one, kTmemO + x * D, x * kTile + (kk / 4) * 64 + (kk % 4) * 8,
                  v_desc.at(kk * 16 * 128), idesc_pv, (!first || kk > 0) ? 1u : 0u);
      if (last) commit(BAR_O_DONE + x);
    };
    auto k_done = [&] {
      commit(BAR_K_EMPTY + ks);
      if (++ks == kStages) {
        ks = 0;
        kp ^= 1;
      }
    };
    auto v_done = [&] {
      commit(BAR_V_EMPTY + vs);
      if (++vs == kStages) {
        vs = 0;
        vp ^= 1;
      }
    };
    uint32_t done0 = 0, done1 = 0;   // tiles of each stream so far
    bool ok = true;
#pragma unroll 1
    for (int segs = 0; ok; ++segs) {
      ok = __all_sync(0xffffffffu, segment(segs));
      const Segment& sg = ms.seg[segs % kSegments];
      const int count = __shfl_sync(0xffffffffu, ok ? sg.count : 0, 0);
      if (count == 0) break;
      const bool b_any = QT == 1 || __shfl_sync(0xffffffffu, sg.live, 0) > kTile;
      __syncwarp();
      if (lane == 0) segment_read(segs);
      ok = wait(BAR_Q_FULL, segs);
      // S of the first tile (one row tile: of the first two), then P V of every tile and S of
      // the stream's next one
#pragma unroll 1
      for (int j = QT == 2 ? -1 : -2; ok && j < count; ++j) {
        const bool s_next = (QT == 2 ? j + 1 : j + 2) < count;
        if (j >= 0) {
          if (!wait(BAR_V_FULL + vs, vp)) { ok = false; break; }
          // O of the segment before has to be out of TMEM
          if (j == 0 && segs > 0 && !wait(BAR_O_FREE, segs - 1)) { ok = false; break; }
        }
        if constexpr (QT == 2) {
          if (j >= 0) {
            if (!wait(BAR_P_FULL + 0, done0++)) { ok = false; break; }
            issue_pv(0, j == 0, !s_next);
          }
          if (s_next) {
            if (!wait(BAR_K_FULL + ks, kp)) { ok = false; break; }
            issue_s(0);
          }
          if (j >= 0) {
            if (b_any) {
              if (!wait(BAR_P_FULL + 1, done1++)) { ok = false; break; }
              issue_pv(1, j == 0, !s_next);
            }
            v_done();
          }
          if (s_next) {
            if (b_any) issue_s(1);
            k_done();
          }
        } else {
          const int x = j & 1;
          if (j >= 0) {
            if (!wait(BAR_P_FULL + x, x ? done1++ : done0++)) { ok = false; break; }
            issue_pv(x, j < 2, !s_next);
            v_done();
          }
          if (s_next) {
            if (!wait(BAR_K_FULL + ks, kp)) { ok = false; break; }
            issue_s(x);
            k_done();
          }
        }
      }
    }
    if (!ok && lane == 0) give_up();
    // Every MMA lane 0 issued has completed before TMEM can be released.
    commit(BAR_MMA_DONE);
    wait(BAR_MMA_DONE, 0);
  } else {
    // ------------------------------------------------------------------ softmax
    const int x = (warp - 4) / 8;                  // stream: 0 = A, 1 = B
    const int half = (warp - 4) / 4 % 2;           // of the tile's keys, and of O's columns
    const int quarter = warp & 3;                  // TMEM lanes [32q, 32q+32)
    const int row = quarter * 32 + lane;           // row within the row tile
    const int my = (QT == 2 ? x * kTile : 0) + row;   // of the unit
    const int tid = threadIdx.x - 128;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * kTile + half * 64;   // this thread's keys of S, then P
    const uint32_t tO = tmem + lane_off + kTmemO;  // O_A; O_B is D columns on
    const float scale = factor_of(a);
    int n0 = 0;               // tiles so far
    int done = 0, ends = 0;   // this stream's tiles and segments with tiles
    bool ok = true;
    // after a wait has run out the loop goes on without data, so that every warp reaches the
    // barriers below
    auto wait = [&](int slot, uint32_t parity, uint64_t limit = kWaitLimitNs) {
      if (ok && !ptx::wait_bounded_warp(bar(slot), parity & 1, abort_p, limit)) {
        ok = false;
        if (lane == 0) give_up();
      }
      return ok;
    };
    // Whether there is a segment s is decided by one warp for all of them, which meet here.
    auto next_segment = [&](int s) {
      if (tid < 32) {
        const bool there = wait(BAR_SEG_FULL + s % kSegments, s / kSegments, segment_limit);
        if (lane == 0) ms.go = there && ms.seg[s % kSegments].count > 0;
      }
      ptx::named_barrier_sync(1, kSoftmaxThreads);
      return ms.go != 0;
    };
    // Q of segment s into shared memory: no S that reads the one before is still to be computed.
    auto load_q = [&](int s) {
      constexpr int kChunks = D / 8, kStep = kSoftmaxThreads / kChunks, kEach = kRows / kStep;
      const Segment& sg = ms.seg[s % kSegments];
      const uint32_t q_and = a.scale_log2 == 0.f ? 0u : ~0u;
      const uint32_t q_xor = a.scale_log2 < 0.f ? 0x80008000u : 0u;
      const int c = tid % kChunks, step_t = token_of(a, kStep), step_h = kStep - step_t * a.G;
      const int live = sg.live, r0 = tid / kChunks;
      int token = token_of(a, sg.r0 + r0), h = sg.r0 + r0 - token * a.G;
      auto next_row = [&] {
        token += step_t;
        h += step_h;
        if (h >= a.G) {
          h -= a.G;
          ++token;
        }
      };
      // the offset of a row's piece in q and o; rows behind the last load the first one's
      const int64_t first = (static_cast<int64_t>(sg.b) * a.T * a.Hq + sg.hk * a.G) * D + c * 8;
      auto place = [&] { return first + static_cast<int64_t>(token * a.Hq + h) * D; };
      const int64_t safe = first + static_cast<int64_t>(token_of(a, sg.r0)) * a.Hq * D;
      uint4 v[kEach];
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        v[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                               (u * kStep + r0 < live ? place() : safe));
        next_row();
      }
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int r = u * kStep + tid / kChunks;
        ptx::st_shared_v4(base + L::kQ + (r / kTile) * L::kTileBytes + (c / 8) * kHalfBytes +
                              r % kTile * 128 + (((c % 8) ^ (r & 7)) << 4),
                          (v[u].x & q_and) ^ q_xor, (v[u].y & q_and) ^ q_xor,
                          (v[u].z & q_and) ^ q_xor, (v[u].w & q_and) ^ q_xor);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(bar(BAR_Q_FULL));
      if (sg.rows > live) {   // the padding's rows
        token = token_of(a, sg.r0 + r0);
        h = sg.r0 + r0 - token * a.G;
#pragma unroll 1
        for (int r = r0; r < sg.rows; r += kStep, next_row()) {
          if (r < live) continue;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + place()) = make_uint4(0, 0, 0, 0);
          if (c == 0)
            a.lse[(static_cast<int64_t>(sg.b) * a.Hq + sg.hk * a.G + h) * a.T + token] = -INFINITY;
        }
      }
    };
    bool go = next_segment(0);
    if (go) load_q(0);
#pragma unroll 1
    for (int segs = 0; go; ++segs) {
      const int live = ms.seg[segs % kSegments].live, count = ms.seg[segs % kSegments].count;
      const bool active = (QT == 2 ? x * kTile : 0) + quarter * 32 < live;   // rows of this warp
      const int j_first = QT == 2 ? 0 : x, j_step = QT == 2 ? 1 : 2;
      const int j_end = QT == 2 && x == 1 && live <= kTile ? 0 : count;
      // offset of the exponents, sum over this thread's keys
      float m = -INFINITY, l = 0.f;

#pragma unroll 1
      for (int j = j_first; j < j_end; j += j_step, ++done) {
        const int n = n0 + j;
        // (a warp that has given up meets its partner all the same)
        const bool known = wait(BAR_INFO + n % kInfoSlots, n / kInfoSlots);
        const bool masked = known && ms.masked[n % kInfoSlots];
        uint32_t vis0 = ~0u, vis1 = ~0u;
        if (masked && active) {
          const Segment& now = ms.seg[segs % kSegments];
          const uint4 loaded = ms.loaded[n % kInfoSlots];
          vis0 = vis1 = 0;
          if (my < now.live) {
            const uint2 vis = visible_bits(a, now.b, now.base, token_of(a, now.r0 + my),
                                           now.first_key + j * kTile + half * 64);
            vis0 = vis.x & (half ? loaded.z : loaded.x);
            vis1 = vis.y & (half ? loaded.w : loaded.y);
          }
          __syncwarp();
        }
        if (!wait(BAR_S_FULL + x, done)) {
          if (active) ptx::named_barrier_sync(2 + x * 4 + quarter, 64);
          continue;
        }
        ptx::tc_fence_after_sync();
        if (active) {
          // S is read twice, for the maximum and for P: kept, it would take the registers of all
          // else
          float mt;
          {
            uint32_t s0[32], s1[32];
            ptx::tmem_ld_32x32b_x32(tS, s0);
            ptx::tmem_ld_32x32b_x32(tS + 32, s1);
            ptx::tmem_wait_ld();
            ptx::reg_fence(s0);
            ptx::reg_fence(s1);
            if (masked) {
#pragma unroll
              for (int t = 0; t < 32; ++t) {
                if (!(vis0 >> t & 1)) s0[t] = 0xff800000u;   // -inf
                if (!(vis1 >> t & 1)) s1[t] = 0xff800000u;
              }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < 32; t += 4) {
              mx[0] = ptx::max3(mx[0], __uint_as_float(s0[t]), __uint_as_float(s0[t + 1]));
              mx[1] = ptx::max3(mx[1], __uint_as_float(s0[t + 2]), __uint_as_float(s0[t + 3]));
              mx[2] = ptx::max3(mx[2], __uint_as_float(s1[t]), __uint_as_float(s1[t + 1]));
              mx[3] = ptx::max3(mx[3], __uint_as_float(s1[t + 2]), __uint_as_float(s1[t + 3]));
            }
            mt = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
          }
          // the row's maximum over both halves (the slots are read before the next S, which the
          // arrivals below let be computed)
          ms.red[x][half][row] = mt;
          ptx::named_barrier_sync(2 + x * 4 + quarter, 64);
          mt = fmaxf(mt, ms.red[x][half ^ 1][row]);
          float alpha = 1.f;
          const bool rescale = __any_sync(0xffffffffu, (mt - m) * scale > kLag<FP16>);
          if (rescale) {
            // every row of this warp to its running maximum; l now, O below
            const float m_new = fmaxf(m, mt);
            alpha = ptx::exp2_approx((m - (m_new == -INFINITY ? 0.f : m_new)) * scale);
            l *= alpha;
            m = m_new;
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          // P over the S of these keys, two of them to a column
          float rs0 = 0.f, rs1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32], pr[16];
            ptx::tmem_ld_32x32b_x32(tS + c * 32, s);
            const uint32_t vis = c ? vis1 : vis0;
            ptx::tmem_wait_ld();
            ptx::reg_fence(s);
            if (masked) {
#pragma unroll
              for (int t = 0; t < 32; ++t)
                if (!(vis >> t & 1)) s[t] = 0xff800000u;
            }
#pragma unroll
            for (int t = 0; t < 16; ++t) {
              float e0, e1;
              ptx::add2(e0, e1, __uint_as_float(s[2 * t]), __uint_as_float(s[2 * t + 1]), -m_use,
                        -m_use);
              ptx::fma2(e0, e1, e0, e1, scale, scale, kShift<FP16>, kShift<FP16>);
              const float p0 = ptx::exp2_approx(e0), p1 = ptx::exp2_approx(e1);
              ptx::add2(rs0, rs1, rs0, rs1, p0, p1);
              pr[t] = pack2<FP16>(p0, p1);
            }
            ptx::tmem_st_32x32b_x16(tS + c * 16, pr);
          }
          l += rs0 + rs1;
          if (rescale && j > j_first) {
            // the product before has completed: it was issued before this S
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              uint32_t orr[32];
              ptx::tmem_ld_32x32b_x32(tO + x * D + half * (D / 2) + c * 32, orr);
              ptx::tmem_wait_ld();
              ptx::reg_fence(orr);
#pragma unroll
              for (int t = 0; t < 32; t += 2) {
                float a0 = __uint_as_float(orr[t]), a1 = __uint_as_float(orr[t + 1]);
                ptx::mul2(a0, a1, a0, a1, alpha, alpha);
                orr[t] = __float_as_uint(a0);
                orr[t + 1] = __float_as_uint(a1);
              }
              ptx::tmem_st_32x32b_x32(tO + x * D + half * (D / 2) + c * 32, orr);
            }
          }
          ptx::tmem_wait_st();
        }
        if (masked && (QT == 1 || x == 0) && wait(BAR_V_FULL + n % kStages, n / kStages)) {
          if (clean_values<D, FP16>(smem_raw + L::kV + (n % kStages) * L::kTileBytes,
                                    ms.loaded[n % kInfoSlots], tid % 256))
            ms.not_finite[segs & 1] = segs + 1;
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before_sync();
        ptx::mbar_arrive(bar(BAR_P_FULL + x));
      }

      // ---- the segment's end. The next one's Q comes first, so that its first S is computed
      // while this one's O leaves.
      if (j_end > j_first) wait(BAR_O_DONE + x, ends++);
      ptx::tc_fence_before_sync();
      go = next_segment(segs + 1);   // (here both streams' products are done)
      ptx::tc_fence_after_sync();
      if (go) load_q(segs + 1);
      // the halves exchange their sums; one row tile: then the streams their offsets and sums
      float fa = 1.f, fb = 0.f;
      if (active) {
        const int pair = 2 + x * 4 + quarter;
        ms.red[x][half][row] = l;
        ptx::named_barrier_sync(pair, 64);
        l += ms.red[x][half ^ 1][row];
        ptx::named_barrier_sync(pair, 64);
        if constexpr (QT == 1) {
          ms.red[x][half][row] = half ? l : m;
          ptx::named_barrier_sync(10 + quarter, 128);
          const float m_a = ms.red[0][0][row], m_b = ms.red[1][0][row];
          m = fmaxf(m_a, m_b);
          const float u = m == -INFINITY ? 0.f : m;
          fa = ptx::exp2_approx((m_a - u) * scale);
          fb = ptx::exp2_approx((m_b - u) * scale);
          l = ms.red[0][1][row] * fa + ms.red[1][1][row] * fb;
          ptx::named_barrier_sync(10 + quarter, 128);
        }
      }
      if (ok && active) {
        const Segment& sn = ms.seg[segs % kSegments];
        const bool whole = sn.whole, two = QT == 1 && sn.count > 1;   // two: both streams have an O
        const bool mine = my < sn.live;
        // (rows behind the last get addresses, too, that nothing is written to)
        const int token = token_of(a, sn.r0 + my), head = sn.hk * a.G + sn.r0 + my - token * a.G;
        const float f = whole ? inverse(l) : 1.f;
        fa *= f;
        fb *= f;
        uint16_t* const o_row = static_cast<uint16_t*>(a.o) +
                                ((static_cast<int64_t>(sn.b) * a.T + token) * a.Hq + head) * D;
        // Where this thread's row of a part goes, and from four columns to the next four.
        float* const part_row =
            SHORT ? short_part + my * 4
                  : a.part_o + (static_cast<int64_t>(sn.slot) * (D / 4) * a.part_rows + my) * 4;
        const int step = (SHORT ? kTile : a.part_rows) * 4;
        const int live_rows = sn.live - (my - lane);   // of this warp's 32
        constexpr int kCols = QT == 2 ? D / 2 : D / 4, kChunk = L::kChunk;
        const int c0 = (QT == 2 ? half : 2 * x + half) * kCols;   // this thread's columns
        // The output of two row tiles: a row's 16-byte pieces are written by consecutive lanes, by
        // way of shared memory (from its own thread each store touches 32 lines: 11000 cycles for
        // 256 rows, not 6000).
        constexpr int kPieces = kChunk / 8;            // of a row's chunk
        uint8_t* const stage = smem_raw + L::kOut + (warp - 4) * (32 * kChunk * 2);
        auto piece = [&](int r, int c) {   // (those of eight rows in different banks)
          return reinterpret_cast<uint4*>(stage + ((r * kPieces + (c ^ ((r >> 2) & 1))) << 4));
        };
#pragma unroll 1
        for (int col = c0; col < c0 + kCols; col += kChunk) {
          uint32_t oa[kChunk], ob[kChunk];
          __syncwarp();
          ptx::tmem_ld_32x32b_x16(tO + (QT == 2 ? x * D : 0) + col, oa);
          if (two) ptx::tmem_ld_32x32b_x16(tO + D + col, ob);
          ptx::tmem_wait_ld();
          ptx::reg_fence(oa);
          if (two) ptx::reg_fence(ob);
          float v[kChunk];
#pragma unroll
          for (int t = 0; t < kChunk; ++t) {
            v[t] = __uint_as_float(oa[t]) * fa;
            if (two) v[t] += __uint_as_float(ob[t]) * fb;
          }
          if (!whole) {
            if (mine) {
#pragma unroll
              for (int t = 0; t < kChunk / 4; ++t)
                *reinterpret_cast<float4*>(part_row + (col / 4 + t) * step) =
                    make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
            }
            continue;
          }
#pragma unroll
          for (int t = 0; t < kPieces; ++t) {
            const uint4 w = make_uint4(
                pack2<FP16>(v[8 * t], v[8 * t + 1]), pack2<FP16>(v[8 * t + 2], v[8 * t + 3]),
                pack2<FP16>(v[8 * t + 4], v[8 * t + 5]), pack2<FP16>(v[8 * t + 6], v[8 * t + 7]));
            if constexpr (QT == 2)
              *piece(lane, t) = w;
            else if (mine)
              *reinterpret_cast<uint4*>(o_row + col + t * 8) = w;
          }
          if constexpr (QT == 2) {
            __syncwarp();
#pragma unroll
            for (int i = lane; i < 32 * kPieces; i += 32) {
              const int r = i / kPieces, c = i % kPieces;
              uint16_t* const to = reinterpret_cast<uint16_t*>(__shfl_sync(
                  0xffffffffu, reinterpret_cast<unsigned long long>(o_row), r));
              if (r < live_rows) *reinterpret_cast<uint4*>(to + col + c * 8) = *piece(r, c);
            }
          }
        }
        __syncwarp();
        if (ms.not_finite[segs & 1] == segs + 1 && mine)
          add_not_finite<FP16>(a, sn, token, D, c0, kCols, whole ? nullptr : part_row, step,
                               whole ? o_row : nullptr);
        if (mine && c0 == 0) {
          if (whole)
            a.lse[(static_cast<int64_t>(sn.b) * a.Hq + head) * a.T + token] =
                lse_at<FP16>(m, l, scale);
          else
            (SHORT ? short_ml + my
                   : a.part_ml + static_cast<int64_t>(sn.slot) * a.part_rows + my)[0] =
                make_float2(m, l);
        }
      }
      n0 += ms.seg[segs % kSegments].count;
      __syncwarp();
      if (lane == 0) segment_read(segs);
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(bar(BAR_O_FREE));
    }
  }

  if constexpr (SHORT) {
    // ------------------------------------------------------------------ join
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int ranks = static_cast<int>(cluster.num_blocks());
    const int b = cta / ranks / a.Hkv, hk = cta / ranks % a.Hkv;
    const Draft dr = draft(a, b);
    const int live = dr.count * a.G, tiles = unit_of<kRows>(a, dr, 0).count;
    // The CTAs with tiles, as bits. Each of them counts, one whose scores are all NaN (its maximum is
    // -inf, its sum is not 0) and one with infinite values as well; the others wrote nothing.
    unsigned parts = 0;
    if (live > 0)
      for (int x = 0; x < ranks; ++x)
        if (tiles * x / ranks < tiles * (x + 1) / ranks) parts |= 1u << x;
    __syncwarp();
    cluster.sync();   // every CTA's part is in its shared memory
    // four columns of a row a thread, the rows shared out over the cluster (a sequence without
    // drafted tokens has nothing but padding, which no segment wrote)
    const int rows = live > 0 ? live : a.T * a.G;
    const float scale = factor_of(a);
#pragma unroll 1
    for (int at = rank * kThreads + threadIdx.x; at < (rows + 7) / 8 * 8 * (D / 4);
         at += ranks * kThreads) {
      // (a part's rows are next to one another, an output's columns)
      const int r = at / (8 * (D / 4)) * 8 + at % 8, c = at / 8 % (D / 4);
      if (r >= rows) continue;
      float m = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int x = 0; x < ranks; ++x) {
        if (!(parts >> x & 1)) continue;
        const float2 ml = *cluster.map_shared_rank(short_ml + r, x);
        const float4 v =
            *reinterpret_cast<const float4*>(cluster.map_shared_rank(short_part + (c * kTile + r) * 4, x));
        const float most = fmaxf(m, ml.x), top = most == -INFINITY ? 0.f : most;
        const float f = ptx::exp2_approx((m - top) * scale);
        const float g = ptx::exp2_approx((ml.x - top) * scale);
        m = most;
        l = l * f + ml.y * g;
        acc.x = acc.x * f + v.x * g;
        acc.y = acc.y * f + v.y * g;
        acc.z = acc.z * f + v.z * g;
        acc.w = acc.w * f + v.w * g;
      }
      const float inv = inverse(l);
      const int token = token_of(a, r), head = hk * a.G + r - token * a.G;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) +
                                ((static_cast<int64_t>(b) * a.T + token) * a.Hq + head) * D + 4 * c) =
          make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
      if (c == 0)
        a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.T + token] = lse_at<FP16>(m, l, scale);
    }
    __syncwarp();
    cluster.sync();   // no CTA leaves while another reads its part
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(ms.tmem_base, kTmemCols);
  }
}

// The parts of a unit that more than one run covers, joined: a thread for four columns of a row, a
// block for 1024 / D consecutive rows of a key head. The part in the first run's slot is followed by
// those of the next CTAs, each in its CTA's first slot.
constexpr int kJoinThreads = 256;
template <int D>
constexpr int kJoinRows = kJoinThreads / (D / 4);

template <int D, bool FP16, int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    fa_paged_tree_join_kernel(const __grid_constant__ Args a, int blocks_per_head) {
  wait_prerequisites();
  launch_dependents();
  const int head = blockIdx.x / blocks_per_head;   // sequence and key head
  const int r = blockIdx.x % blocks_per_head * kJoinRows<D> + threadIdx.x % kJoinRows<D>;
  if (r >= a.T * a.G) return;
  const int b = head / a.Hkv, hk = head % a.Hkv, col = threadIdx.x / kJoinRows<D>, my = r % ROWS;
  const int i = token_of(a, r), h = hk * a.G + r - i * a.G;
  const int2 u = a.units[static_cast<int64_t>(head) * a.blocks + r / ROWS];
  const int drafted = draft(a, b).count;
  uint2* const dst = reinterpret_cast<uint2*>(
      static_cast<uint16_t*>(a.o) + ((static_cast<int64_t>(b) * a.T + i) * a.Hq + h) * D + 4 * col);
  float* const lse = a.lse + (static_cast<int64_t>(b) * a.Hq + h) * a.T + i;
  if (i >= drafted) {
    // padding: of a unit without any token nobody else writes it
    if (token_of(a, r - my) >= drafted) {
      *dst = make_uint2(0, 0);
      if (col == 0) *lse = -INFINITY;
    }
    return;
  }
  if (u.y == 0) return;   // one run's, and written
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const float scale = factor_of(a);
#pragma unroll 4
  for (int p = 0; p < u.y; ++p) {
    const int64_t slot = p == 0 ? u.x : 2 * (u.x / 2 + p);
    const float2 ml = a.part_ml[slot * a.part_rows + my];
    const float4 f = *reinterpret_cast<const float4*>(
        a.part_o + ((slot * (D / 4) + col) * a.part_rows + my) * 4);
    const float n = fmaxf(m, ml.x), top = n == -INFINITY ? 0.f : n;
    const float old = ptx::exp2_approx((m - top) * scale);
    const float now = ptx::exp2_approx((ml.x - top) * scale);
    m = n;
    l = l * old + ml.y * now;
    acc.x = acc.x * old + f.x * now;
    acc.y = acc.y * old + f.y * now;
    acc.z = acc.z * old + f.z * now;
    acc.w = acc.w * old + f.w * now;
  }
  const float inv = inverse(l);
  *dst = make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
  if (col == 0) *lse = lse_at<FP16>(m, l, scale);
}

// Row tiles of a unit, and with it its rows: two where a key head has more than 128 rows.
int row_tiles(int T, int Hq, int Hkv) { return static_cast<int64_t>(T) * (Hq / Hkv) > kTile ? 2 : 1; }

// The smallest calls: 0, or the CTAs of a cluster that has one unit. A unit of up to kShortTiles
// tiles for each CTA of a cluster, and few enough units that all clusters run at once, takes one
// launch without a workspace: 8 units of 1009 tokens (d=64) 10.3 us a replay instead of 14.2, and a
// launch less for the caller. Units of one CTA may take a second turn.
constexpr int kShortTiles = 4;
int resident_clusters(int ctas) {   // of one CTA on each SM, as the runtime counts them on a GB300
  return ctas == 8 ? 15 : ctas == 4 ? 36 : ctas == 2 ? 76 : 152;
}
int choose_short(int B, int T, int Hq, int Hkv, int64_t tiles) {
  if (row_tiles(T, Hq, Hkv) > 1) return 0;
  const int64_t units = static_cast<int64_t>(B) * Hkv;
  for (int ctas = 8; ctas >= 2; ctas /= 2)
    if (units <= resident_clusters(ctas) && ctas / 2 < tiles)
      return tiles <= ctas * kShortTiles ? ctas : 0;
  return units <= 2 * resident_clusters(1) && tiles <= kShortTiles ? 1 : 0;
}

// What a unit's start and end cost in a run, in tiles: of 3 to 16 the best, or within 1 % of it, for 32
// to 256 units is 6 (64 units of up to 32K tokens 117.6 us and, with two row tiles, 138.4; with 8 118.8
// and 138.8). Where few CTAs have such a step, the bandwidth that it leaves goes to the others and is
// missing at the end: 16 units of up to 64K tokens 67.4 us, with 8 65.0; 8 units 60.7 and 60.3.
// 512 units of up to 4096 tokens would take 130.5 us with 4 instead of 133: a third value for 2 %.
int unit_cost(int64_t units) { return units <= 16 ? 8 : 6; }

// Workspace: the parts' O, their offsets and sums, the units' parts; nothing where a unit is one
// tile, and never split.
struct Layout {
  int64_t ctas, blocks, part_rows;
  bool join;
  size_t part_ml, units, end;
};
Layout layout(int B, int T, int Hq, int Hkv, int d, int64_t capacity) {
  Layout l;
  const int64_t rows = static_cast<int64_t>(T) * (Hq / Hkv), unit = row_tiles(T, Hq, Hkv) * kTile;
  l.blocks = (rows + unit - 1) / unit;
  l.part_rows = std::min(rows, unit);
  l.ctas = std::min<int64_t>(kSms, B * Hkv * l.blocks * ((capacity + kTile - 1) / kTile));
  l.join = capacity > kTile;
  l.part_ml = static_cast<size_t>(2 * l.ctas * l.part_rows * d) * 4;
  l.units = l.part_ml + static_cast<size_t>(2 * l.ctas * l.part_rows) * 8;
  l.end = l.join ? l.units + static_cast<size_t>(B * Hkv * l.blocks) * 8 : 0;
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
  a.units = l.join ? reinterpret_cast<int2*>(ws + l.units) : nullptr;
  a.B = c.B;
  a.T = p.T;
  a.Hq = p.Hq;
  a.Hkv = c.Hkv;
  a.G = p.Hq / c.Hkv;
  a.g_magic = a.G > 1 && a.G < 2048 ? static_cast<uint32_t>(((1ull << 32) + a.G - 1) / a.G) : 0;
  a.blocks = static_cast<int>(l.blocks);
  a.part_rows = static_cast<int>(l.part_rows);
  a.page_shift = shift_of(c.page_size);
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.box_rows = std::min(c.page_size, kTile);
  a.window_left = p.window_left;
  a.unit_cost = unit_cost(static_cast<int64_t>(c.B) * c.Hkv * l.blocks);
  a.scale_log2 = p.scale_log2;
  CUtensorMap tm_k, tm_v;
  if (!encode_pages(&tm_k, c.k_pages, c, a.box_rows, 1, FP16) ||
      !encode_pages(&tm_v, c.v_pages, c, a.box_rows, 1, FP16))
    return cudaErrorInvalidValue;
  const int smem = static_cast<int>(Smem<D, QT>::kDynamic);
  if constexpr (QT == 1) {
    if (const int cluster = choose_short(c.B, p.T, p.Hq, c.Hkv, (capacity + kTile - 1) / kTile)) {
      auto kernel = fa_paged_tree_kernel<D, FP16, 1, true>;
      const cudaError_t err =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err != cudaSuccess) return err;
      return launch_paged(kernel, static_cast<int64_t>(c.B) * c.Hkv * cluster, kThreads, smem,
                          stream, cluster > 1 ? cluster : 0, tm_k, tm_v, a);
    }
  }
  auto kernel = fa_paged_tree_kernel<D, FP16, QT, false>;
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  err = launch_paged(kernel, l.ctas, kThreads, smem, stream, 0, tm_k, tm_v, a);
  if (err != cudaSuccess || !l.join) return err;
  const int per_head = (p.T * a.G + kJoinRows<D> - 1) / kJoinRows<D>;
  return launch_paged(fa_paged_tree_join_kernel<D, FP16, QT * kTile>,
                      static_cast<int64_t>(c.B) * c.Hkv * per_head, kJoinThreads, 0, stream, 0, a,
                      per_head);
}

template <int D, bool FP16>
cudaError_t launch_rows(const TreeParams& p, cudaStream_t stream) {
  return row_tiles(p.T, p.Hq, p.c.Hkv) == 1 ? launch_impl<D, FP16, 1>(p, stream)
                                            : launch_impl<D, FP16, 2>(p, stream);
}

}  // namespace

size_t paged_tree_workspace(int B, int T, int Hq, int Hkv, int d, int page_size, int max_pages) {
  const int64_t capacity = static_cast<int64_t>(max_pages) * page_size;
  if (choose_short(B, T, Hq, Hkv, (capacity + kTile - 1) / kTile)) return 0;
  return layout(B, T, Hq, Hkv, d, capacity).end;
}

cudaError_t launch_paged_tree(const TreeParams& p, cudaStream_t stream) {
  if (p.c.d == 64)
    return p.fp16 ? launch_rows<64, true>(p, stream) : launch_rows<64, false>(p, stream);
  return p.fp16 ? launch_rows<128, true>(p, stream) : launch_rows<128, false>(p, stream);
}

cudaError_t read_and_clear_tree_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
