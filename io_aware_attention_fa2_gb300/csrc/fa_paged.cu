// fa_paged.cu -- the paged key-value cache: append and evict (include/fa.h has the layouts and
// the rules for bad block-table entries and lengths).
#include <cooperative_groups.h>

#include <algorithm>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;

constexpr int kErrTimeout = -8, kErrPage = -13;   // FA_ERR_TIMEOUT, FA_ERR_PAGE

// Page of the table entry at `at`, or -1 (recorded) when it is outside the pool.
__device__ __forceinline__ int page_at(const int* table, int64_t at, int num_pages) {
  const int page = table[at];
  if (page >= 0 && page < num_pages) return page;
  record_page_error();
  return -1;
}

// ---------------------------------------------------------------------------------------------
// Append. A copy, bound by HBM: one block for each new token, whose Hkv * d values are contiguous
// in both layouts, so that a page's address is looked up once a token and all accesses are whole
// 16-byte rows. Four prompts of up to 8192 tokens, Hkv=16 d=128 with weights (436 MB): 71 us,
// 6.1 TB/s, 90 % of the measured copy rate. One token of 16 sequences: 4.2 us.
__global__ void __launch_bounds__(128)
    fa_paged_append_kernel(const uint4* k, const uint4* v, const float* w, uint4* k_pages,
                           uint4* v_pages, float* weights, const int* table, const int* seqlens,
                           const int* new_lens, int N, int Hkv, int d, int page_size,
                           int num_pages, int max_pages) {
  wait_prerequisites();
  launch_dependents();
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
    const uint4 kc = k[src + c], vc = v[src + c];   // both loads before the stores
    k_pages[dst + c] = kc;
    v_pages[dst + c] = vc;
  }
  if (weights)
    for (int h = threadIdx.x; h < Hkv; h += blockDim.x)
      weights[(static_cast<int64_t>(page) * Hkv + h) * page_size + row] =
          w ? w[(static_cast<int64_t>(b) * Hkv + h) * N + i] : 0.f;
}

// ---------------------------------------------------------------------------------------------
// Evict, in two kernels: which tokens stay (kept), then their move. What has to be read and
// written is the weights (4 bytes a token) and the kept rows once each way (4 d bytes a token).
//
// Selection, for each (sequence, key head): the want-th largest weight among the tokens before
// the recent ones, by radix selection on the weights as ordered 32-bit keys (digits of 11, 11
// and 10 bits), then the equal ones from the oldest until there are enough. The keys are read
// once and kept in shared memory. The move is bound by HBM, the selection by instructions and
// latency: eight sequences of up to 32768 tokens to 4096, Hkv=8 d=128 (277 MB): 65 us, of which
// the selection 19 (64 CTAs) and the move 47 (268 MB, 85 % of the measured copy rate). In the
// selection: weights and tables 5 us, histograms 2.6 + 2.1 + 1.7, counting 1.7, placing 4.8.
// Measured slower: one kernel of eight CTAs for each head that selects and moves (134 us; 3 us
// for every exchange of a histogram); several copies of the histogram against equal bins (+1 us);
// a token a lane with two ballots (+0.5 us); a run of tokens for each thread (67 instead of 68 us
// a replay here, but 99 instead of 86 where 300000 tokens have the heavy ones side by side: each
// lane writes to lines of its own).
namespace cg = cooperative_groups;

struct EvictArgs {
  uint4* k_pages;
  uint4* v_pages;
  float* weights;
  const int* table;
  const int* seqlens;
  const int* out_table;
  int* kept;
  int* new_seqlens;
  int Hkv, page_shift, num_pages, max_pages, out_pages, budget, recent;   // 2^page_shift tokens
};

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048, kBinsPerThread = kBins / kSelectThreads;
constexpr int kMaxCache = 49152;   // keys a CTA keeps in shared memory; further ones are read from
                                   // the pages in every pass

// Weights as unsigned numbers in the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void copy_async_16(uint4* to, const float* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void wait_async_copies() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Checks of a sequence's tables, by all threads of a block: `bad` when a page is outside the pool
// or a page of dst stands in src at a later place, `own` when one stands in src at all. Warp w of
// `warps` that share dst takes every warps-th entry. `bits`: kBins words of shared memory, zero
// before; they get a bit for each page of src, so that only entries of dst that may be in src at
// another place are looked for (src and dst have thousands of entries each for long sequences).
struct TableChecks {
  bool bad, own;
};
__device__ __forceinline__ TableChecks check_tables(const int* src, int src_used, const int* dst,
                                                    int dst_used, int num_pages, int w, int warps,
                                                    uint32_t* bits) {
  const int lane = threadIdx.x % 32;
  TableChecks c{false, false};
  for (int j = threadIdx.x; j < src_used; j += blockDim.x) {
    const int page = src[j];
    if (page < 0 || page >= num_pages)
      c.bad = true;
    else
      atomicOr(&bits[(page >> 5) & (kBins - 1)], 1u << (page & 31));
  }
  __syncthreads();
  for (int i = w; i < dst_used; i += warps) {   // dst_used <= src_used
    const int page = dst[i];
    if (page < 0 || page >= num_pages) {
      c.bad = true;
    } else if (src[i] == page) {
      c.own = true;
    } else if (bits[(page >> 5) & (kBins - 1)] >> (page & 31) & 1) {
      for (int j = lane; j < src_used; j += 32)
        if (src[j] == page) {
          c.own = true;
          if (j > i) c.bad = true;
        }
    }
  }
  return c;
}

// CTAS CTAs (a cluster) for each (sequence, key head), each with its share of the candidates:
// the flags, histograms and counts are exchanged through distributed shared memory. One CTA
// needs no exchange, which costs 3 us a digit. `cache` keys fit in the dynamic shared memory.
template <int CTAS>
__global__ void __launch_bounds__(kSelectThreads, 1)
    fa_paged_select_kernel(const __grid_constant__ EvictArgs a, int cache_keys) {
  extern __shared__ __align__(16) uint32_t smem[];   // groups of four keys behind the histograms
  uint32_t* const hist = smem;                            // [kBins] (two of them with a cluster)
  __shared__ uint32_t s_warp[kSelectWarps], s_found[2];
  __shared__ int2 s_count, s_warp_count[kSelectWarps];   // candidates above and at the threshold
  __shared__ int s_bad;                                  // flag of this CTA's share of the checks
  const int rank = CTAS > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int wide = rank * kSelectThreads + tid, width = CTAS * kSelectThreads;
  // all CTAs of the unit: shared memory written before is readable in the others after
  auto sync_all = [&] {
    if constexpr (CTAS > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  auto of_rank = [&](auto* p, int r) {
    if constexpr (CTAS > 1)
      return cg::this_cluster().map_shared_rank(p, r);
    else
      return p;
  };
  const int64_t unit = blockIdx.x / CTAS;
  const int b = static_cast<int>(unit / a.Hkv), hk = static_cast<int>(unit % a.Hkv);
  const int* const src_table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int* const dst_table = a.out_table + static_cast<int64_t>(b) * a.out_pages;
  int* const kept = a.kept + unit * a.budget;
  wait_prerequisites();
  launch_dependents();

  const int raw_len = a.seqlens[b];
  const bool bad_len = raw_len < 0 || raw_len > a.max_pages << a.page_shift;
  const int len = bad_len ? 0 : raw_len, new_len = min(len, a.budget);
  auto in_pool = [&](int page) { return page >= 0 && page < a.num_pages; };
  if (tid == 0) s_bad = bad_len;
  for (int i = tid; i < (CTAS > 1 ? 2 : 1) * kBins; i += kSelectThreads) hist[i] = 0;
  __syncthreads();

  const bool select = len > a.budget;
  const int n = select ? len - a.recent : 0;         // candidates: tokens [0, n)
  uint32_t want = select ? a.budget - a.recent : 0;  // of them stay
  // this CTA's: [t0, t0 + mine), in groups of four, which lie in one page
  const int share = (n + 4 * CTAS - 1) / (4 * CTAS) * 4;
  const int t0 = min(rank * share, n), mine = min(share, n - t0);
  const int groups = (mine + 3) / 4, cached = min(groups, cache_keys / 4);
  uint4* const cache = reinterpret_cast<uint4*>(smem + (CTAS > 1 ? 2 : 1) * kBins);
  const int in_page = (1 << a.page_shift) - 1;
  auto group_at = [&](int g, int page) {
    const int t = t0 + 4 * g;
    return a.weights + ((static_cast<int64_t>(page) * a.Hkv + hk) << a.page_shift) + (t & in_page);
  };
  // Behind the last candidate the lowest key: it has no smaller ones to count it before, and of
  // equal ones it comes after all candidates, so that it needs no test anywhere.
  auto keys_of = [&](int i, float4 w) {
    return make_uint4(order_key(w.x), i + 1 < mine ? order_key(w.y) : 0u,
                      i + 2 < mine ? order_key(w.z) : 0u, i + 3 < mine ? order_key(w.w) : 0u);
  };
  auto load_group = [&](int g) {
    return keys_of(4 * g, *reinterpret_cast<const float4*>(
                              group_at(g, src_table[(t0 + 4 * g) >> a.page_shift])));
  };
  // The weights are on their way while the tables are checked. (With a page outside the pool
  // the sequence is given up below, and nothing reads the group.)
#pragma unroll 8
  for (int g = tid; g < cached; g += kSelectThreads) {
    const int page = src_table[(t0 + 4 * g) >> a.page_shift];
    if (in_pool(page)) copy_async_16(cache + g, group_at(g, page));
  }
  if (check_tables(src_table, (len + in_page) >> a.page_shift, dst_table,
                   (new_len + in_page) >> a.page_shift, a.num_pages, rank * kSelectWarps + warp,
                   CTAS * kSelectWarps, hist)
          .bad)
    s_bad = 1;
  __syncthreads();
  for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;   // (counted in after sync_all)
  wait_async_copies();   // of this thread, which is the one that makes keys of them
  // f(first token of the group within this CTA's, its four keys), group g of every `step`
  auto for_groups = [&](int g0, int g1, int step, auto&& f) {
    int g = g0;
#pragma unroll 4
    for (; g < min(g1, cached); g += step) f(4 * g, cache[g]);
    for (; g < g1; g += step) f(4 * g, load_group(g));
  };

  sync_all();
  int bad = 0;
#pragma unroll
  for (int r = 0; r < CTAS; ++r) bad |= *of_rank(&s_bad, r);
  if (bad) {
    for (int i = wide; i < a.budget; i += width) kept[i] = -1;
    if (wide == 0) {
      record_page_error();
      if (hk == 0) a.new_seqlens[b] = raw_len;
    }
    if constexpr (CTAS > 1) sync_all();   // no CTA leaves while another reads its flag
    return;
  }
  if (wide == 0 && hk == 0) a.new_seqlens[b] = new_len;

  uint32_t prefix = 0;   // digits found so far
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0};
    const int shift = kShift[pass], bits = pass == 2 ? 10 : 11;
    uint32_t* const h = hist + (CTAS > 1 ? (pass & 1) * kBins : 0);
    auto count_key = [&](uint32_t key) {
      if (pass == 0 || (key >> (shift + bits)) == prefix)
        atomicAdd(&h[(key >> shift) & ((1u << bits) - 1)], 1u);
    };
    if (want)
      for_groups(tid, groups, kSelectThreads, [&](int i, uint4 key) {
        if (pass == 0 && i < 4 * cached) {
          key = keys_of(i, make_float4(__uint_as_float(key.x), __uint_as_float(key.y),
                                       __uint_as_float(key.z), __uint_as_float(key.w)));
          cache[i / 4] = key;
        }
        count_key(key.x);
        count_key(key.y);
        count_key(key.z);
        count_key(key.w);
      });
    sync_all();
    if (want) {
      // two bins a thread, from the top; `before`: the keys in the bins of earlier threads
      const int top = kBins - kBinsPerThread * (tid + 1);
      uint32_t high = 0, low = 0;
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        const uint2 x = *reinterpret_cast<const uint2*>(of_rank(h + top, r));
        low += x.x;
        high += x.y;
      }
      uint32_t inc = high + low;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      uint32_t before = lane < warp ? s_warp[lane] : 0u;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
      before += inc - high - low;
      if (before < want && want <= before + high + low) {
        const bool is_high = want <= before + high;
        s_found[0] = top + (is_high ? 1 : 0);
        s_found[1] = is_high ? before : before + high;
      }
    }
    // a cluster's third pass takes the first histogram again, which every CTA has read by now
    if (pass < 2 && (CTAS == 1 || pass == 1))
      for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    if (want) {
      prefix = prefix << bits | s_found[0];
      want -= s_found[1];   // of the keys that start with prefix
    }
  }

  if (!select) {
    for (int i = wide; i < a.budget; i += width) kept[i] = i < len ? i : -1;
    if constexpr (CTAS > 1) sync_all();
    return;
  }
  // The tokens above the threshold and the oldest `want` at it, in order: every warp counts a
  // run of its own, then places it behind the runs before.
  const int limit = static_cast<int>(want);
  if (a.budget > a.recent) {
    const int per_warp = (groups + kSelectThreads - 1) / kSelectThreads * 32;
    const int g0 = min(warp * per_warp, groups), g1 = min(g0 + per_warp, groups);
    // keys above the threshold in the low half, at it in the high half: at most 4 of a group
    auto count4 = [&](uint4 key) {
      uint32_t c = 0;
      for (uint32_t k : {key.x, key.y, key.z, key.w})
        c += k > prefix ? 1u : k == prefix ? 0x10000u : 0u;
      return c;
    };
    int2 count = make_int2(0, 0);
    for_groups(g0 + lane, g1, 32, [&](int, uint4 key) {
      const uint32_t c = count4(key);
      count.x += c & 0xffff;
      count.y += c >> 16;
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      count.x += __shfl_xor_sync(0xffffffffu, count.x, off);
      count.y += __shfl_xor_sync(0xffffffffu, count.y, off);
    }
    if (lane == 0) s_warp_count[warp] = count;
    __syncthreads();
    const int2 of_lane = s_warp_count[lane];
    int above = lane < warp ? of_lane.x : 0, equal = lane < warp ? of_lane.y : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      above += __shfl_xor_sync(0xffffffffu, above, off);
      equal += __shfl_xor_sync(0xffffffffu, equal, off);
    }
    if constexpr (CTAS > 1) {
      if (tid == kSelectThreads - 1) s_count = make_int2(above + count.x, equal + count.y);
      sync_all();
      for (int r = 0; r < rank; ++r) {
        const int2 c = *of_rank(&s_count, r);
        above += c.x;
        equal += c.y;
      }
    }
    // a group a lane: its place comes from a scan of the groups' counts
    for (int g = g0; g < g1; g += 32) {
      const int at = g + lane;
      uint4 key = make_uint4(0, 0, 0, 0);
      uint32_t c = 0;
      if (at < g1) {
        key = at < cached ? cache[at] : load_group(at);
        c = count4(key);
      }
      uint32_t inc = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
      if (c) {   // the lane's kept tokens are consecutive ones
        int same = equal + static_cast<int>((inc - c) >> 16), token = t0 + 4 * at;
        int* to = kept + above + static_cast<int>((inc - c) & 0xffff) + min(same, limit);
        for (uint32_t k : {key.x, key.y, key.z, key.w}) {
          const bool level = k == prefix;
          if (k > prefix || (level && same < limit)) *to++ = token;
          same += level;
          ++token;
        }
      }
      above += static_cast<int>(all & 0xffff);
      equal += static_cast<int>(all >> 16);
    }
  }
  for (int i = wide; i < a.recent; i += width) kept[a.budget - a.recent + i] = n + i;
  if constexpr (CTAS > 1) sync_all();   // no CTA leaves while another reads its counts
}

// The move: kept token i goes to row i of out_table's pages. A cluster of eight CTAs for each
// (sequence, key head), in rounds of the cluster's width. Where out_table names pages of the
// sequence itself, a cluster barrier between a round's reads and its writes keeps the order: a
// token's new place is never behind its old one, so a later round's sources lie behind every
// earlier destination. Reads go past L1: a row may share its line with one that another SM
// writes.
constexpr int kMoveThreads = 512, kMoveCluster = 8;
constexpr int kMoveTokens = 8;   // 16-byte loads in flight for each lane

template <int D>
__global__ void __cluster_dims__(kMoveCluster, 1, 1) __launch_bounds__(kMoveThreads, 2)
    fa_paged_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kLanes = D / 4;   // a row's K and V, 16 bytes a lane
  constexpr int kTokens = 32 / kLanes * kMoveTokens;   // tokens of a warp in a round
  constexpr int kWarps = kMoveThreads / 32, kRound = kTokens * kWarps * kMoveCluster;
  __shared__ int s_own;
  __shared__ uint32_t s_bits[kBins];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t unit = blockIdx.x / kMoveCluster;
  const int b = static_cast<int>(unit / a.Hkv), hk = static_cast<int>(unit % a.Hkv);
  const int* const src_table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int* const dst_table = a.out_table + static_cast<int64_t>(b) * a.out_pages;
  const int* const kept = a.kept + unit * a.budget;
  const int shift = a.page_shift, in_page = (1 << shift) - 1;
  // whether a destination is a page of the sequence (on the arguments alone: this runs beside
  // the selection)
  const int len = min(max(a.seqlens[b], 0), a.max_pages << shift), new_len = min(len, a.budget);
  const int src_used = (len + in_page) >> shift, dst_used = (new_len + in_page) >> shift;
  if (tid == 0) s_own = 0;
  for (int i = tid; i < kBins; i += kMoveThreads) s_bits[i] = 0;
  __syncthreads();
  if (check_tables(src_table, src_used, dst_table, dst_used, a.num_pages, rank * kWarps + warp,
                   kMoveCluster * kWarps, s_bits)
          .own)
    s_own = 1;
  cluster.sync();
  int own_pages = 0;
#pragma unroll
  for (int r = 0; r < kMoveCluster; ++r) own_pages |= *cluster.map_shared_rank(&s_own, r);
  cluster.sync();   // no CTA leaves while another reads its flag
  wait_prerequisites();
  // (a sequence that was given up keeps nothing: its kept is all -1)
  const int rows = new_len > 0 && load_l2(kept) >= 0 ? new_len : 0;

  const int part = lane % kLanes;
  const int64_t chunk = part % (D / 8);
  uint4* const pool = part < D / 8 ? a.k_pages : a.v_pages;
  for (int r0 = 0; r0 < rows; r0 += kRound) {
    // lane e < kTokens looks up token i0 + e
    const int i = r0 + (rank * kWarps + warp) * kTokens + lane;
    int64_t src = -1, dst = -1, w_dst = 0;
    float w = 0.f;
    if (lane < kTokens && i < rows) {
      const int t = load_l2(kept + i);
      const int64_t src_page = src_table[t >> shift], dst_page = dst_table[i >> shift];
      const int src_row = t & in_page, dst_row = i & in_page;
      src = (((src_page << shift) + src_row) * a.Hkv + hk) * (D / 8);
      dst = (((dst_page << shift) + dst_row) * a.Hkv + hk) * (D / 8);
      if (src == dst) {   // in place already
        src = -1;
      } else {
        w = load_l2(a.weights + ((src_page * a.Hkv + hk) << shift) + src_row);
        w_dst = ((dst_page * a.Hkv + hk) << shift) + dst_row;
      }
    }
    uint4 v[kMoveTokens];
#pragma unroll
    for (int u = 0; u < kMoveTokens; ++u) {
      const int64_t from = __shfl_sync(0xffffffffu, src, u * (32 / kLanes) + lane / kLanes);
      if (from >= 0) v[u] = load_l2(pool + from + chunk);
    }
    if (own_pages) cluster.sync();
#pragma unroll
    for (int u = 0; u < kMoveTokens; ++u) {
      const int e = u * (32 / kLanes) + lane / kLanes;
      const int64_t from = __shfl_sync(0xffffffffu, src, e);
      const int64_t to = __shfl_sync(0xffffffffu, dst, e);
      if (from >= 0) pool[to + chunk] = v[u];
    }
    if (src >= 0) a.weights[w_dst] = w;
  }
}

template <int CTAS>
cudaError_t launch_select(const EvictArgs& a, int64_t units, cudaStream_t stream) {
  // the longest share of candidates a CTA can get
  const int64_t most =
      ((static_cast<int64_t>(a.max_pages) << a.page_shift) + 4 * CTAS - 1) / (4 * CTAS) * 4;
  const int cache_keys = static_cast<int>(std::min<int64_t>(most, kMaxCache));
  constexpr int kHist = (CTAS > 1 ? 2 : 1) * kBins;
  const int smem = (kHist + cache_keys) * 4;
  auto kernel = fa_paged_select_kernel<CTAS>;
  // the limit is the function's, not the launch's: the same for all calls, which may overlap
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kHist + kMaxCache) * 4);
  if (err != cudaSuccess) return err;
  return launch_chained(kernel, units * CTAS, kSelectThreads, smem, stream, CTAS > 1 ? CTAS : 0, a,
                        cache_keys);
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  return launch_chained(
      fa_paged_append_kernel, static_cast<int64_t>(c.B) * p.N, 128, 0, stream, 0,
      static_cast<const uint4*>(p.k), static_cast<const uint4*>(p.v), p.w,
      static_cast<uint4*>(c.k_pages), static_cast<uint4*>(c.v_pages), c.weights, c.block_table,
      c.seqlens, p.new_lens, p.N, c.Hkv, c.d, c.page_size, c.num_pages, c.max_pages);
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  EvictArgs a;
  a.k_pages = static_cast<uint4*>(c.k_pages);
  a.v_pages = static_cast<uint4*>(c.v_pages);
  a.weights = c.weights;
  a.table = c.block_table;
  a.seqlens = c.seqlens;
  a.out_table = p.out_table;
  a.kept = p.kept;
  a.new_seqlens = p.new_seqlens;
  a.Hkv = c.Hkv;
  a.page_shift = 0;
  while (1 << a.page_shift < c.page_size) ++a.page_shift;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.out_pages = p.out_pages;
  a.budget = p.budget;
  a.recent = p.recent;
  const int64_t units = static_cast<int64_t>(c.B) * c.Hkv;
  // One CTA for a head's selection while its tokens fit in its shared memory, else eight.
  cudaError_t err = static_cast<int64_t>(c.max_pages) * c.page_size <= kMaxCache
                        ? launch_select<1>(a, units, stream)
                        : launch_select<8>(a, units, stream);
  if (err != cudaSuccess) return err;
  return launch_chained(c.d == 64 ? fa_paged_move_kernel<64> : fa_paged_move_kernel<128>,
                        units * kMoveCluster, kMoveThreads, 0, stream, 0, a);
}

cudaError_t read_and_clear_paged_error(int* value) {
  int bits = 0;
  cudaError_t err = read_and_clear_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_decode_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_key_weights_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_pool_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_tree_error(&bits);
  *value = bits & kTimeoutBit ? kErrTimeout : bits & kPageBit ? kErrPage : 0;
  return err;
}

}  // namespace fa
