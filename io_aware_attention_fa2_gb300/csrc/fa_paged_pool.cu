// fa_paged_pool.cu -- the paged cache's pages as sequences branch and change their lengths: accept
// (drafted tokens that stay), copy, fork, resize (include/fa.h has the rules).
#include <cooperative_groups.h>

#include <algorithm>

#include "fa_paged.cuh"

namespace fa {

namespace {

using namespace paged;
namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------------------------
// Accept. The path from the accepted token up to its tree's root, then the rows of that path
// moved behind the context: path[j] >= j, so in rounds over ascending j, each with all its reads
// before its writes, no row is written before it has been read. A few tokens of each sequence:
// bound by the latency of a chain of loads (lengths, parents, table, rows): 64 sequences of 64 drafted
// tokens, Hkv=8 d=128 with weights, 3.1 us a replay. One block for each (sequence, key head), which
// finds the path by itself.
constexpr int kAcceptThreads = 128, kAcceptTokens = 8;   // 16-byte loads in flight for each lane

struct AcceptArgs {
  uint4* k_pages;
  uint4* v_pages;
  float* weights;
  const int* table;
  const int* seqlens;
  const int* parents;
  const int* leaf;
  const int* new_lens;
  int* path;
  int* new_seqlens;
  int T, Hkv, page_shift, num_pages, max_pages;
};

template <int D>
__global__ void __launch_bounds__(kAcceptThreads)
    fa_paged_accept_kernel(const __grid_constant__ AcceptArgs a) {
  constexpr int kLanes = D / 4;                        // a row's K and V, 16 bytes a lane
  constexpr int kTokens = 32 / kLanes * kAcceptTokens; // tokens of a warp in a round
  constexpr int kWarps = kAcceptThreads / 32, kRound = kTokens * kWarps;
  __shared__ short s_parent[kMaxDraft], s_path[kMaxDraft];
  __shared__ int s_count, s_bad;
  const int b = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  wait_prerequisites();
  launch_dependents();

  const Draft dr = draft_of(a.seqlens, a.new_lens, b, a.T, a.max_pages << a.page_shift);
  const int leaf = a.leaf[b];
  if (tid == 0) s_bad = dr.count < 0 || leaf < -1 || leaf >= dr.count;
  // (parents that are not earlier tokens are found below if the path meets them)
  if (a.parents)
    for (int i = tid; i < dr.count; i += kAcceptThreads) {
      const int parent = a.parents[static_cast<int64_t>(b) * a.T + i];
      s_parent[i] = static_cast<short>(parent >= -1 && parent < i ? parent : -2);
    }
  __syncthreads();
  const bool given_up = s_bad;
  if (!given_up && tid == 0) {
    int n = 0, at = leaf;   // from the leaf: the path's other end first
    for (; at >= 0; at = a.parents ? s_parent[at] : at - 1) s_path[n++] = static_cast<short>(at);
    if (at < -1) s_bad = 1;
    s_count = n;
  }
  __syncthreads();
  const int count = given_up ? 0 : s_count;
  const int* const table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int in_page = (1 << a.page_shift) - 1;
  auto from = [&](int j) { return dr.base + s_path[count - 1 - j]; };
  // every page that a moved row leaves or enters
  if (!s_bad)
    for (int j = tid; j < count; j += kAcceptThreads)
      if (from(j) != dr.base + j)
        for (int t : {from(j), dr.base + j}) {
          const int page = table[t >> a.page_shift];
          if (page < 0 || page >= a.num_pages) s_bad = 1;
        }
  __syncthreads();
  const bool bad = s_bad;
  if (hk == 0) {
    for (int j = tid; j < a.T; j += kAcceptThreads)
      a.path[static_cast<int64_t>(b) * a.T + j] = !bad && j < count ? s_path[count - 1 - j] : -1;
    if (tid == 0) {
      a.new_seqlens[b] = bad ? a.seqlens[b] : dr.base + count;
      if (bad) record_page_error();
    }
  }
  if (bad) return;

  const int part = lane % kLanes;
  const int64_t chunk = part % (D / 8);
  uint4* const pool = part < D / 8 ? a.k_pages : a.v_pages;
  for (int r0 = 0; r0 < count; r0 += kRound) {
    // lane e < kTokens looks up token j of the path
    const int j = r0 + warp * kTokens + lane;
    int64_t src = -1, dst = -1, w_dst = 0;
    float w = 0.f;
    if (lane < kTokens && j < count && from(j) != dr.base + j) {
      const int t = from(j), to = dr.base + j;
      const int64_t src_page = table[t >> a.page_shift], dst_page = table[to >> a.page_shift];
      src = (((src_page << a.page_shift) + (t & in_page)) * a.Hkv + hk) * (D / 8);
      dst = (((dst_page << a.page_shift) + (to & in_page)) * a.Hkv + hk) * (D / 8);
      if (a.weights) {
        w = load_l2(a.weights + ((src_page * a.Hkv + hk) << a.page_shift) + (t & in_page));
        w_dst = ((dst_page * a.Hkv + hk) << a.page_shift) + (to & in_page);
      }
    }
    uint4 v[kAcceptTokens];
#pragma unroll
    for (int u = 0; u < kAcceptTokens; ++u) {
      const int64_t at = __shfl_sync(0xffffffffu, src, u * (32 / kLanes) + lane / kLanes);
      if (at >= 0) v[u] = load_l2(pool + at + chunk);
    }
    __syncthreads();   // the round's reads, then its writes
#pragma unroll
    for (int u = 0; u < kAcceptTokens; ++u) {
      const int e = u * (32 / kLanes) + lane / kLanes;
      const int64_t at = __shfl_sync(0xffffffffu, src, e), to = __shfl_sync(0xffffffffu, dst, e);
      if (at >= 0) pool[to + chunk] = v[u];
    }
    if (a.weights && src >= 0) a.weights[w_dst] = w;
    __syncthreads();   // a later round reads behind what this one has written
  }
}

// ---------------------------------------------------------------------------------------------
// Copy. Bound by HBM: 4096 pages of 64 tokens, Hkv=8 d=128 with weights (2.2 GB both ways) 311 us,
// 7.0 TB/s, as fast as a plain copy; 16 pages of 16 tokens 1.7 us. The first rows of a page are
// contiguous in K and in V: a block has 16 KiB of one of them, all its loads before its stores.
// Weights, [Hkv][page_size] of a page, go to the blocks of K.
constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int kCopyChunks = kCopyThreads * kCopyLoads;   // 16 bytes each

struct CopyArgs {
  uint4* k_pages;
  uint4* v_pages;
  float* weights;
  const int* src;
  const int* dst;
  const int* rows;
  int Hkv, d, page_size, num_pages, parts;   // blocks for a page of K (or V)
};

__global__ void __launch_bounds__(kCopyThreads)
    fa_paged_copy_kernel(const __grid_constant__ CopyArgs a) {
  wait_prerequisites();
  launch_dependents();
  const int m = blockIdx.x / (2 * a.parts), at = blockIdx.x % (2 * a.parts);
  const int part = at % a.parts;
  const int src = a.src[m], dst = a.dst[m];
  if (src < 0 && dst < 0) return;   // no copy
  const int rows = a.rows ? a.rows[m] : a.page_size;
  if (src < 0 || dst < 0 || src >= a.num_pages || dst >= a.num_pages || rows < 0 ||
      rows > a.page_size) {
    record_page_error();
    return;
  }
  const int64_t row = static_cast<int64_t>(a.Hkv) * a.d / 8, page = row * a.page_size;
  const int64_t n = row * rows, first = static_cast<int64_t>(part) * kCopyChunks + threadIdx.x;
  uint4* const pool = at < a.parts ? a.k_pages : a.v_pages;
  const uint4* const from = pool + src * page;
  uint4* const to = pool + dst * page;
  uint4 v[kCopyLoads];
#pragma unroll
  for (int u = 0; u < kCopyLoads; ++u)
    if (first + u * kCopyThreads < n) v[u] = from[first + u * kCopyThreads];
#pragma unroll
  for (int u = 0; u < kCopyLoads; ++u)
    if (first + u * kCopyThreads < n) to[first + u * kCopyThreads] = v[u];
  if (a.weights && at < a.parts) {
    const int64_t all = static_cast<int64_t>(a.Hkv) * a.page_size;
    for (int64_t i = static_cast<int64_t>(part) * kCopyThreads + threadIdx.x; i < all;
         i += static_cast<int64_t>(a.parts) * kCopyThreads)
      if (static_cast<int>(i & (a.page_size - 1)) < rows)
        a.weights[dst * all + i] = a.weights[src * all + i];
  }
}

// ---------------------------------------------------------------------------------------------
// Sum of x over the threads before this one, and (in *all) over the block.
template <int THREADS>
__device__ __forceinline__ int block_scan(int x, int* s_warp, int* all) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  __syncthreads();   // s_warp may still be read by an earlier call
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const int w = lane < THREADS / 32 ? s_warp[lane] : 0;
  int before = lane < warp ? w : 0, sum = w;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  *all = sum;
  return before + inc - x;
}

// Free pages of the pool as the call finds them (a number outside the pool is recorded).
__device__ __forceinline__ int free_pages_of(const PagePool& p) {
  const int n = load_l2(p.num_free);
  if (n < 0 || n > p.num_pages) {
    record_page_error();
    return 0;
  }
  return n;
}
// The page at place i of the stack, which leaves it; -1 (recorded) when it is outside the pool.
__device__ __forceinline__ int take_page(const PagePool& p, int i) {
  const int page = load_l2(p.free_pages + i);
  p.free_pages[i] = -1;
  if (page < 0 || page >= p.num_pages) {
    record_page_error();
    return -1;
  }
  p.refs[page] = 1;
  return page;
}

// ---------------------------------------------------------------------------------------------
// Fork: lengths, pages from the pool and the list of copies by one block; then the tables' rows and
// the references of shared pages, in a second launch with a block for each kForkThreads entries, or
// by the same block where the tables are small. Bound by latency, or by the atomics: a plan of 256
// sequences 4.7 us, their 330000 entries 8.2 (launches alone).
constexpr int kForkThreads = 1024;
constexpr int kSmallTables = 8192;   // entries of a call's tables that one block has

__device__ __forceinline__ void fork_plan(const ForkParams& p, int* s_warp) {
  const int have = free_pages_of(p.pool);
  const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
  int taken = 0;
  for (int c0 = 0; c0 < p.C; c0 += kForkThreads) {
    const int c = c0 + threadIdx.x;
    int len = -1, from = -1;
    if (c < p.C) {
      from = p.source[c];
      if (from == -1) {
        len = 0;   // a new sequence
      } else if (from >= 0 && from < p.B) {
        len = p.seqlens[from];
        if (len < 0 || len > capacity) len = -1;
      }
      if (len < 0) record_page_error();
    }
    int tail = len > 0 ? len & ((1 << p.page_shift) - 1) : 0, src = -1, dst = -1;
    if (tail > 0) {
      src = p.block_table[static_cast<int64_t>(from) * p.max_pages + (len >> p.page_shift)];
      if (src < 0 || src >= p.pool.num_pages) {   // nothing to copy: its entry is -1, too
        record_page_error();
        tail = 0;
      }
    }
    int all;
    const int place = taken + block_scan<kForkThreads>(tail > 0, s_warp, &all);
    if (c < p.C) {
      if (tail > 0) {
        if (place < have)
          dst = take_page(p.pool, have - 1 - place);
        else
          len = -1;   // the pool is empty
      }
      p.out_seqlens[c] = len;
      p.copy_src[c] = dst < 0 ? -1 : src;
      p.copy_dst[c] = dst;
      p.copy_rows[c] = dst < 0 ? 0 : tail;
    }
    taken += all;
  }
  if (threadIdx.x == 0) *p.pool.num_free = have - min(taken, have);
}

// Entry `col` of new sequence c's row.
__device__ __forceinline__ void fork_entry(const ForkParams& p, int c, int col) {
  const int len = load_l2(p.out_seqlens + c);
  const int full = len > 0 ? len >> p.page_shift : 0;
  int page = -1;
  if (col < full) {
    page = p.block_table[static_cast<int64_t>(p.source[c]) * p.max_pages + col];
    if (page >= 0 && page < p.pool.num_pages) {
      atomicAdd(p.pool.refs + page, 1);
    } else {
      record_page_error();
      page = -1;
    }
  } else if (col == full && len > 0 && (len & ((1 << p.page_shift) - 1))) {
    page = load_l2(p.copy_dst + c);
  }
  p.out_table[static_cast<int64_t>(c) * p.max_pages + col] = page;
}

__global__ void __launch_bounds__(kForkThreads)
    fa_paged_fork_plan_kernel(const __grid_constant__ ForkParams p, int small) {
  __shared__ int s_warp[32];
  wait_prerequisites();
  launch_dependents();
  fork_plan(p, s_warp);
  if (!small) return;
  __syncthreads();
  for (int i = threadIdx.x; i < p.C * p.max_pages; i += kForkThreads)
    fork_entry(p, i / p.max_pages, i % p.max_pages);
}

__global__ void __launch_bounds__(kForkThreads)
    fa_paged_fork_kernel(const __grid_constant__ ForkParams p, int blocks_per_row) {
  wait_prerequisites();
  launch_dependents();
  const int c = blockIdx.x / blocks_per_row;
  const int col = (blockIdx.x % blocks_per_row) * kForkThreads + threadIdx.x;
  if (col < p.max_pages) fork_entry(p, c, col);
}

// ---------------------------------------------------------------------------------------------
// Resize: first the pages that shorter sequences give back, then those that longer ones take. Bound
// by latency (a few pages), or by the atomics and scattered accesses of the SMs at work:
//   - up to kSmallTables entries that change, one CTA: two calls for 16 sequences of 258 pages 10.0 us
//     (replays; 13.9 by sixteen);
//   - more, a cluster of sixteen: 65536 pages of 64 sequences taken and given back 19 us;
//   - tables of kLargeTables entries of many sequences, all SMs by a cooperative launch: 524288
//     pages of 152 sequences taken and given back 26.5 us, not 66.4; 131072 20.6, not 27.1; 65536
//     19.9, not 20.1; of 32 sequences 524288 in 41.5, not 64.0, of 16 in 65.9, not 63.9 (a CTA for each
//     sequence at most, see below). A few pages of such tables 14.1 us, not 12.1: a cooperative launch
//     starts when what is in front of it has ended. So are all tables past kSmallTables on a stream
//     that has only some of the SMs: a CTA on each of those.
// A fork of 64 sequences of up to 32K tokens into 256 and its end, where up to five tables give up
// each page at once: 26 us, not 51.
//
// The order of the stack is the tables' order, whatever the number of threads and their timing: a
// page that several tables give back at once goes by the last of them. Each gives up its
// reference; the one that took the last reference pushes the page, unless the page was given up
// by others of this call as well. Only if there is such a page do all bid for theirs: -1 - the
// place in the order, by an atomic minimum on the references; the one whose bid stands pushes it.
// What the CTAs count goes to the others through distributed shared memory, or through `granted`,
// which has an element for each and gets its values at the end.
//
// A warp has consecutive items (entries that are given back, or taken), kBatch at a time for each
// lane, so that as many accesses are on their way; a lane finds its first item's sequence by search
// and the others' by steps.
constexpr int kResizeThreads = 1024, kResizeCluster = 16, kBatch = 4;
constexpr int kLargeTables = 1 << 17, kLargeBatch = 32;
constexpr int kFlag = 1 << 30;             // beside a count (one CTA has fewer entries than that)

// The table entry of item f, then of items 32 further on each. The items of sequence b are the
// entries behind the page of its token lens[b] - 1.
struct EntryWalk {
  const ResizeParams& p;
  const int* prefix;   // [B + 1], shared memory
  const int* lens;
  int b, f, end;       // sequence, item, the sequence's last item + 1
  int* at;
  __device__ __forceinline__ void find() {
    const int64_t first = (static_cast<int64_t>(lens[b]) + (1 << p.page_shift) - 1) >> p.page_shift;
    at = p.block_table + static_cast<int64_t>(b) * p.max_pages + first + f - prefix[b];
    end = prefix[b + 1];
  }
  __device__ __forceinline__ EntryWalk(const ResizeParams& p, const int* prefix, const int* lens, int f)
      : p(p), prefix(prefix), lens(lens), f(f) {
    int lo = 0, hi = p.B;   // prefix[lo] <= f < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (prefix[mid] <= f)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    find();
  }
  // The entry, or null behind item `last` - 1; then on to the next.
  __device__ __forceinline__ int* next(int last) {
    if (f >= last) return nullptr;
    if (f >= end) {
      while (prefix[b + 1] <= f) ++b;
      find();
    }
    int* const entry = at;
    f += 32;
    at += 32;
    return entry;
  }
};

template <bool ALL>
__global__ void __launch_bounds__(kResizeThreads, 1)
    fa_paged_resize_kernel(const __grid_constant__ ResizeParams p) {
  extern __shared__ __align__(16) int s_prefix[];   // [B + 1] releases, [B + 1] takes
  __shared__ int s_warp[32], s_total, s_before;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = ALL ? blockIdx.x : static_cast<int>(cluster.block_rank());
  int ranks = ALL ? gridDim.x : static_cast<int>(cluster.num_blocks());
  auto meet = [&] {   // all CTAs, with what they have written
    if (ranks == 1)
      __syncthreads();
    else if constexpr (ALL)
      cg::this_grid().sync();
    else
      cluster.sync();
  };
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t capacity = static_cast<int64_t>(p.max_pages) << p.page_shift;
  int* const s_release = s_prefix;
  int* const s_take = s_prefix + p.B + 1;
  wait_prerequisites();
  launch_dependents();

  // the prefixes over the sequences, by every CTA for itself
  const int have = free_pages_of(p.pool);
  auto pages_of = [&](int tokens) { return (tokens + (1 << p.page_shift) - 1) >> p.page_shift; };
  int releases = 0, takes = 0;
  for (int b0 = 0; b0 < p.B; b0 += kResizeThreads) {
    const int b = b0 + tid;
    int gone = 0, more = 0;
    if (b < p.B) {
      const int from = p.old_lens[b], to = p.new_lens[b];
      if (from >= 0 && to >= 0 && from <= capacity && to <= capacity) {
        const int a = pages_of(from), z = pages_of(to);
        gone = max(a - z, 0);
        more = max(z - a, 0);
      } else if (rank == 0) {
        record_page_error();
      }
    }
    int all;
    const int r = releases + block_scan<kResizeThreads>(gone, s_warp, &all);
    releases += all;
    const int t = takes + block_scan<kResizeThreads>(more, s_warp, &all);
    takes += all;
    if (b < p.B) {
      s_release[b] = r;
      s_take[b] = t;
    }
  }
  if (tid == 0) {
    s_release[p.B] = releases;
    s_take[p.B] = takes;
  }
  __syncthreads();
  // A few entries of large tables are one CTA's (which waits for no other).
  if (static_cast<int64_t>(releases) + takes <= kSmallTables) {
    if (rank > 0) return;
    ranks = 1;
  }
  // this warp's items of n
  const int warps = ranks * (kResizeThreads / 32), w = rank * (kResizeThreads / 32) + warp;
  auto first_item = [&](int n, int at) {
    return static_cast<int>(static_cast<int64_t>(n) * at / warps);
  };

  int pushed = 0;
  if (releases > 0) {
    const int f0 = first_item(releases, w), f1 = first_item(releases, w + 1);
    // batch(i, entries) for the lane's items f0 + lane + 32 i, kBatch entries at a time
    auto for_items = [&](auto&& batch) {
      if (f0 + lane >= f1) return;
      EntryWalk walk(p, s_release, p.new_lens, f0 + lane);
      for (int i = 0; f0 + lane + 32 * i < f1; i += kBatch) {
        int* at[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) at[u] = walk.next(f1);
        batch(i, at);
      }
    };
    // Bit i: of the lane's item i. Past 64 items a lane there are no bits, and all bid.
    const bool bits = f1 - f0 <= 2048;
    uint64_t last = 0, other = 0;   // took the last reference; did not
    bool contest = !bits;
    for_items([&](int i, int* (&at)[kBatch]) {
      int page[kBatch], old[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) page[u] = at[u] ? *at[u] : -1;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        old[u] = 0;
        if (page[u] >= 0 && page[u] < p.pool.num_pages)
          old[u] = atomicSub(p.pool.refs + page[u], 1);
        else
          page[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!at[u]) continue;
        if (old[u] <= 0) {   // outside the pool, or held by no table
          if (page[u] >= 0) atomicAdd(p.pool.refs + page[u], 1);
          record_page_error();
          *at[u] = -1;
        } else if (bits) {
          (old[u] == 1 ? last : other) |= 1ull << (i + u);
        }
      }
    });
    meet();
    // a page without references that this call gave up more than once
    if (bits && other)
      for_items([&](int i, int* (&at)[kBatch]) {
        int left[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          left[u] = other >> (i + u) & 1 ? load_l2(p.pool.refs + *at[u]) : 1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) contest |= left[u] == 0;
      });
    // Pages to push by this warp's lanes, `count` each: by those of warps before this one, in
    // `before`, and by all, in `pushed`; and whether `flag` is set in any thread.
    int before = 0;
    auto count_all = [&](int count, bool flag) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) count += __shfl_xor_sync(0xffffffffu, count, off);
      int all;
      before = block_scan<kResizeThreads>(lane == 0 ? count : 0, s_warp, &all);
      before = __shfl_sync(0xffffffffu, before, 0);
      const int mine = all | (__syncthreads_or(flag) ? kFlag : 0);
      if (tid == 0) (ALL ? p.granted[rank] : s_total) = mine;
      meet();
      int of_rank = 0;
      if (tid < ranks) of_rank = ALL ? load_l2(p.granted + tid) : *cluster.map_shared_rank(&s_total, tid);
      const bool any = __syncthreads_or(of_rank & kFlag);
      const int earlier = block_scan<kResizeThreads>(of_rank & (kFlag - 1), s_warp, &pushed);
      if (tid == rank) s_before = earlier;
      __syncthreads();
      before += s_before;
      return any;
    };
    const bool bid = count_all(__popcll(last), contest);
    // whether item i is the one that pushes its page
    auto pushes = [&](int i, int page) {
      if (!bid) return (last >> i & 1) != 0;
      return page >= 0 && load_l2(p.pool.refs + page) == -1 - (f0 + lane + 32 * i);
    };
    if (bid) {
      for_items([&](int i, int* (&at)[kBatch]) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int page = at[u] ? *at[u] : -1;
          if (page >= 0 && load_l2(p.pool.refs + page) <= 0)
            atomicMin(p.pool.refs + page, -1 - (f0 + lane + 32 * (i + u)));
        }
      });
      meet();
      int count = 0;
      for_items([&](int i, int* (&at)[kBatch]) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) count += at[u] && pushes(i + u, *at[u]);
      });
      count_all(count, false);
    }
    // the warp's items in order: 32 of them for each i
    {
      EntryWalk walk(p, s_release, p.new_lens, min(f0 + lane, releases - 1));
      walk.f = f0 + lane;   // (past the last item it is at none of them)
      const int steps = (f1 - f0 + 31) / 32;
      for (int i = 0; i < steps; i += kBatch) {
        int* at[kBatch];
        int page[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          at[u] = walk.next(f1);
          page[u] = at[u] ? *at[u] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const bool mine = at[u] && pushes(i + u, page[u]);
          const unsigned all_mine = __ballot_sync(0xffffffffu, mine);
          if (mine) {
            const int place = have + before + __popc(all_mine & ((1u << lane) - 1));
            if (place < p.pool.num_pages)
              p.pool.free_pages[place] = page[u];
            else
              record_page_error();   // more free pages than the pool has
            if (bid) p.pool.refs[page[u]] = 0;
          }
          if (at[u]) *at[u] = -1;
          before += __popc(all_mine);
        }
      }
    }
    pushed = min(pushed, p.pool.num_pages - have);
    meet();   // the stack is whole; every CTA has read the counts
  }

  // The takes. What fits is a prefix of them: up to the largest one within the stack, found by
  // every CTA for itself.
  const int stack = have + pushed;
  int taken = 0;
  for (int b = tid; b < p.B; b += kResizeThreads)
    if (s_take[b + 1] <= stack) taken = max(taken, s_take[b + 1]);
  taken = __reduce_max_sync(0xffffffffu, taken);
  __syncthreads();
  if (lane == 0) s_warp[warp] = taken;
  __syncthreads();
  taken = __reduce_max_sync(0xffffffffu, s_warp[lane]);
  {
    const int f0 = first_item(taken, w), f1 = first_item(taken, w + 1);
    if (f0 + lane < f1) {
      EntryWalk walk(p, s_take, p.old_lens, f0 + lane);
      for (int f = f0 + lane; f < f1; f += 32 * kBatch) {
        int page[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          page[u] = f + 32 * u < f1 ? load_l2(p.pool.free_pages + stack - 1 - (f + 32 * u)) : -1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          int* const at = walk.next(f1);
          if (!at) break;
          if (page[u] >= 0 && page[u] < p.pool.num_pages) {
            p.pool.refs[page[u]] = 1;
          } else {
            record_page_error();
            page[u] = -1;
          }
          p.pool.free_pages[stack - 1 - (f + 32 * u)] = -1;
          *at = page[u];
        }
      }
    }
  }
  for (int b = rank * kResizeThreads + tid; b < p.B; b += ranks * kResizeThreads) {
    const int from = p.old_lens[b], to = p.new_lens[b];
    const bool ok = from >= 0 && to >= 0 && from <= capacity && to <= capacity;
    const bool fits = s_take[b + 1] == s_take[b] || s_take[b + 1] <= stack;
    p.granted[b] = ok && fits ? to : from;
  }
  if (ranks > 1 && releases == 0) meet();   // every CTA has read num_free
  if (rank == 0 && tid == 0) *p.pool.num_free = stack - taken;
}

}  // namespace

cudaError_t launch_paged_accept(const AcceptParams& p, cudaStream_t stream) {
  const PagedCache& c = p.c;
  AcceptArgs a;
  a.k_pages = static_cast<uint4*>(c.k_pages);
  a.v_pages = static_cast<uint4*>(c.v_pages);
  a.weights = c.weights;
  a.table = c.block_table;
  a.seqlens = c.seqlens;
  a.parents = p.parents;
  a.leaf = p.leaf;
  a.new_lens = p.new_lens;
  a.path = p.path;
  a.new_seqlens = p.new_seqlens;
  a.T = p.T;
  a.Hkv = c.Hkv;
  a.page_shift = shift_of(c.page_size);
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  return launch_paged(c.d == 64 ? fa_paged_accept_kernel<64> : fa_paged_accept_kernel<128>,
                      static_cast<int64_t>(c.B) * c.Hkv, kAcceptThreads, 0, stream, 0, a);
}

cudaError_t launch_paged_copy(const CopyParams& p, cudaStream_t stream) {
  CopyArgs a;
  a.k_pages = static_cast<uint4*>(p.k_pages);
  a.v_pages = static_cast<uint4*>(p.v_pages);
  a.weights = p.weights;
  a.src = p.src;
  a.dst = p.dst;
  a.rows = p.rows;
  a.Hkv = p.Hkv;
  a.d = p.d;
  a.page_size = p.page_size;
  a.num_pages = p.num_pages;
  const int64_t chunks = static_cast<int64_t>(p.page_size) * p.Hkv * p.d / 8;
  a.parts = static_cast<int>((chunks + kCopyChunks - 1) / kCopyChunks);
  return launch_paged(fa_paged_copy_kernel, static_cast<int64_t>(p.M) * 2 * a.parts, kCopyThreads,
                      0, stream, 0, a);
}

cudaError_t launch_paged_fork(const ForkParams& p, cudaStream_t stream) {
  const int small = static_cast<int64_t>(p.C) * p.max_pages <= kSmallTables;
  cudaError_t err = launch_paged(fa_paged_fork_plan_kernel, 1, kForkThreads, 0, stream, 0, p, small);
  if (err != cudaSuccess || small) return err;
  const int blocks = (p.max_pages + kForkThreads - 1) / kForkThreads;
  return launch_paged(fa_paged_fork_kernel, static_cast<int64_t>(p.C) * blocks, kForkThreads, 0,
                      stream, 0, p, blocks);
}

template <bool ALL>
cudaError_t prepare_resize() {
  constexpr int kMost = 2 * (kMaxPoolBatch + 1) * 4;
  return cudaFuncSetAttribute(fa_paged_resize_kernel<ALL>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
}

cudaError_t launch_paged_resize(const ResizeParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.B) * p.max_pages;
  const size_t smem = 2 * (p.B + 1) * 4;
  cudaError_t err;
  if (entries > kSmallTables) {
    int device, all;
    if ((err = cudaGetDevice(&device)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&all, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
      return err;
    // (where a stream has only some of the SMs, a cluster of sixteen need not fit)
    const int sms = stream_sms(stream, all);
    if (sms < all || (entries >= kLargeTables && p.B >= kLargeBatch)) {
      if ((err = prepare_resize<true>()) != cudaSuccess) return err;
      return launch_together(fa_paged_resize_kernel<true>, std::min(p.B, sms), kResizeThreads, smem,
                             stream, p);
    }
  }
  err = prepare_resize<false>();
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(fa_paged_resize_kernel<false>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  const int ctas = entries <= kSmallTables ? 1 : kResizeCluster;
  return launch_paged(fa_paged_resize_kernel<false>, ctas, kResizeThreads, smem, stream,
                      ctas > 1 ? ctas : 0, p);
}

cudaError_t read_and_clear_pool_error(int* bits) { return read_and_clear_error(bits); }

}  // namespace fa
