// fa_paged.cu -- the paged key-value cache: append and evict (include/fa.h has the layouts and
// the rules for bad block-table entries and lengths).
#include <cooperative_groups.h>

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
// Evict. A cluster of eight CTAs for each (sequence, key head): each CTA has an eighth of the
// candidates, and the histograms, counts and flags are exchanged through distributed shared
// memory. What has to be read and written is the weights (4 bytes a token) and the kept rows
// twice (4 d bytes a token each way).
//
// Which ones stay: the want-th largest weight among the tokens before the recent ones, found by
// radix selection on the weights as ordered 32-bit keys (digits of 11, 11 and 10 bits, one
// histogram over the cluster each), then the equal ones from the oldest until there are enough.
// The keys are read once and kept in shared memory.
//
// The move: kept token i goes to row i of out_table's pages, in rounds of the cluster's width. When
// out_table names pages of the sequence itself, a cluster barrier between a round's reads and
// its writes keeps the order: a token's new place is never behind its old one, so a later round's
// sources lie behind every earlier destination.
namespace cg = cooperative_groups;

constexpr int kEvictThreads = 512, kEvictCluster = 8;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictCache = 12288;   // keys of a CTA's eighth in shared memory; further ones are
                                     // read from the pages in every pass
constexpr int kMoveTokens = 4;       // tokens in flight for each 32 lanes
constexpr size_t kEvictSmem = (2 * kEvictBins + kEvictCache) * 4;

// Weights as unsigned numbers in the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictArgs {
  uint4* k_pages;
  uint4* v_pages;
  float* weights;
  const int* table;
  const int* seqlens;
  const int* out_table;
  int* kept;
  int* new_seqlens;
  int Hkv, page_size, num_pages, max_pages, out_pages, budget, recent;
};

template <int D>
__global__ void __cluster_dims__(kEvictCluster, 1, 1) __launch_bounds__(kEvictThreads, 3)
    fa_paged_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint4 smem_raw[];
  uint32_t* const hist = reinterpret_cast<uint32_t*>(smem_raw);   // [2][kEvictBins]
  uint32_t* const cache = hist + 2 * kEvictBins;
  __shared__ uint32_t s_warp[kEvictWarps], s_found[2];
  __shared__ int2 s_count, s_warp_count[kEvictWarps];   // candidates above and at the threshold
  __shared__ int s_bad, s_own_pages;   // flags of this CTA's share of the checks
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int wide = rank * kEvictThreads + tid, width = kEvictCluster * kEvictThreads;
  const int64_t unit = blockIdx.x / kEvictCluster;
  const int b = static_cast<int>(unit / a.Hkv), hk = static_cast<int>(unit % a.Hkv);
  const int ps = a.page_size;
  const int* const src_table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int* const dst_table = a.out_table + static_cast<int64_t>(b) * a.out_pages;
  int* const kept = a.kept + unit * a.budget;

  const int raw_len = a.seqlens[b];
  const bool bad_len = raw_len < 0 || raw_len > a.max_pages * ps;
  const int len = bad_len ? 0 : raw_len, new_len = min(len, a.budget);
  const int src_used = (len + ps - 1) / ps, dst_used = (new_len + ps - 1) / ps;
  auto in_pool = [&](int page) { return page >= 0 && page < a.num_pages; };
  if (tid == 0) {
    s_bad = bad_len;
    s_own_pages = 0;
  }
  for (int i = tid; i < 2 * kEvictBins; i += kEvictThreads) hist[i] = 0;
  __syncthreads();
  // the pages are in the pool, and no destination stands in the sequence at a later place
  for (int i = wide; i < src_used; i += width)
    if (!in_pool(src_table[i])) s_bad = 1;
  for (int i = wide; i < dst_used; i += width)
    if (!in_pool(dst_table[i])) s_bad = 1;
  for (int64_t x = wide; x < static_cast<int64_t>(dst_used) * src_used; x += width) {
    const int i = static_cast<int>(x / src_used), j = static_cast<int>(x % src_used);
    if (dst_table[i] == src_table[j]) {
      s_own_pages = 1;
      if (j > i) s_bad = 1;
    }
  }

  // ---- selection
  const bool select = len > a.budget;
  const int n = select ? len - a.recent : 0;         // candidates: tokens [0, n)
  uint32_t want = select ? a.budget - a.recent : 0;  // of them stay
  const int share = (n + kEvictCluster - 1) / kEvictCluster;
  const int t0 = min(rank * share, n), mine = min(share, n - t0);   // this CTA's: [t0, t0 + mine)
  auto load_key = [&](int t) {
    const int page = src_table[t / ps];
    // (a bad page: the sequence is given up below)
    return in_pool(page) ? order_key(__ldcg(
                               a.weights + (static_cast<int64_t>(page) * a.Hkv + hk) * ps + t % ps))
                         : 0u;
  };
  const int cached = min(mine, kEvictCache);
#pragma unroll 4
  for (int i = tid; i < cached; i += kEvictThreads) cache[i] = load_key(t0 + i);
  __syncthreads();
  auto key_at = [&](int i) { return i < cached ? cache[i] : load_key(t0 + i); };

  bool own_pages = false;
  uint32_t prefix = 0;   // digits found so far
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0};
    const int shift = kShift[pass], bits = pass == 2 ? 10 : 11;
    uint32_t* const h = hist + (pass & 1) * kEvictBins;
    if (want) {
      for (int i = tid; i < mine; i += kEvictThreads) {
        const uint32_t key = key_at(i);
        if (pass == 0 || (key >> (shift + bits)) == prefix)
          atomicAdd(&h[(key >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    cluster.sync();
    if (pass == 0) {
      // the first exchange carries the flags, too
      int bad = 0, own = 0;
      for (int r = 0; r < kEvictCluster; ++r) {
        bad |= *cluster.map_shared_rank(&s_bad, r);
        own |= *cluster.map_shared_rank(&s_own_pages, r);
      }
      if (bad) {
        for (int i = wide; i < a.budget; i += width) kept[i] = -1;
        if (wide == 0) {
          record_page_error();
          if (hk == 0) a.new_seqlens[b] = raw_len;
        }
        cluster.sync();   // no CTA leaves while another reads its flags
        return;
      }
      own_pages = own;
    }
    if (want) {
      // four bins a thread, from the top: bins below thread tid's are those of later threads
      uint32_t bin[4] = {0, 0, 0, 0};
      const int top = kEvictBins - 4 - 4 * tid;
      for (int r = 0; r < kEvictCluster; ++r) {
        const uint4 x = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(h + top, r));
        bin[0] += x.w;
        bin[1] += x.z;
        bin[2] += x.y;
        bin[3] += x.x;
      }
      const uint32_t sum = bin[0] + bin[1] + bin[2] + bin[3];
      uint32_t inc = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      uint32_t before = inc - sum;
      for (int w = 0; w < warp; ++w) before += s_warp[w];
      if (before < want && want <= before + sum) {
        int e = 0;
        while (before + bin[e] < want) before += bin[e++];
        s_found[0] = top + 3 - e;
        s_found[1] = before;
      }
      __syncthreads();
      prefix = prefix << bits | s_found[0];
      want -= s_found[1];   // of the keys that start with prefix
    }
    if (pass == 1) {
      // every CTA has read the first histogram: it serves the third pass
      for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
    }
  }

  // ---- kept: the tokens above the threshold and the oldest `want` at it, in order
  if (select) {
    const bool any = a.budget > a.recent;
    const int per_warp = (mine + 32 * kEvictWarps - 1) / (32 * kEvictWarps) * 32;
    const int w0 = min(warp * per_warp, mine), w1 = min(w0 + per_warp, mine);
    int2 count = make_int2(0, 0);
    for (int i = w0; i < w1; i += 32) {
      const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
      const bool in = any && i + lane < w1;
      count.x += __popc(__ballot_sync(0xffffffffu, in && key > prefix));
      count.y += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
    }
    if (lane == 0) s_warp_count[warp] = count;
    __syncthreads();
    if (tid == 0) {
      int2 sum = make_int2(0, 0);
      for (int w = 0; w < kEvictWarps; ++w) {
        sum.x += s_warp_count[w].x;
        sum.y += s_warp_count[w].y;
      }
      s_count = sum;
    }
    cluster.sync();
    int above = 0, equal = 0;   // before this warp's candidates
    for (int r = 0; r < rank; ++r) {
      const int2 c = *cluster.map_shared_rank(&s_count, r);
      above += c.x;
      equal += c.y;
    }
    for (int w = 0; w < warp; ++w) {
      above += s_warp_count[w].x;
      equal += s_warp_count[w].y;
    }
    const unsigned below = (1u << lane) - 1;
    for (int i = w0; i < w1; i += 32) {
      const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
      const bool in = any && i + lane < w1;
      const unsigned up = __ballot_sync(0xffffffffu, in && key > prefix);
      const unsigned at = __ballot_sync(0xffffffffu, in && key == prefix);
      const int rank_at = equal + __popc(at & below);
      const bool keep = (up >> lane & 1) || ((at >> lane & 1) && rank_at < static_cast<int>(want));
      if (keep)
        kept[above + __popc(up & below) + min(rank_at, static_cast<int>(want))] = t0 + i + lane;
      above += __popc(up);
      equal += __popc(at);
    }
    for (int i = wide; i < a.recent; i += width) kept[a.budget - a.recent + i] = n + i;
  } else {
    for (int i = wide; i < a.budget; i += width) kept[i] = i < len ? i : -1;
  }
  if (wide == 0 && hk == 0) a.new_seqlens[b] = new_len;
  cluster.sync();   // kept is complete; and no shared memory is read from another CTA after this

  // ---- move: a row's K and V take D / 4 lanes, 16 bytes each
  constexpr int kLanes = D / 4, kTokens = 32 / kLanes * kMoveTokens;   // tokens of a warp
  constexpr int kRound = kTokens * kEvictWarps * kEvictCluster;
  for (int r0 = 0; r0 < new_len; r0 += kRound) {
    // lane e < kTokens looks up token i0 + e
    const int i = r0 + (rank * kEvictWarps + warp) * kTokens + lane;
    int64_t src = -1, dst = -1, w_dst = 0;
    float w = 0.f;
    if (lane < kTokens && i < new_len) {
      const int t = __ldcg(kept + i);
      const int64_t src_page = src_table[t / ps], dst_page = dst_table[i / ps];
      const int src_row = t % ps, dst_row = i % ps;
      src = ((src_page * ps + src_row) * a.Hkv + hk) * (D / 8);
      dst = ((dst_page * ps + dst_row) * a.Hkv + hk) * (D / 8);
      if (src == dst) {   // in place already
        src = -1;
      } else {
        w = __ldcg(a.weights + (src_page * a.Hkv + hk) * ps + src_row);
        w_dst = (dst_page * a.Hkv + hk) * ps + dst_row;
      }
    }
    const int part = lane % kLanes;
    const int64_t chunk = part % (D / 8);
    uint4* const pool = part < D / 8 ? a.k_pages : a.v_pages;
    uint4 v[kMoveTokens];
#pragma unroll
    for (int u = 0; u < kMoveTokens; ++u) {
      const int64_t from = __shfl_sync(0xffffffffu, src, u * (32 / kLanes) + lane / kLanes);
      if (from >= 0) v[u] = __ldcg(pool + from + chunk);
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

template <int D>
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
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
  a.page_size = c.page_size;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.out_pages = p.out_pages;
  a.budget = p.budget;
  a.recent = p.recent;
  const int smem = static_cast<int>(kEvictSmem);
  cudaError_t err = cudaFuncSetAttribute(fa_paged_evict_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const int64_t ctas = static_cast<int64_t>(c.B) * c.Hkv * kEvictCluster;
  fa_paged_evict_kernel<D><<<static_cast<unsigned>(ctas), kEvictThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t stream) {
  return p.c.d == 64 ? launch_evict<64>(p, stream) : launch_evict<128>(p, stream);
}

cudaError_t read_and_clear_paged_error(int* value) {
  int bits = 0;
  cudaError_t err = read_and_clear_error(&bits);
  if (err == cudaSuccess) err = read_and_clear_decode_error(&bits);
  *value = bits & kTimeoutBit ? kErrTimeout : bits & kPageBit ? kErrPage : 0;
  return err;
}

}  // namespace fa
