// evict.cu -- eviction from the paged cache by accumulated weight: which tokens
// stay (an exact radix select for each request), and the rows that move.
//
// A key has no position, so the tokens that stay need not keep their order: the
// request's cache shrinks to its first `left` places, whose dropped tokens' places
// are taken by the kept tokens from behind.  Places that are read (from `left` on)
// and places that are written (below it) are disjoint, so the rows move in place,
// in any order, and only about left (1 - left / n) of them move, where keeping the
// order would move nearly all.
#include <atomic>

#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kMaxThreads = 1024;  // of a CTA of the selection
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 40960;    // keys of a CTA's share that fit shared memory (160 KB)
constexpr int kCopies = 8;         // of a histogram, for lanes that meet in a bin
// two words for each 32 of the 2^22 / kMaxCluster places that a share may have
constexpr int kMaxWordBytes = (1 << 22) / kMaxCluster / 4;

// In the workspace header, behind the status word; both are 0 between calls.
struct Counters {
  int32_t* moves;   // moves listed so far
  uint32_t* ended;  // blocks of the moving kernel that have ended
};
__host__ __device__ __forceinline__ Counters counters(uint8_t* ws) {
  return {reinterpret_cast<int32_t*>(ws + 64), reinterpret_cast<uint32_t*>(ws + 128)};
}

// Moves are of distinct slots, from and to distinct places: at most half the cache.
int64_t max_moves(const ServeShape& s) { return s.n_pages * s.page / 2 + 1; }

struct Moves {
  int32_t *src, *dst;
};
Moves moves_of(const ServeShape& s, uint8_t* ws) {
  int32_t* at = reinterpret_cast<int32_t*>(ws + kHeader);
  return {at, at + round_up((size_t)max_moves(s), 64)};
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_input_f(const float* p) {
  return __int_as_float(ld_input(reinterpret_cast<const int32_t*>(p)));
}

// A weight as an integer in the same order, the two zeros alike, NaN below all.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  return w != w ? 0u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// The sum of x over the threads before this one, and over all of them; every thread
// of the CTA, `sums` [32] in shared memory, which may be used again after it.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sums, uint32_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const uint32_t w = lane < warps ? sums[lane] : 0u;
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
  *all = __reduce_add_sync(0xffffffffu, w);
  __syncthreads();
  return before + incl - x;
}

// A cluster has a request, each CTA of it consecutive places.  Cached: their keys
// lie in shared memory, else they are read again in each pass.
//
// Four passes of eight bits find the left-th largest key.  Then a bit for each place
// says whether its token stays; words of 32 places are a thread's, so that two scans
// of population counts number the equal keys, the freed places and the movers.
template <bool Cached>
__global__ void __launch_bounds__(kMaxThreads) select_kernel(
    const float* w, const int32_t* table, const int32_t* seq, const int32_t* keep,
    int32_t n_first, int32_t n_last, float* w_out, Moves moves, int64_t list_len,
    Counters counts, int max_blocks, int page_log2, int64_t n_pages, int max_words,
    uint32_t* status) {
  extern __shared__ uint32_t smem[];
  uint32_t* above_w = smem;               // [word] keys above the threshold
  uint32_t* equal_w = smem + max_words;   // [word] keys equal to it
  uint32_t* keys = smem + 2 * max_words;
  __shared__ uint32_t hist[kCopies][257];
  __shared__ uint32_t sum_hist[2][256];   // of this CTA, in turns
  __shared__ uint32_t sums[32];
  __shared__ uint32_t found[3];           // the digit, keys above it, keys with it
  __shared__ uint32_t totals[2];          // freed places and movers of this CTA
  __shared__ uint32_t first_move;         // of the request, in the leader
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const int b = blockIdx.x / size;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t cap = max_blocks << page_log2, in_page = (1 << page_log2) - 1;
  const int32_t n = ld_input(seq + b), want = ld_input(keep + b);
  if (n < 0 || n > cap || want < 0) {  // the same in the whole cluster
    if (tid == 0 && rank == 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    return;
  }
  const int32_t left = min(n, want);
  const int32_t* row = table + (int64_t)b * max_blocks;
  const int32_t share = ((n + (int)size - 1) / (int)size + 31) & ~31;
  const int32_t lo = min(n, (int)rank * share), hi = min(n, lo + share);
  auto slot_of = [&](int32_t j) -> int32_t {
    const int32_t p = ld_input(row + (j >> page_log2));
    if (p < 0 || p >= n_pages) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      return -1;
    }
    return (p << page_log2) + (j & in_page);
  };
  if (left == n || left == 0) {  // all stay, or none
    if (w_out != w)
      for (int32_t j = lo + tid; j < min(hi, left); j += nt) {
        const int32_t s = slot_of(j);
        if (s >= 0) w_out[s] = ld_input_f(w + s);
      }
    return;
  }
  auto read_key = [&](int32_t j) -> uint32_t {
    if (j < n_first || j >= n - n_last) return 0xff800000u;  // +inf
    const int32_t s = slot_of(j);
    return s < 0 ? 0u : order_key(ld_input_f(w + s));
  };
  auto key_of = [&](int32_t j) { return Cached ? keys[j - lo] : read_key(j); };
  if (Cached) {
#pragma unroll 4
    for (int32_t j = lo + tid; j < hi; j += nt) keys[j - lo] = read_key(j);
  }

  // ---- the left-th largest key, eight bits at a time from the top
  uint32_t prefix = 0u;            // its bits so far
  uint32_t rest = (uint32_t)left;  // its rank among the keys with that prefix
  uint32_t ties = 0u;              // keys equal to it in the CTAs before
  uint32_t* mine = hist[lane & (kCopies - 1)];
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < kCopies * 257; i += nt) hist[i / 257][i % 257] = 0u;
    __syncthreads();
    const uint32_t above = pass ? 0xffffffffu << (shift + 8) : 0u;
#pragma unroll 4
    for (int32_t j = lo + tid; j < hi; j += nt) {
      const uint32_t k = key_of(j);
      if ((k & above) == prefix) atomicAdd(mine + ((k >> shift) & 255u), 1u);
    }
    __syncthreads();
    // of this CTA, then of the cluster; thread t has digit 255 - t
    uint32_t* here = sum_hist[pass & 1];
    uint32_t all = 0u;
    if (tid < 256) {
      for (int i = 0; i < kCopies; ++i) all += hist[i][255 - tid];
      here[255 - tid] = all;
    }
    if (size > 1) {
      // (the other buffer is read until the barrier of the next pass)
      cluster_arrive();
      cluster_wait();
      if (tid < 256) {
        all = 0u;
        const uint32_t at = smem_u32(here + 255 - tid);
        uint32_t c[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) c[r] = r < (int)size ? ld_cluster(at_rank(at, r)) : 0u;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) all += c[r];
      }
    }
    uint32_t sum;
    const uint32_t before = block_scan(tid < 256 ? all : 0u, sums, &sum);
    if (tid < 256 && before < rest && rest <= before + all) {
      found[0] = 255u - tid;
      found[1] = before;
      found[2] = all;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    rest -= found[1];
  }
  const bool all_ties = rest == found[2];
  if (!all_ties)
    for (uint32_t r = 0; r < rank; ++r)
      ties += ld_cluster(at_rank(smem_u32(sum_hist[1] + found[0]), r));

  // ---- which keys are above the threshold, which equal to it: a bit each
  const int words = (hi - lo + 31) >> 5;
#pragma unroll 4
  for (int x = warp; x < words; x += nt >> 5) {
    const int32_t j = lo + 32 * x + lane;
    const uint32_t k = j < hi ? key_of(j) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, j < hi && k > prefix);
    const uint32_t eq = __ballot_sync(0xffffffffu, j < hi && k == prefix);
    if (lane == 0) {
      above_w[x] = gt;
      equal_w[x] = eq;
    }
  }
  __syncthreads();
  // ---- `rest` of the equal ones stay, those of the lowest places; each thread has
  // consecutive words
  const int each = (words + nt - 1) / nt, x0 = min(words, tid * each), x1 = min(words, x0 + each);
  uint32_t all;
  if (!all_ties) {
    uint32_t eq = 0u;
    for (int x = x0; x < x1; ++x) eq += __popc(equal_w[x]);
    uint32_t at = ties + block_scan(eq, sums, &all);
    for (int x = x0; x < x1; ++x) {
      uint32_t e = equal_w[x], stay = 0u;
      for (; e && at < rest; ++at) {
        stay |= e & (0u - e);
        e &= e - 1u;
      }
      at += __popc(e);
      equal_w[x] = stay;
    }
  }
  // the places of word x that are below `end`
  auto below = [&](int x, int32_t end) {
    const int32_t m = end - lo - 32 * x;
    return m <= 0 ? 0u : m >= 32 ? 0xffffffffu : (1u << m) - 1u;
  };
  uint32_t n_holes = 0u, n_movers = 0u;
  for (int x = x0; x < x1; ++x) {
    const uint32_t kept = above_w[x] | equal_w[x], low = below(x, left);
    above_w[x] = kept;
    n_holes += __popc(~kept & low & below(x, hi));
    n_movers += __popc(kept & ~low);
  }
  uint32_t h = block_scan(n_holes, sums, &all);
  if (tid == 0) totals[0] = all;
  uint32_t m = block_scan(n_movers, sums, &all);
  if (tid == 0) totals[1] = all;
  __syncthreads();
  uint32_t all_moves = 0u;
  if (size > 1) {
    cluster_arrive();
    cluster_wait();
  }
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < (int)size) {
      const uint32_t a = ld_cluster(at_rank(smem_u32(totals), r));
      all_moves += a;
      if (r < (int)rank) {
        h += a;
        m += ld_cluster(at_rank(smem_u32(totals + 1), r));
      }
    }
  if (rank == 0 && tid == 0) {
    const int32_t at = all_moves ? atomicAdd(counts.moves, (int32_t)all_moves) : 0;
    // a page that stands in two places: more moves than the cache has slots for
    const bool fits = at >= 0 && at + (int64_t)all_moves <= list_len;
    if (!fits) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    first_move = fits ? (uint32_t)at : 0xffffffffu;
  }
  if (w_out != w) {  // the tokens that stay where they are
#pragma unroll 4
    for (int32_t j = lo + tid; j < min(hi, left); j += nt)
      if (above_w[(j - lo) >> 5] >> ((j - lo) & 31) & 1u) {
        const int32_t s = slot_of(j);
        if (s >= 0) w_out[s] = ld_input_f(w + s);
      }
  }
  __syncthreads();
  if (size > 1) {
    cluster_arrive();
    cluster_wait();
  }
  const uint32_t at = ld_cluster(at_rank(smem_u32(&first_move), 0));
  // the leader's shared memory lives until the others have read it
  if (size > 1) cluster_arrive();
  if (at != 0xffffffffu) {
    for (int x = x0; x < x1; ++x) {
      const uint32_t kept = above_w[x], low = below(x, left);
      uint32_t holes = ~kept & low & below(x, hi), movers = kept & ~low;
      int32_t page = -1, first = 0;  // the page of the last place, its first slot
      auto slot = [&](uint32_t bit) {
        const int32_t j = lo + 32 * x + (int)bit;
        if (j >> page_log2 != page) {
          page = j >> page_log2;
          first = slot_of(page << page_log2);
        }
        return first < 0 ? -1 : first + (j & in_page);
      };
      for (; holes; holes &= holes - 1u) moves.dst[at + h++] = slot(__ffs(holes) - 1);
      for (; movers; movers &= movers - 1u) moves.src[at + m++] = slot(__ffs(movers) - 1);
    }
  }
  if (size > 1) cluster_wait();
}

// A warp takes kRows rows at a time, 16 bytes a lane and load; the list's entries of
// its next rows are on their way while it copies.
template <int D, bool V>
__global__ void __launch_bounds__(256) move_kernel(Moves moves, int64_t list_len, uint4* k_pages,
                                                   uint4* v_pages, const float* w, float* w_out,
                                                   Counters counts, int64_t n_slots) {
  constexpr int kPieces = D / 8;                     // of a row
  constexpr int kRows = (V ? 128 : 256) / kPieces;   // 8 loads a lane
  constexpr int kLoads = kRows * kPieces / 32;       // of a tensor
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int32_t listed = ld_input(counts.moves);
  const int64_t n = listed < 0 || listed > list_len ? list_len : listed;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 32) * kRows;
  int64_t x = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * kRows;
  // lane l < kRows has the slots of the rows x + l; src < 0: nothing to move
  int32_t src = -1, dst = 0;
  auto entry = [&](int64_t at) {
    src = -1;
    if (lane < kRows && at + lane < n) {
      src = ld_input(moves.src + at + lane);
      dst = ld_input(moves.dst + at + lane);
      // bad pages; and entries that no request wrote, where a page stands twice
      if ((uint32_t)src >= n_slots || (uint32_t)dst >= n_slots) src = -1;
    }
  };
  entry(x);
  for (; x < n; x += step) {
    uint4 a[kLoads], v[kLoads];
    int64_t to[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int piece = u * 32 + lane, r = piece / kPieces;
      const int32_t from = __shfl_sync(0xffffffffu, src, r), at = __shfl_sync(0xffffffffu, dst, r);
      to[u] = from < 0 ? -1 : (int64_t)at * kPieces + piece % kPieces;
      if (from < 0) continue;
      a[u] = ld_input(k_pages + (int64_t)from * kPieces + piece % kPieces);
      if (V) v[u] = ld_input(v_pages + (int64_t)from * kPieces + piece % kPieces);
    }
    const int32_t w_src = src, w_dst = dst;
    float weight = 0.f;
    if (w_src >= 0) weight = ld_input_f(w + w_src);
    entry(x + step);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (to[u] < 0) continue;
      k_pages[to[u]] = a[u];
      if (V) v_pages[to[u]] = v[u];
    }
    if (w_src >= 0) w_out[w_dst] = weight;
  }
  // the last block to end leaves the counters as the next call wants them
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(counts.ended, gridDim.x - 1) == gridDim.x - 1)
    *counts.moves = 0;
}

}  // namespace

size_t evict_ws(const ServeShape& s) { return 2 * round_up((size_t)max_moves(s), 64) * 4; }

cudaError_t launch_evict(const LaunchCtx& c, const ServeShape& s, const float* w_pages,
                         const int32_t* table, const int32_t* seq, const int32_t* keep,
                         int32_t n_first, int32_t n_last, __nv_bfloat16* k_pages,
                         __nv_bfloat16* v_pages, float* w_out, uint8_t* ws) {
  // a CTA for each 4096 tokens that a request may have, at most kMaxCluster, and a
  // thread for each four of its share
  const int64_t cap = (int64_t)s.max_blocks * s.page;
  int size = 1;
  while (size < kMaxCluster && cap > (int64_t)size * 4096) size *= 2;
  const int64_t share = ((cap + size - 1) / size + 31) & ~(int64_t)31;
  const int64_t words = share / 32;
  int threads = 256;
  while (threads < kMaxThreads && share > (int64_t)threads * 4) threads *= 2;
  const bool cached = share <= kMaxKeys;
  const size_t smem = (size_t)(2 * words + (cached ? share : 0)) * 4;
  cudaError_t e;
  static std::atomic<uint64_t> prepared{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxKeys * 4 + kMaxKeys / 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(select_kernel<false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxWordBytes);
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  const Moves moves = moves_of(s, ws);
  const Counters counts = counters(ws);
  const int64_t list_len = max_moves(s);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.B * size));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, cached ? select_kernel<true> : select_kernel<false>, w_pages,
                         table, seq, keep, n_first, n_last, w_out, moves, list_len, counts,
                         s.max_blocks, s.page_log2, s.n_pages, (int)words, c.status);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(c.num_sms * 4));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    return cudaLaunchKernelEx(&cfg, kern, moves, list_len, reinterpret_cast<uint4*>(k_pages),
                              reinterpret_cast<uint4*>(v_pages), w_pages, w_out, counts,
                              (int64_t)(s.n_pages * s.page));
  };
  if (v_pages) {
    if (s.D == 128) return run(move_kernel<128, true>);
    if (s.D == 256) return run(move_kernel<256, true>);
    return run(move_kernel<512, true>);
  }
  if (s.D == 128) return run(move_kernel<128, false>);
  if (s.D == 256) return run(move_kernel<256, false>);
  return run(move_kernel<512, false>);
}

}  // namespace dsa
