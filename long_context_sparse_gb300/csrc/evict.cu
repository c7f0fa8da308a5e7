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

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 49152;  // keys of a CTA's share that fit shared memory (192 KB)

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

// A cluster has a request, each CTA of it consecutive places.  Cached: their keys
// lie in shared memory, else they are read again in each pass.
template <bool Cached>
__global__ void __launch_bounds__(kSelThreads) select_kernel(
    const float* w, const int32_t* table, const int32_t* seq, const int32_t* keep,
    int32_t n_first, int32_t n_last, float* w_out, Moves moves, int64_t list_len,
    Counters counts, int max_blocks, int page_log2, int64_t n_pages, uint32_t* status) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];              // the digit of the threshold, keys above it
  __shared__ uint32_t warp_ties[kSelWarps], warp_holes[kSelWarps], warp_movers[kSelWarps];
  __shared__ uint32_t totals[2];             // holes and movers of this CTA
  __shared__ uint32_t first_move;            // of the request, in the leader
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int32_t share = (n + (int)size - 1) / (int)size;
  const int32_t lo = min(n, (int)rank * share), hi = min(n, lo + share);
  auto slot_of = [&](int32_t j) -> int32_t {
    const int32_t p = ld_input(row + (j >> page_log2));
    if (p < 0 || p >= n_pages) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      return -1;
    }
    return (p << page_log2) + (j & in_page);
  };
  if (left == n) {  // all stay
    if (w_out != w)
      for (int32_t j = lo + tid; j < hi; j += kSelThreads) {
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
  if (Cached)
    for (int32_t j = lo + tid; j < hi; j += kSelThreads) keys[j - lo] = read_key(j);

  // ---- the left-th largest key, eight bits at a time from the top
  uint32_t prefix = 0u;  // its bits so far
  uint32_t rest = (uint32_t)left;  // its rank among the keys with that prefix
  uint32_t ties = 0u;              // of this CTA, then of the CTAs before it
  for (int shift = 24; shift >= 0 && left > 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    for (int32_t j0 = lo; j0 < hi; j0 += kSelThreads) {
      const int32_t j = j0 + tid;
      const uint32_t k = j < hi ? key_of(j) : 0u;
      const bool in = j < hi && (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
      // equal digits of a warp count once
      const uint32_t d = in ? (k >> shift) & 255u : 256u;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (in && lane == __ffs(same) - 1) atomicAdd(hist + d, __popc(same));
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      // lane l sums digits 255 - 8 l .. 248 - 8 l over the cluster
      uint32_t c[8], sum = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = 0u;
        for (uint32_t r = 0; r < size; ++r)
          c[e] += ld_cluster(at_rank(smem_u32(hist + 255 - 8 * lane - e), r));
        sum += c[e];
      }
      uint32_t above = sum;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, above, s);
        if (lane >= s) above += x;
      }
      above -= sum;
      if (above < rest && rest <= above + sum) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (above < rest && rest <= above + c[e]) {
            found[0] = 255u - 8u * lane - e;
            found[1] = above;
          }
          above += c[e];
        }
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    rest -= found[1];
    if (shift == 0) {
      ties = 0u;
      for (uint32_t r = 0; r < rank; ++r) ties += ld_cluster(at_rank(smem_u32(hist + found[0]), r));
    }
    cluster_arrive();  // the histograms have been read
    cluster_wait();
  }
  // ---- `rest` of the keys equal to `prefix` stay, those of the lowest places
  const int32_t chunk = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int32_t w_lo = min(hi, lo + warp * chunk), w_hi = min(hi, w_lo + chunk);
  uint32_t mine = 0u;
  for (int32_t j = w_lo + lane; j < w_hi; j += 32) mine += left > 0 && key_of(j) == prefix;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) warp_ties[warp] = mine;
  __syncthreads();
  for (int x = 0; x < warp; ++x) ties += warp_ties[x];
  // which of the warp's places j0 .. j0 + 31 keep their token; ties: equal keys before
  auto kept_of = [&](int32_t j0, uint32_t& ties_before) {
    const int32_t j = j0 + lane;
    const uint32_t k = j < w_hi ? key_of(j) : 0u;
    const bool equal = j < w_hi && left > 0 && k == prefix;
    const uint32_t eq = __ballot_sync(0xffffffffu, equal);
    const bool stays = j < w_hi && left > 0 &&
                       (k > prefix ||
                        (equal && ties_before + __popc(eq & ((1u << lane) - 1u)) < rest));
    ties_before += __popc(eq);
    return __ballot_sync(0xffffffffu, stays);
  };
  // the lanes of j0 .. j0 + 31 whose places are below `end`
  auto below = [&](int32_t j0, int32_t end) {
    return end <= j0 ? 0u : end - j0 >= 32 ? 0xffffffffu : (1u << (end - j0)) - 1u;
  };
  uint32_t holes = 0u, movers = 0u, t = ties;
  for (int32_t j0 = w_lo; j0 < w_hi; j0 += 32) {
    const uint32_t kept = kept_of(j0, t), all = below(j0, w_hi), low = below(j0, left);
    holes += __popc(~kept & all & low);
    movers += __popc(kept & ~low);
  }
  if (lane == 0) {
    warp_holes[warp] = holes;
    warp_movers[warp] = movers;
  }
  __syncthreads();
  if (tid < 2) {
    uint32_t sum = 0u;
    for (int x = 0; x < kSelWarps; ++x) sum += tid ? warp_movers[x] : warp_holes[x];
    totals[tid] = sum;
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  uint32_t h = 0u, m = 0u;  // before this warp's
  for (int x = 0; x < warp; ++x) {
    h += warp_holes[x];
    m += warp_movers[x];
  }
  uint32_t all_moves = 0u;
  for (uint32_t r = 0; r < size; ++r) {
    const uint32_t a = ld_cluster(at_rank(smem_u32(totals), r));
    all_moves += a;
    if (r < rank) {
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
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  const uint32_t at = ld_cluster(at_rank(smem_u32(&first_move), 0));
  cluster_arrive();  // the leader's shared memory is no longer read after the wait below
  if (at != 0xffffffffu) {
    t = ties;
    for (int32_t j0 = w_lo; j0 < w_hi; j0 += 32) {
      const uint32_t kept = kept_of(j0, t), all = below(j0, w_hi), low = below(j0, left);
      const uint32_t hole = ~kept & all & low, mover = kept & ~low, me = 1u << lane;
      const uint32_t before = me - 1u;
      const int32_t j = j0 + lane;
      if (hole & me) moves.dst[at + h + __popc(hole & before)] = slot_of(j);
      if (mover & me) moves.src[at + m + __popc(mover & before)] = slot_of(j);
      if (w_out != w && (kept & low & me)) {
        const int32_t s = slot_of(j);
        if (s >= 0) w_out[s] = ld_input_f(w + s);
      }
      h += __popc(hole);
      m += __popc(mover);
    }
  }
  cluster_wait();
}

// One 16-byte piece of a row per thread and tensor, kUnroll in flight.
constexpr int kUnroll = 4;

template <int D>
__global__ void __launch_bounds__(256) move_kernel(
    Moves moves, int64_t list_len, uint4* k_pages, uint4* v_pages, const float* w, float* w_out,
    Counters counts, int64_t n_slots) {
  constexpr int kPieces = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t listed = ld_input(counts.moves);
  const int64_t n = (listed < 0 || listed > list_len ? list_len : listed) * (int64_t)kPieces;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t x0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x0 < n;
       x0 += kUnroll * step) {
    int32_t src[kUnroll], dst[kUnroll];  // src < 0: nothing to move
    uint4 a[kUnroll], v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t x = x0 + u * step;
      src[u] = -1;
      if (x < n) {
        src[u] = ld_input(moves.src + x / kPieces);
        dst[u] = ld_input(moves.dst + x / kPieces);
        // bad pages; and entries that no request wrote, where a page stands twice
        if ((uint32_t)src[u] >= n_slots || (uint32_t)dst[u] >= n_slots) src[u] = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (src[u] < 0) continue;
      const int64_t at = (int64_t)src[u] * kPieces + (x0 + u * step) % kPieces;
      a[u] = ld_input(k_pages + at);
      if (v_pages) v[u] = ld_input(v_pages + at);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (src[u] < 0) continue;
      const int64_t piece = (x0 + u * step) % kPieces, at = (int64_t)dst[u] * kPieces + piece;
      k_pages[at] = a[u];
      if (v_pages) v_pages[at] = v[u];
      if (piece == 0) w_out[dst[u]] = ld_input_f(w + src[u]);
    }
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
  // a CTA for each 4096 tokens that a request may have, at most kMaxCluster
  const int64_t cap = (int64_t)s.max_blocks * s.page;
  int size = 1;
  while (size < kMaxCluster && cap > (int64_t)size * 4096) size *= 2;
  const int64_t share = (cap + size - 1) / size;
  const bool cached = share <= kMaxKeys;
  const size_t smem = cached ? (size_t)share * 4 : 0;
  cudaError_t e;
  static std::atomic<uint64_t> prepared{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxKeys * 4);
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
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, cached ? select_kernel<true> : select_kernel<false>, w_pages,
                         table, seq, keep, n_first, n_last, w_out, moves, list_len, counts,
                         s.max_blocks, s.page_log2, s.n_pages, c.status);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(c.num_sms * 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    return cudaLaunchKernelEx(&cfg, kern, moves, list_len, reinterpret_cast<uint4*>(k_pages),
                              reinterpret_cast<uint4*>(v_pages), w_pages, w_out, counts,
                              (int64_t)(s.n_pages * s.page));
  };
  if (s.D == 128) return run(move_kernel<128>);
  if (s.D == 256) return run(move_kernel<256>);
  return run(move_kernel<512>);
}

}  // namespace dsa
