// evict.cu -- eviction from the paged cache by accumulated weight: which tokens
// stay (an exact radix select for each request), and the rows that move.
//
// A key has no position, so the tokens that stay need not keep their order: the
// request's cache shrinks to its first `left` places, whose dropped tokens' places
// are taken by the kept tokens from behind.  Places that are read (from `left` on)
// and places that are written (below it) are disjoint, so the rows move in place,
// in any order, and only about left (1 - left / n) of them move, where keeping the
// order would move nearly all.
//
// Bounds (in a graph).  64 requests of up to 4096 tokens of 512: 30 us with the pages' release
// (4), of which the copy 12 (73 MB) and the selection 15; 131071 tokens to 32768, K and V: 52
// us, of which the copy 17 (102 MB, 6 TB/s) and the selection 31.  The selection reads
// next to nothing: it is a chain of lookups, four histograms, their exchanges through the
// cluster (about 5000 cycles each with 16 CTAs), scans and a reservation.
#include <algorithm>
#include <atomic>

#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kMaxThreads = 1024;  // of a CTA of the selection
constexpr int kMaxCluster = 16;    // where the device has room for it, else 8
constexpr int kCopies = 8;         // of a histogram, for lanes that meet in a bin
constexpr int kMaxShare = 1 << 19;  // places of a CTA, at most: its masks take a bit each, twice
constexpr int kMaxSmem = 192 * 1024;  // of a CTA, beside the histograms (17 KB)
static_assert(kMaxSmem >= kMaxShare / 4 + 1024 * kMaxCluster, "masks and the cluster's counts");

// In the workspace header, behind the status word; both are 0 between calls.
struct Counters {
  // moves listed so far; past the list's end (where a page stands twice) none is made.
  // 64 bits: 65536 requests of 2^21 moves
  unsigned long long* moves;
  uint32_t* ended;  // blocks of the moving kernel that have ended
};
__host__ __device__ __forceinline__ Counters counters(uint8_t* ws) {
  return {reinterpret_cast<unsigned long long*>(ws + 64), reinterpret_cast<uint32_t*>(ws + 128)};
}

// Each move takes its row from a slot of its own (a request whose tokens on bad pages
// are to move lists none).  Where no page is bad, to one of its own too: half as many.
int64_t max_moves(const ServeShape& s) { return s.n_pages * s.page; }

struct Moves {
  int32_t *src, *dst;
};

// Of each slot's token the position in its request, and of each request the next one; or
// nullptr.
struct Ages {
  int32_t* pos;
  const int32_t* next;
};
// What a token is ranked by.
struct Ranked {
  float x;
  int32_t pos;
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
__device__ __forceinline__ uint64_t ld_input_u64(const unsigned long long* p) {
  uint64_t v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}

// A weight as an integer in the same order, the two zeros alike, NaN below all, but
// above kBadPage, the key of a token on a page outside the cache.
constexpr uint32_t kBadPage = 0u;
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  return w != w ? 1u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// The sum of x over the threads before this one, and over all of them; every thread
// of the CTA, `sums` [32] in shared memory, which may be used again after it.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* sums, uint64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint64_t incl = x;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint64_t o = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  uint64_t w = lane < warps ? sums[lane] : 0ull;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint64_t o = __shfl_up_sync(0xffffffffu, w, s);
    if (lane >= s) w += o;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return (warp ? before : 0ull) + incl - x;
}

// A cluster has a request, each CTA of it consecutive places.  Where their masks and keys
// fit `room` words the keys lie in shared memory, else they are read again in each pass.
//
// Passes of eight bits, four at most, find the left-th largest key: each CTA counts
// its keys, the cluster's leader adds up the counts, and a warp of it finds the
// digit.  Then a bit for each place says whether its token stays, and scans of
// population counts over groups of eight places number the equal keys, the freed
// places and the movers.
//
// The first (up to end_first) and the last n_last tokens are so by place or, Aged, by their
// positions, which are looked up beside the ranks (64 requests of 1500 to 4096 tokens, none
// protected: 21.1 us at 20.6; 131071 tokens 40.8 at 39.5).
template <bool Aged>
__global__ void __launch_bounds__(kMaxThreads) select_kernel(
    const float* w, const float* ranks, Ages ages, const int32_t* table, const int32_t* seq,
    const int32_t* keep, int32_t end_first, int64_t n_last, float* w_out, Moves moves,
    int64_t list_len, Counters counts, int max_blocks, int page_log2, int64_t n_pages,
    int32_t room, uint32_t* status) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  uint32_t* cluster_sums = smem;  // [CTA][256] where there are several: the leader's, by 16 bytes
  __shared__ alignas(16) uint32_t hist[2][kCopies][256];  // in turns
  __shared__ uint64_t sums[32];
  __shared__ alignas(16) uint32_t sum_hist[256];          // the leader's: of the cluster
  // the digit, keys above it, keys with it, and of those the ones in the CTAs before
  __shared__ uint32_t found[4];
  __shared__ uint32_t totals[2];          // freed places and movers of this CTA
  __shared__ uint32_t first_move;         // of the request, in the leader
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int b = blockIdx.x / size;
  for (int i = tid; i < kCopies * 64; i += nt)
    reinterpret_cast<uint4*>(hist[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  if (size > 1) cluster_arrive();  // this CTA has begun: its shared memory may be written to
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (size > 1) cluster_wait();
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
  uint32_t* above_w = smem + (size > 1 ? 256 * size : 0u);  // [word of 32 places] keys above
  uint32_t* equal_w = above_w + (share >> 5);               // the threshold; equal to it
  uint32_t* keys = equal_w + (share >> 5);
  const bool cached = share + (share >> 5) * 2 <= room;
  // the slot of place j on page p, or -1
  auto slot_on = [&](int32_t p, int32_t j) -> int32_t {
    if (p < 0 || p >= n_pages) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      return -1;
    }
    return (p << page_log2) + (j & in_page);
  };
  // f(j, slot, value(slot)) of the places j0, j0 + nt, .. below `end` that `which`
  // picks: kAhead pages, then kAhead values on their way at a time
  auto values_of = [&](auto value, int32_t j0, int32_t end, auto which, auto f) {
    constexpr int kAhead = 4;
    for (; j0 < end; j0 += kAhead * nt) {
      int32_t p[kAhead], s[kAhead];
      decltype(value(0)) x[kAhead];
      bool on[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int32_t j = j0 + u * nt;
        on[u] = j < end && which(j);
        if (on[u]) p[u] = ld_input(row + (j >> page_log2));
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        s[u] = on[u] ? slot_on(p[u], j0 + u * nt) : -1;
        if (s[u] >= 0) x[u] = value(s[u]);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (on[u]) f(j0 + u * nt, s[u], x[u]);
    }
  };
  auto any = [](int32_t) { return true; };
  auto weight = [&](int32_t s) { return ld_input_f(w + s); };
  auto ranked = [&](int32_t s) {
    return Ranked{ld_input_f(ranks + s), Aged ? ld_input(ages.pos + s) : 0};
  };
  if (left == n || left == 0) {  // all stay, or none
    if (w_out != w)
      values_of(weight, lo + tid, min(hi, left), any, [&](int32_t, int32_t s, float x) {
        if (s >= 0) w_out[s] = x;
      });
    return;
  }
  // the first of the last n_last, by position or by place
  const int32_t recent =
      (int32_t)max((Aged ? ld_input(ages.next + b) : n) - n_last, (int64_t)INT32_MIN);
  auto to_key = [&](int32_t j, int32_t s, const Ranked& r) {
    if (s < 0) return kBadPage;
    const int32_t at = Aged ? r.pos : j;
    return at <= end_first || at >= recent ? 0xff800000u /* +inf */ : order_key(r.x);
  };
  if (cached)
    values_of(ranked, lo + tid, hi, any,
              [&](int32_t j, int32_t s, const Ranked& r) { keys[j - lo] = to_key(j, s, r); });
  // f(j, key) of the places j0, j0 + nt, .. below hi
  auto each_key = [&](int32_t j0, auto f) {
    if (cached) {
#pragma unroll 4
      for (int32_t j = j0; j < hi; j += nt) f(j, keys[j - lo]);
    } else {
      values_of(ranked, j0, hi, any,
                [&](int32_t j, int32_t s, const Ranked& r) { f(j, to_key(j, s, r)); });
    }
  };

  // ---- the left-th largest key, eight bits at a time from the top
  uint32_t prefix = 0u;            // its bits so far, the rest 0
  uint32_t rest = (uint32_t)left;  // its rank among the keys with that prefix
  __syncthreads();
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass, turn = pass & 1;
    const uint32_t above = pass ? 0xffffffffu << (shift + 8) : 0u;
    uint32_t* mine = hist[turn][lane & (kCopies - 1)];
    each_key(lo + tid, [&](int32_t, uint32_t k) {
      if ((k & above) == prefix) atomicAdd(mine + ((k >> shift) & 255u), 1u);
    });
    __syncthreads();
    if (tid < 256) {
      uint32_t sum = 0u;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) sum += hist[turn][i][tid];
      if (size > 1) st_cluster_u32(at_rank(smem_u32(cluster_sums + rank * 256 + tid), 0), sum);
      else sum_hist[tid] = sum;
    }
    for (int i = tid; i < kCopies * 64; i += nt)  // for the next pass
      reinterpret_cast<uint4*>(hist[turn ^ 1])[i] = make_uint4(0u, 0u, 0u, 0u);
    if (size > 1) {
      cluster_arrive();
      cluster_wait();
      if (rank == 0 && tid < 256) {
        uint32_t sum = 0u;
#pragma unroll 8
        for (uint32_t r = 0; r < size; ++r) sum += cluster_sums[r * 256 + tid];
        sum_hist[tid] = sum;
      }
    }
    if (rank == 0) __syncthreads();
    if (warp == 0 && rank == 0) {
      const int d0 = 8 * (31 - lane);  // lane l has the digits d0 .. d0 + 7
      const uint4 a = *reinterpret_cast<const uint4*>(sum_hist + d0);
      const uint4 c = *reinterpret_cast<const uint4*>(sum_hist + d0 + 4);
      const uint32_t n8[8] = {c.w, c.z, c.y, c.x, a.w, a.z, a.y, a.x};  // digits downwards
      uint32_t sum = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += n8[e];
      uint32_t before = sum;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, before, s);
        if (lane >= s) before += o;
      }
      before -= sum;
      const uint32_t who =
          __ballot_sync(0xffffffffu, before < rest && rest <= before + sum);
      uint32_t digit = 0u, over = 0u, with = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < rest && rest <= before + n8[e]) {
          digit = (uint32_t)(d0 + 7 - e);
          over = before;
          with = n8[e];
        }
        before += n8[e];
      }
      digit = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
      over = __shfl_sync(0xffffffffu, over, __ffs(who) - 1);
      with = __shfl_sync(0xffffffffu, with, __ffs(who) - 1);
      if (size > 1) {
        // lane r: to CTA r, with the keys of the CTAs before it that share the prefix
        const uint32_t mine = lane < (int)size ? cluster_sums[lane * 256 + digit] : 0u;
        uint32_t ties = mine;
#pragma unroll
        for (int s = 1; s < kMaxCluster; s <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, ties, s);
          if (lane >= s) ties += o;
        }
        if (lane < (int)size) {
          const uint32_t at = at_rank(smem_u32(found), lane);
          st_cluster_u32(at, digit);
          st_cluster_u32(at + 4, over);
          st_cluster_u32(at + 8, with);
          st_cluster_u32(at + 12, ties - mine);
        }
      } else if (lane == 0) {
        found[0] = digit;
        found[1] = over;
        found[2] = with;
        found[3] = 0u;
      }
    }
    if (size > 1) {
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
    prefix |= found[0] << shift;
    rest -= found[1];
    if (rest == found[2]) break;  // all keys with this prefix stay: the same in the cluster
  }
  const bool all_ties = rest == found[2];
  const uint32_t ties = found[3];

  // ---- which keys are above the threshold, which equal to it: a bit each
  const int words = (hi - lo + 31) >> 5;
  {
    const int32_t first = lo + 32 * warp + lane;  // whole warps, in step
    auto flags = [&](int32_t j, uint32_t k) {
      const uint32_t gt = __ballot_sync(0xffffffffu, j < hi && k > prefix);
      const uint32_t eq = __ballot_sync(0xffffffffu, j < hi && k == prefix);
      if (lane == 0) {
        above_w[(j - lo) >> 5] = gt;
        equal_w[(j - lo) >> 5] = eq;
      }
    };
#pragma unroll 4
    for (int32_t j = first; j - lane < hi; j += nt) {
      uint32_t k = 0u;
      if (j < hi) {
        if (cached) k = keys[j - lo];
        else {
          const int32_t s = slot_on(ld_input(row + (j >> page_log2)), j);
          k = s < 0 ? kBadPage : to_key(j, s, ranked(s));
        }
      }
      flags(j, k);
    }
  }
  __syncthreads();
  // ---- `rest` of the equal ones stay, those of the lowest places; each thread has
  // consecutive groups of eight places
  uint8_t* above_b = reinterpret_cast<uint8_t*>(above_w);
  uint8_t* equal_b = reinterpret_cast<uint8_t*>(equal_w);
  const int groups = 4 * words, each = (groups + nt - 1) / nt;
  const int x0 = min(groups, tid * each), x1 = min(groups, x0 + each);
  // the page of this thread's first group, on its way meanwhile
  int32_t page = x0 < x1 && lo + 8 * x0 < n ? ld_input(row + ((lo + 8 * x0) >> page_log2)) : -1;
  uint64_t all;
  if (!all_ties) {
    uint32_t eq = 0u;
    for (int x = x0; x < x1; ++x) eq += __popc(equal_b[x]);
    uint32_t at = ties + (uint32_t)block_scan(eq, sums, &all);
    for (int x = x0; x < x1; ++x) {
      uint32_t e = equal_b[x], stay = 0u;
      for (; e && at < rest; ++at) {
        stay |= e & (0u - e);
        e &= e - 1u;
      }
      at += __popc(e);
      equal_b[x] = (uint8_t)stay;
    }
  }
  // the places of group x that are below `end`
  auto below = [&](int x, int32_t end) {
    const int32_t m = end - lo - 8 * x;
    return m <= 0 ? 0u : m >= 8 ? 0xffu : (1u << m) - 1u;
  };
  uint64_t mine = 0ull;  // freed places, movers << 32
  for (int x = x0; x < x1; ++x) {
    const uint32_t kept = above_b[x] | equal_b[x], low = below(x, left);
    above_b[x] = (uint8_t)kept;
    mine += __popc(~kept & low & below(x, hi)) + ((uint64_t)__popc(kept & ~low) << 32);
  }
  mine = block_scan(mine, sums, &all);
  uint32_t h = (uint32_t)mine, m = (uint32_t)(mine >> 32);
  if (tid == 0) {
    totals[0] = (uint32_t)all;
    totals[1] = (uint32_t)(all >> 32);
  }
  __syncthreads();
  if (size > 1) {
    cluster_arrive();
    cluster_wait();
    // lane r has CTA r's
    uint32_t freed = 0u, movers = 0u;
    if (lane < (int)size) {
      freed = ld_cluster(at_rank(smem_u32(totals), lane));
      movers = ld_cluster(at_rank(smem_u32(totals + 1), lane));
    }
    h += __reduce_add_sync(0xffffffffu, lane < (int)rank ? freed : 0u);
    m += __reduce_add_sync(0xffffffffu, lane < (int)rank ? movers : 0u);
    all = __reduce_add_sync(0xffffffffu, freed);
  }
  if (rank == 0 && tid == 0) {
    // where tokens on bad pages stay, all others do, and those that leave are on bad pages
    // too: nothing to copy
    const uint32_t count = prefix == kBadPage ? 0u : (uint32_t)all;
    const uint64_t at = count ? atomicAdd(counts.moves, (unsigned long long)count) : 0ull;
    // a page that stands in two places: more moves than the cache has slots for
    const bool fits = at + count <= (uint64_t)list_len;
    if (!fits) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    first_move = fits && count ? (uint32_t)at : 0xffffffffu;
  }
  if (w_out != w) {
    // the tokens that stay where they are; each CTA has as many places below `left`,
    // whosever share they lie in
    const int32_t part = (left + (int)size - 1) / (int)size, from = min(left, (int)rank * part);
    values_of(
        weight, from + tid, min(left, from + part),
        [&](int32_t j) {
          const uint32_t r = (uint32_t)(j / share), i = (uint32_t)(j - (int)r * share);
          return (ld_cluster(at_rank(smem_u32(above_w + (i >> 5)), r)) >> (i & 31u) & 1u) != 0u;
        },
        [&](int32_t, int32_t s, float x) {
          if (s >= 0) w_out[s] = x;
        });
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
      const int32_t j = lo + 8 * x;  // eight places lie on one page
      const uint32_t kept = above_b[x], low = below(x, left);
      uint32_t holes = ~kept & low & below(x, hi), movers = kept & ~low;
      if (x > x0 && (holes | movers)) page = ld_input(row + (j >> page_log2));
      const int32_t slot = holes | movers ? slot_on(page, j) : -1;
      for (; holes; holes &= holes - 1u, ++h)
        if (DSA_IN_BOUNDS(at + h < list_len, status))
          moves.dst[at + h] = slot < 0 ? -1 : slot + __ffs(holes) - 1;
      for (; movers; movers &= movers - 1u, ++m)
        if (DSA_IN_BOUNDS(at + m < list_len, status))
          moves.src[at + m] = slot < 0 ? -1 : slot + __ffs(movers) - 1;
    }
  }
  if (size > 1) cluster_wait();
}

constexpr int kMoveBlocks = 5;  // on an SM

// A warp takes kRows rows at a time, 16 bytes a lane and load; the list's entries of
// its next rows are on their way while it copies.
template <int D, bool V>
__global__ void __launch_bounds__(256, kMoveBlocks)
    move_kernel(Moves moves, int64_t list_len, uint4* k_pages, uint4* v_pages, const float* w,
                float* w_out, int32_t* pos, Counters counts, int64_t n_slots) {
  constexpr int kPieces = D / 8;                     // of a row
  constexpr int kRows = (V ? 64 : 128) / kPieces;    // 4 loads a lane
  constexpr int kLoads = kRows * kPieces / 32;       // of a tensor
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  // (past the list's end: the requests that did not fit are not in it, and what stands
  // in their place is an older call's)
  const uint64_t listed = ld_input_u64(counts.moves);
  const int64_t n = listed > (uint64_t)list_len ? 0 : (int64_t)listed;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 32) * kRows;
  int64_t x = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * kRows;
  // lane l < kRows has the slots of the rows x + l; src < 0: nothing to move
  int32_t src = -1, dst = 0;
  auto entry = [&](int64_t at) {
    src = -1;
    if (lane < kRows && at + lane < n) {
      src = ld_input(moves.src + at + lane);
      dst = ld_input(moves.dst + at + lane);
      // (a move to a bad page)
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
    int32_t place = 0;
    if (w_src >= 0) {
      weight = ld_input_f(w + w_src);
      if (pos) place = ld_input(pos + w_src);
    }
    entry(x + step);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (to[u] < 0) continue;
      k_pages[to[u]] = a[u];
      if (V) v_pages[to[u]] = v[u];
    }
    if (w_src >= 0) {
      w_out[w_dst] = weight;
      if (pos) pos[w_dst] = place;
    }
  }
  // the last block to end leaves the counters as the next call wants them
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(counts.ended, gridDim.x - 1) == gridDim.x - 1)
    *counts.moves = 0ull;
}

// Whether a cluster of kMaxCluster of the selection's largest CTAs finds room.
template <bool Aged>
bool fits_wide(int smem) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCluster);
  cfg.blockDim = dim3(kMaxThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, select_kernel<Aged>, &cfg) == cudaSuccess) return n > 0;
  cudaGetLastError();
  return false;
}

// Once on a device: whether clusters of the selection may have kMaxCluster CTAs.
template <bool Aged>
cudaError_t prepare(int device, bool* is_wide) {
  static std::atomic<uint64_t> prepared{0}, wide{0};
  const uint64_t bit = 1ull << (device & 63);
  if (!(prepared.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(select_kernel<Aged>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(select_kernel<Aged>,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (fits_wide<Aged>(kMaxSmem)) wide.fetch_or(bit, std::memory_order_relaxed);
    prepared.fetch_or(bit, std::memory_order_release);
  }
  *is_wide = wide.load(std::memory_order_relaxed) & bit;
  return cudaSuccess;
}

}  // namespace

size_t evict_ws(const ServeShape& s) { return 2 * round_up((size_t)max_moves(s), 64) * 4; }

cudaError_t launch_evict(const LaunchCtx& c, const ServeShape& s, const float* w_pages,
                         const float* rank_pages, int32_t* pos_pages, const int32_t* next_pos,
                         const int32_t* table, const int32_t* seq, const int32_t* keep,
                         int64_t n_first, int64_t n_last, __nv_bfloat16* k_pages,
                         __nv_bfloat16* v_pages, float* w_out, uint8_t* ws) {
  const bool aged = pos_pages != nullptr;
  bool wide;
  cudaError_t e = aged ? prepare<true>(c.device, &wide) : prepare<false>(c.device, &wide);
  if (e != cudaSuccess) return e;
  // A CTA for each 4096 tokens that a request may have, at most kMaxCluster, while an SM
  // has one (which a CTA of 1024 threads takes to itself): a cache is seldom as long as it
  // may get, and clusters that queue for SMs cost all.  us of the call with CTAs up to
  // one, two an SM and without that limit: 64 requests of up to 4096 tokens that may have
  // 131072 21 32 117; 16 of up to 65536 85 112 111; 64 of 100000 to 131072 730 686 -.  One
  // request of 131071 with 4, 8, 16 CTAs 75 54 47; 64 that may have 4096 with 1, 2, 4, 8
  // CTAs 23.1 25.7 25.8 28.5.  A thread for each four places of a share (for 64 of 4096
  // 23.1, with eight 24.0, with sixteen 27.7).
  const int64_t cap = (int64_t)s.max_blocks * s.page;
  const int most = wide ? kMaxCluster : 8;
  int size = 1;
  while (size < most && ((cap > (int64_t)size * 4096 && s.B * size * 2 <= c.num_sms) ||
                         cap > (int64_t)size * kMaxShare))
    size *= 2;
  const int64_t share = ((cap + size - 1) / size + 31) & ~(int64_t)31;
  int threads = 256;
  while (threads < kMaxThreads && share > (int64_t)threads * 4) threads *= 2;
  // Masks of the longest cache, and its keys or as many as there is room for: a share whose
  // keys take more than half an SM's shared memory has a CTA of 1024 threads, whose registers
  // leave no room for a second one (200 requests of 20000 to 32768 tokens to 8192: 185 us,
  // with half the memory and keys read again in each pass 210).
  const int64_t sums = size > 1 ? 1024 * size : 0, masks = share / 4;
  const int64_t full = sums + masks + share * 4;
  const int64_t smem = full <= kMaxSmem ? full : kMaxSmem;
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
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, aged ? select_kernel<true> : select_kernel<false>, w_pages,
                         rank_pages, Ages{pos_pages, next_pos}, table, seq, keep,
                         (int32_t)std::min(n_first - 1, (int64_t)INT32_MAX), n_last, w_out,
                         moves, list_len, counts, s.max_blocks, s.page_log2, s.n_pages,
                         (int32_t)((smem - sums) / 4), c.status);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(c.num_sms * kMoveBlocks));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    return cudaLaunchKernelEx(&cfg, kern, moves, list_len, reinterpret_cast<uint4*>(k_pages),
                              reinterpret_cast<uint4*>(v_pages), w_pages, w_out, pos_pages, counts,
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
