// key_weights.cu -- what the cached tokens of each request receive of its rows'
// attention: w[j] = sum over the rows r that see j of exp(scale q_r . k_j - lse_r),
// on 5th-generation tensor cores by pairs of SMs.
//
// Products of a tile of 256 keys, by a cluster of two CTAs (cta_group::2, M = 256),
// with the keys on the accumulator's lanes and up to 256 (token, head) rows as
// columns:  S^T[key, row] = K_tile . Q^T.  A thread has one key, so a key's sum
// over the rows never leaves it: no exchange, no atomics on sums.  Each CTA holds
// its 128 keys' K, which stay while the request's row blocks come by, and half of
// each block's Q: 32 KB of Q brought in by each CTA of a pair at d = 512 feed 512
// cycles of MMAs times 8, where a CTA alone would take in twice as much.
//
// Work.  A unit is a key tile against a row block, in order of request, tile, block;
// units cost what bounds them (K's way from HBM, or the MMAs) and the pairs share
// the sum evenly.  A tile whose blocks fall to several pairs is joined by the last
// of them to end, which adds their sums in the order of the pairs, so that results
// repeat.
//
// Warps.  A planner walks through the units and tells the others of the next four: what
// to load, the pages, -lse.  One warp loads K, one Q; a scout lets the issuer in to the
// chunks (64 dims) that are there; eight warps take the accumulators, two of 256 columns
// in turns, exponentiate and add up.
//
// Numbers.  Scores, weights and sums are fp32.  A score is off by as much as 2^-22 of the sum
// of its |q_i k_i| scale, as measured: so the tensor cores add up d products (1e-5 at d = 512
// and scores up to 14, where fp32 products added one after the other are off by 1.6e-6).  A
// weight is off by that times itself, a sum of many by fp32's own roundings too.  Over 70
// batches the errors were 2e-8 to 1.5e-6 of the norm of all weights.
//
// Bounds (in a graph; eager calls one after the other take 10 us at least).  64 requests of one
// token, 64 heads of 512, up to 8192 tokens: 49 us for 275 MB, 5 of them to start, then 6.3
// TB/s.  Windows of 20 to 64 tokens over up to 20000: 67 to 72 us (eager 73 to 79) for 117
// GFLOP (68% of the time the tensor pipe works); a chunk of 256 columns takes its MMAs 512
// cycles, and the reads of TMEM beside them hold them up.  Small units: 16 rows against 100
// tokens 1.5 us each at d = 128 and 2.0 at d = 512, of a planner's step, loads, MMAs and sums
// one behind the other.  d = 128: the exponentials (64 trees of 8 nodes, 64 heads, up to 4000
// tokens: 35 us, of which 14 are theirs alone).
#include <atomic>

#include "attn_common.cuh"
#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kTile = 256;          // keys of a pair's tile
constexpr int kBlock = 256;         // rows of a unit, at most
constexpr int kMaxPairs = 80;
constexpr int kEpiWarps = 8;        // 4 TMEM lane quadrants x 2 sets of columns
constexpr int kKWarp = 8, kScoutWarp = 9, kMmaWarp = 10, kQWarp = 11;
constexpr int kPlanWarp = 12;
constexpr int kThreads = 32 * 13;
constexpr int kKSlots = 8;          // of 128 keys x 64 dims
constexpr uint32_t kKBytes = 16384;
constexpr int kQParts = 20;         // of 32 rows x 64 dims; a chunk's slot has 1, 2 or 4
constexpr uint32_t kQBytes = 4096;
constexpr int kUnits = 4;           // units that are planned ahead
constexpr uint32_t kTail = 8192;
constexpr uint32_t kSmem = 1024 + kKSlots * kKBytes + kQParts * kQBytes + kTail;
constexpr int kBars = 2 * kKSlots + 2 * kQParts + 6 + 2 * kUnits;
// cost of a tile against few rows, in units of 512 cycles: its K comes from HBM in
// about 6000 (256 KB at d = 512 and at a pair's share of the rate), while the MMAs of
// 64 rows take 1024
constexpr int kTileCost = 12;

// What the issuer is to do with a chunk: its parts of Q << 8, K slot << 12, accumulator
// << 16, parts of a Q slot << 20, Q slot << 24, and
constexpr uint32_t kGo = 1, kFirst = 2, kLast = 4, kFreeK = 8, kFreeQ = 16;

// A unit as the planner tells it to the other warps of its CTA.
struct alignas(16) Unit {
  int32_t row0, rows;  // first of all rows, rows
  int32_t at;          // first row, from the request's
  int32_t pos;         // place of the tile's first key
  int32_t len, base;   // of the request
  uint32_t what;       // bits below; parts << 16, a slot's parts << 20
  uint32_t pairs;      // first and (<< 8) last pair that have units of the tile
  // first cache row of the pages of this CTA's keys; n_pages * page_size: none
  int32_t page_row[8];
};
constexpr uint32_t kDead = 1;    // no row of it sees a key of the tile
constexpr uint32_t kBegins = 2;  // the first of this pair's units of the tile
constexpr uint32_t kEnds = 4;    // the last of them
constexpr uint32_t kWhole = 8;   // (with kEnds) there are no others
constexpr uint32_t kLoadK = 16, kLoadQ = 32;
constexpr uint32_t kDropQ = 64;  // its Q is not used again
constexpr uint32_t kEnd = 128;   // no unit: there are no more

// Counters of the pairs that have ended with a tile that began in pair p: a byte
// each for the two CTAs, in the workspace header behind the status word.  0 between
// calls.
static_assert(64 + 2 * kMaxPairs <= (int)kHeader, "counters");

struct Args {
  const float* lse;
  const int32_t *table, *seq, *cu;
  const int32_t* bits;  // or nullptr
  int words;
  const float* w;
  float* w_out;
  float* parts;       // [pair][rank][head, tail][128]
  uint32_t* counters;
  float decay, scale;
  int B, H, max_blocks, page_log2;
  int64_t T, n_pages;
  uint32_t* status;
  uint64_t timeout_ns;
};

struct Req {
  int32_t row0, rows;  // first row (token * H), rows; rows < 0: offsets out of order or range
  int32_t len, base;   // own tokens; place of the step's first
  int32_t tiles, blocks;
  int32_t cost;        // of a unit
};

__device__ __forceinline__ Req load_req(const Args& a, int b) {
  const int32_t c0 = ld_input(a.cu + b), c1 = ld_input(a.cu + b + 1);
  int32_t len = ld_input(a.seq + b);
  if (len < 0 || len > a.max_blocks << a.page_log2) len = 0;  // latched by CTA 0
  // (compared before any difference or product of them, which may wrap)
  const bool ok = c0 >= 0 && c0 <= c1 && c1 <= a.T;
  Req r;
  r.row0 = ok ? c0 * a.H : 0;
  r.rows = ok ? (c1 - c0) * a.H : -1;
  r.len = len;
  r.base = ok ? len - (c1 - c0) : len;
  r.tiles = r.rows > 0 ? (len + kTile - 1) / kTile : 0;
  r.blocks = (r.rows + kBlock - 1) / kBlock;
  // (a division is a long chain; most requests have one block)
  r.cost = max(kTileCost, (r.rows + 63) / 64 * 2);
  if (r.blocks > 1) r.cost = (r.cost + r.blocks - 1) / r.blocks;
  return r;
}
__device__ __forceinline__ bool has_units(const Args& a, int b) {
  const int32_t len = ld_input(a.seq + b);
  return ld_input(a.cu + b) < ld_input(a.cu + b + 1) && len > 0 &&
         len <= a.max_blocks << a.page_log2;
}
__device__ __forceinline__ int64_t units_of(const Req& r) {
  return (int64_t)r.tiles * r.blocks;
}
__device__ __forceinline__ int64_t ceil_div(int64_t x, int64_t y) {
  return ((x | y) >> 31) == 0 ? (int64_t)(((uint32_t)x + (uint32_t)y - 1u) / (uint32_t)y)
                              : (x + y - 1) / y;
}

// The units of one pair's share [start, end) of the cost, in order: those whose cost
// begins there.  A whole warp, in step.
struct Walk {
  int64_t start, end, cb;  // cb: cost before request b
  int64_t left;            // units of request b still to come
  int32_t b, tile, block;
  bool first;              // no unit of request b so far
  Req r;

  // units of request b that begin before the share's end
  __device__ __forceinline__ int64_t units_before_end() const {
    const int64_t n = units_of(r);
    return n * r.cost <= end - cb ? n : ceil_div(end - cb, r.cost);
  }
  __device__ __forceinline__ void begin(const Args& a, int64_t s, int64_t e, int64_t c, int b0) {
    start = s;
    end = e;
    cb = c;
    b = b0;
    left = 0;
    first = true;
    tile = block = 0;
    r = Req{};
    r.cost = 1;
    if (s >= e) {
      end = cb = 0;
      return;
    }
    r = load_req(a, b);
    const int64_t u0 = s > cb ? ceil_div(s - cb, r.cost) : 0;
    left = units_before_end() - u0;
    if (left < 0) left = 0;
    if (r.blocks > 0) {
      tile = (int32_t)(u0 / r.blocks);
      block = (int32_t)(u0 - (int64_t)tile * r.blocks) - 1;  // next() goes one on
      if (block < 0) {
        block = r.blocks - 1;
        --tile;
      }
    }
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if (left > 0) {
      if (++block == r.blocks) {
        block = 0;
        ++tile;
      }
      --left;
      return true;
    }
    cb += units_of(r) * r.cost;
    if (cb >= end) return false;
    // the next request with units; idle ones are passed 32 at a time
    uint32_t some = 0;
    while (!some && ++b < a.B) {
      const int x = b + (int)(threadIdx.x & 31);
      some = __ballot_sync(0xffffffffu, x < a.B && has_units(a, x));
      b += some ? __ffs(some) - 1 : 31;
    }
    if (!some) return false;
    r = load_req(a, b);
    left = units_before_end() - 1;
    tile = block = 0;
    first = true;
    return true;
  }
  // rows of the unit, and the columns that they take
  __device__ __forceinline__ int32_t rows() const { return min(kBlock, r.rows - block * kBlock); }
  __device__ __forceinline__ int32_t parts() const {
    const int32_t n = rows();
    return n <= 64 ? 1 : n <= 128 ? 2 : 4;
  }
  // of a slot: the same for all blocks of the request
  __device__ __forceinline__ int32_t slot_parts() const { return r.blocks > 1 ? 4 : parts(); }
  // Q stays for all tiles of the request where it has one block and that fits
  template <int D>
  __device__ __forceinline__ bool q_stays() const {
    return r.blocks == 1 && parts() * (D / 64) <= kQParts;
  }
  // no row of the block sees a key of the tile
  __device__ __forceinline__ bool dead(const Args& a) const {
    return !a.bits &&
           (int64_t)(tile * kTile - r.base) * a.H > (int64_t)(block * kBlock + rows() - 1);
  }
  __device__ __forceinline__ bool tile_ends() const { return block == r.blocks - 1 || left == 0; }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
// The ring of Q: slots of `parts` parts.  When that changes it begins anew, once all
// slots of the old kind are free.  A bit for each barrier: the parity of its next use.
struct QRing {
  uint32_t parts = 4, count = kQParts / 4, at = 0, phase = 0;

  // whether slots of n parts are another kind
  __device__ __forceinline__ bool other(uint32_t n) const { return n != parts; }
  __device__ __forceinline__ void begin(uint32_t n) {
    parts = n;
    count = (uint32_t)kQParts / n;
    at = 0;
  }
  __device__ __forceinline__ uint32_t parity() const { return (phase >> at) & 1u; }
  // the slot of the c-th chunk from `from` on, and the parity of that use of it
  __device__ __forceinline__ uint32_t slot(uint32_t from, uint32_t c) const {
    uint32_t q = from + c;
    if (q >= count) q -= count;
    return q >= count ? q - count : q;  // 5 slots of 8 chunks: round twice
  }
  __device__ __forceinline__ uint32_t parity(uint32_t q, uint32_t c) const {
    return ((phase >> q) & 1u) ^ (c >= count ? 1u : 0u);
  }
  __device__ __forceinline__ void used(uint32_t n) {
    for (uint32_t u = ((1u << n) - 1u) << at; u; u >>= count) phase ^= u & ((1u << count) - 1u);
    at = slot(at, n);
  }
};
static_assert(kQParts / 4 * 2 >= 8 && kQParts + 8 < 32, "chunks that go round the ring");

// Bounded waits for what TMA and the tensor cores do, or for TMEM that has been
// read: no memory written by the other CTA's threads is read behind them, so that
// they need no acquisition beyond the CTA (as PairWaiter has it).
struct LocalWaiter {
  PairWaiter w;
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    const bool done = mbar_try_wait(bar, parity) || w.wait1(bar, parity);
    return __all_sync(0xffffffffu, done);
  }
};

// Whether the phase is over; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// How many chunks from `done` on are ready, of those below `end`, where bit c of `mask`
// says that of chunk c.
__device__ __forceinline__ uint32_t run_of(uint32_t mask, uint32_t done, uint32_t end) {
  return min((uint32_t)__ffs(~(mask >> done)) - 1u, end - done);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap q2_map,
                       const __grid_constant__ CUtensorMap q4_map,
                       const __grid_constant__ CUtensorMap k_map, const Args a) {
  constexpr int kChunks = D / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sK = (raw + 1023u) & ~1023u;
  const uint32_t sQ = sK + kKSlots * kKBytes;
  uint8_t* tail = smem_raw + (sK - raw) + kKSlots * kKBytes + kQParts * kQBytes;
  Unit* units = reinterpret_cast<Unit*>(tail);
  float* neg_s = reinterpret_cast<float*>(units + kUnits);  // [unit % kUnits][column] -lse
  float* red_s = neg_s + kUnits * kBlock;          // [tile & 1][key] the other columns' sums
  uint32_t* live_s = reinterpret_cast<uint32_t*>(red_s + 256);  // [unit][8] columns that count
  uint64_t* bars = reinterpret_cast<uint64_t*>(live_s + 8 * kUnits);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + kBars);  // abort, tmem, joins
  volatile uint32_t* cmd = misc + 4;                           // [turn & 1][8], see the scout
  int64_t* scratch = reinterpret_cast<int64_t*>(misc + 20);   // [16], then the share
  static_assert(kUnits * (sizeof(Unit) + 4 * kBlock + 32) + 1024 + kBars * 8 + 80 + 24 * 8 <= kTail,
                "tail");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const uint32_t bar0 = smem_u32(bars);
  auto k_full = [&](uint32_t s) { return bar0 + 8u * s; };               // leader: both landed
  auto k_empty = [&](uint32_t s) { return bar0 + 8u * (kKSlots + s); };
  auto q_full = [&](uint32_t s) { return bar0 + 8u * (2 * kKSlots + s); };  // leader
  auto q_empty = [&](uint32_t s) { return bar0 + 8u * (2 * kKSlots + kQParts + s); };
  const uint32_t bx = bar0 + 8u * (2 * kKSlots + 2 * kQParts);
  auto s_full = [&](uint32_t u) { return bx + 8u * (u & 1u); };
  auto s_empty = [&](uint32_t u) { return bx + 16 + 8u * (u & 1u); };    // leader
  const uint32_t epi = bx + 32, done_bar = bx + 40;
  auto u_full = [&](uint32_t n) { return bx + 48 + 8u * (n % kUnits); };
  auto u_empty = [&](uint32_t n) { return bx + 48 + 8u * (kUnits + n % kUnits); };
  const LocalWaiter W{{misc, at_rank(smem_u32(misc), peer), a.status, a.timeout_ns}};

  if (tid == 0) {
    for (uint32_t s = 0; s < kKSlots; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (uint32_t s = 0; s < kQParts; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
    }
    for (uint32_t u = 0; u < 2; ++u) {
      mbar_init(s_full(u), 1);
      mbar_init(s_empty(u), 2 * kEpiWarps);
    }
    for (uint32_t u = 0; u < kUnits; ++u) {
      mbar_init(u_full(u), 1);
      mbar_init(u_empty(u), kEpiWarps + (rank == 0 ? 3 : 2));  // K, Q; scout
    }
    mbar_init(epi, kEpiWarps);
    mbar_init(done_bar, 1);
    misc[0] = 0u;
    scratch[16] = scratch[17] = 0;  // the share, should the lengths change under the kernel
    fence_mbar_init();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(misc + 1)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_arrive();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this pair's share of the cost, and the request where it begins.  Up to 32
  // requests: the planner by itself, while the others go on to wait for it.  More: all
  // threads, kThreads requests at a time, once for the sum and, where that took more than
  // one turn, again up to the share's start.
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  int64_t total = 0, chunk = 0, start = 0, end = 0;
  int64_t first_cost = 0;  // cost before the request
  int first_b = 0;         // its number
  {
    // the cost of request b
    auto cost_of = [&](int b, int& bad) -> int64_t {
      if (b >= a.B) return 0;
      const Req r = load_req(a, b);
      bad |= r.rows < 0;
      const int32_t n = blockIdx.x == 0 ? ld_input(a.seq + b) : 0;
      if (n < 0 || n > a.max_blocks << a.page_log2)
        latch_error(a.status, DSA_ERR_DEVICE_BAD_INDEX);
      return units_of(r) * r.cost;
    };
    auto before = [&](int64_t x) {  // the sum over this lane and those before it
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x += o;
      }
      return x;
    };
    auto divide = [&](int bad, int64_t all) {
      total = bad ? 0 : all;  // offsets that do not ascend within [0, T]: nothing is computed
      if (bad && blockIdx.x == 0 && lane == 0) latch_error(a.status, DSA_ERR_DEVICE_BAD_INDEX);
      // (a share of a unit's cost at least: then the pairs of a tile have no gap)
      chunk = max(ceil_div(total, pairs), (int64_t)kTileCost);
      start = min(total, pair * chunk);
      end = min(total, start + chunk);
    };
    int bad = 0;
    if (a.B <= 32) {
      if (warp == kPlanWarp) {
        const int64_t mine = cost_of(lane, bad), incl = before(mine);
        divide(__any_sync(0xffffffffu, bad), __shfl_sync(0xffffffffu, incl, 31));
        const uint32_t who = __ballot_sync(0xffffffffu, start < end && incl > start);
        first_b = who ? __ffs(who) - 1 : 0;  // the first whose end is beyond it
        first_cost = __shfl_sync(0xffffffffu, incl - mine, first_b);
      }
    } else {
      int64_t mine = 0, incl = 0, all = 0;  // of the last turn
      auto turn = [&](int b0) {
        mine = cost_of(b0 + tid, bad);
        incl = before(mine);
        if (lane == 31) scratch[warp] = incl;
        __syncthreads();
        all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w == warp) incl += all;
          all += scratch[w];
        }
        __syncthreads();
      };
      int64_t sum = 0;
      for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        turn(b0);
        sum += all;
      }
      divide(__syncthreads_or(bad), sum);
      int64_t* share = scratch + 16;
      int64_t c = 0;
      for (int b0 = 0; b0 < a.B && start < end && c <= start; b0 += kThreads) {
        if (a.B > kThreads) turn(b0);
        const int64_t c0 = c + incl - mine;
        if (c0 <= start && start < c0 + mine) {
          share[0] = c0;
          share[1] = b0 + tid;
        }
        c += all;
      }
      __syncthreads();
      first_cost = share[0];
      first_b = (int)share[1];
    }
  }
  cluster_wait();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // an allocation of all 512 columns starts at column 0
  const int page = 1 << a.page_log2, nb_log2 = 7 - a.page_log2;
  const int nb = 1 << nb_log2;  // page boxes of a chunk
  const int32_t no_row = (int32_t)(a.n_pages << a.page_log2);  // out of range: zeros
  // the n-th unit, for those that are told of it
  auto unit = [&](uint32_t n, Unit& u) {
    if (!W.wait(u_full(n), (n / kUnits) & 1u)) return false;
    const uint4* from = reinterpret_cast<const uint4*>(units + n % kUnits);
    reinterpret_cast<uint4*>(&u)[0] = from[0];
    reinterpret_cast<uint4*>(&u)[1] = from[1];
    return !(u.what & kEnd);
  };
  auto seen = [&](uint32_t n) {  // by this warp, which does not look at it again
    __syncwarp();
    if (lane == 0) mbar_arrive(u_empty(n));
  };

  if (warp == kPlanWarp) {
    // ====== planner: walks through the units, a unit ahead of what it tells, so that
    // its questions to memory (lengths, pages, lse) are answered by then.  (A step to
    // another request is some 700 cycles of one warp, which small units do not hide: 760
    // requests of up to 100 tokens at d = 128 take 19.9 us, and 24.2 with a walk in each
    // warp.)
    Walk walk;
    walk.begin(a, start, end, first_cost, first_b);
    float l[kBlock / 32] = {};
    int32_t page_id = -1, row = no_row;
    uint32_t nu = 0;
    bool ok = true, have = false, k_here = false, head = false;
    for (bool started = false;; started = true) {
      const Walk x = walk;
      const bool told = have;
      float neg[kBlock / 32];
#pragma unroll
      for (int i = 0; i < kBlock / 32; ++i) neg[i] = -l[i];
      const int32_t id = page_id;
      if (told) walk.first = false;
      if (!started || told) {
        have = walk.next(a);
        if (have) {
          const int32_t n = walk.dead(a) ? 0 : walk.rows();
          const int32_t* from =
              reinterpret_cast<const int32_t*>(a.lse) + walk.r.row0 + walk.block * kBlock;
#pragma unroll
          for (int i = 0; i < kBlock / 32; ++i) {
            l[i] = -INFINITY;
            if (32 * i + lane < n) l[i] = __int_as_float(ld_input(from + 32 * i + lane));
          }
          if (walk.block == 0 || walk.first) {
            const int32_t pos = walk.tile * kTile + (int)rank * 128 + lane * page;
            page_id = 0;
            if (lane < nb && pos < walk.r.len)
              page_id = ld_input(a.table + (int64_t)walk.b * a.max_blocks + (pos >> a.page_log2));
          }
        }
      }
      if (!told) {
        if (started || !have) break;
        continue;
      }
      uint32_t what = (x.dead(a) ? kDead : 0u) | (x.tile_ends() ? kEnds : 0u);
      if (x.block == 0 || x.first) {
        what |= kBegins;
        k_here = false;
        head = x.block != 0;  // the tile began in a pair before
        row = no_row;
        if (lane < nb && x.tile * kTile + (int)rank * 128 + lane * page < x.r.len) {
          if (id < 0 || id >= a.n_pages) latch_error(a.status, DSA_ERR_DEVICE_BAD_INDEX);
          else row = id << a.page_log2;
        }
      }
      if (what == kDead) continue;
      const bool stays = x.q_stays<D>();
      if (!(what & kDead)) {
        if (!k_here) what |= kLoadK;
        k_here = true;
        if (!stays || x.first) what |= kLoadQ;
        if (!stays || x.left == 0) what |= kDropQ;
      }
      uint32_t between = 0;
      if (what & kEnds) {
        if (!head && x.block == x.r.blocks - 1) {
          what |= kWhole;
        } else {
          const int64_t c0 = x.cb + (int64_t)x.tile * x.r.blocks * x.r.cost;
          between = (uint32_t)(c0 / chunk) |
                    (uint32_t)((c0 + (int64_t)(x.r.blocks - 1) * x.r.cost) / chunk) << 8;
        }
      }
      if (!(ok = W.wait(u_empty(nu), ((nu / kUnits) & 1u) ^ 1u))) break;
      Unit* u = units + nu % kUnits;
      if (lane == 0) {
        u->row0 = x.r.row0 + x.block * kBlock;
        u->rows = x.rows();
        u->at = x.block * kBlock;
        u->pos = x.tile * kTile;
        u->len = x.r.len;
        u->base = x.r.base;
        u->what = what | (uint32_t)x.parts() << 16 | (uint32_t)x.slot_parts() << 20;
        u->pairs = between;
      }
      if (lane < nb) u->page_row[lane] = row;
#pragma unroll
      for (int i = 0; i < kBlock / 32; ++i) {
        neg_s[nu % kUnits * kBlock + 32 * i + lane] = neg[i];
        const uint32_t live = __ballot_sync(0xffffffffu, neg[i] != INFINITY);
        if (lane == 0) live_s[nu % kUnits * 8 + i] = live;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(u_full(nu));
      ++nu;
    }
    if (ok && W.wait(u_empty(nu), ((nu / kUnits) & 1u) ^ 1u)) {
      if (lane == 0) {
        units[nu % kUnits].what = kEnd;
        mbar_arrive(u_full(nu));
      }
      __syncwarp();
    }
  } else if (warp == kKWarp) {
    // ============================================================ K by TMA
    const uint32_t lead = at_rank(bar0, 0);
    uint32_t kc = 0;  // chunks so far
    bool ok = true;
    Unit u;
    for (uint32_t nu = 0; ok && unit(nu, u); ++nu) {
      const int32_t row = units[nu % kUnits].page_row[lane & (nb - 1)];
      seen(nu);
      if (!(u.what & kLoadK)) continue;
      // boxes behind the last token are left out: what lies there gives sums of keys
      // that are not, and stays with them
      const int32_t keys = min(kTile, u.len - u.pos);
      const uint32_t bytes = (uint32_t)((keys + page - 1) & -page) * 128u;
      const int32_t boxes = (keys - (int)rank * 128 + page - 1) >> a.page_log2;  // of this CTA
      // all chunks whose slots are free at once: lane c looks at chunk c's, and the lanes
      // take the boxes of them
      const uint32_t mine = kc + (uint32_t)lane;
      uint32_t done = 0;
      while (done < kChunks) {
        const bool is = lane < kChunks && mbar_test(k_empty(mine % kKSlots),
                                                    ((mine / kKSlots) & 1u) ^ 1u);
        uint32_t n = run_of(__ballot_sync(0xffffffffu, is), done, kChunks);
        if (n == 0) {
          const uint32_t x = kc + done;
          if (!(ok = W.wait(k_empty(x % kKSlots), ((x / kKSlots) & 1u) ^ 1u))) break;
          n = 1;
        }
        if (rank == 0 && (uint32_t)lane - done < n) mbar_expect_tx(k_full(mine % kKSlots), bytes);
        for (uint32_t i = 0; i < n << nb_log2; i += 32) {
          const uint32_t c = done + ((i + lane) >> nb_log2), box = lane & (nb - 1);
          if (c < done + n && (int32_t)box < boxes) {
            const uint32_t s = (kc + c) % kKSlots;
            tma_load_pair(sK + s * kKBytes + box * (uint32_t)page * 128u, &k_map, (int)c * 64, row,
                          lead + 8u * s);
          }
        }
        done += n;
      }
      kc += kChunks;
    }
    // the leader's last arrival here is done_bar's: the CTA outlives it
    if (ok && rank != 0 && kc > 0) W.wait(done_bar, 0);
  } else if (warp == kQWarp) {
    // ============================================================ Q by TMA
    const uint32_t lead = at_rank(bar0, 0);
    QRing ring;
    bool ok = true;
    Unit u;
    for (uint32_t nu = 0; ok && unit(nu, u); ++nu) {
      seen(nu);
      if (!(u.what & kLoadQ)) continue;
      const uint32_t n = (u.what >> 16) & 15u, slot = u.what >> 20;
      if (ring.other(slot)) {
        for (ring.at = 0; ring.at < ring.count && ok; ++ring.at)
          ok = W.wait(q_empty(ring.at), ring.parity() ^ 1u);
        if (!ok) break;
        ring.begin(slot);
      }
      const CUtensorMap* map = n == 4 ? &q4_map : n == 2 ? &q2_map : &q_map;
      const int32_t row = u.row0 + (int)(rank * n) * 32;
      // as K: lane c has chunk c, whose slot's use before has to be this unit's or older
      const uint32_t q = ring.slot(ring.at, lane & 7), par = ring.parity(q, lane & 7);
      uint32_t done = 0;
      while (done < kChunks) {
        const uint32_t upto = min((uint32_t)kChunks, done + ring.count);
        const bool is = (uint32_t)lane >= done && (uint32_t)lane < upto &&
                        mbar_test(q_empty(q), par ^ 1u);
        uint32_t m = run_of(__ballot_sync(0xffffffffu, is), done, upto);
        if (m == 0) {
          const uint32_t x = __shfl_sync(0xffffffffu, q, done);
          if (!(ok = W.wait(q_empty(x), __shfl_sync(0xffffffffu, par, done) ^ 1u))) break;
          m = 1;
        }
        if ((uint32_t)lane - done < m) {
          if (rank == 0) mbar_expect_tx(q_full(q), 2 * kQBytes * n);
          tma_load_pair(sQ + q * slot * kQBytes, map, lane * 64, row,
                        lead + 8u * (2 * kKSlots + q));
        }
        done += m;
      }
      ring.used(kChunks);
    }
  } else if (warp == kScoutWarp && rank == 0) {
    // ====== scout: looks for the issuer's operands (a wait of the issuer's own would
    // queue behind its MMAs) and lets it in to all chunks that are there, with a word
    // for each that says what to issue.  (One chunk at a time, with two waits and a
    // barrier, is 520 cycles of this warp, where a chunk's MMAs take 512 at most.)
    uint32_t kc = 0, q0 = 0, ns = 0, n_bar = 0;
    QRing ring;
    bool ok = true;
    auto let_in = [&](uint32_t word) {  // lane i's, i < 8; 0 ends them
      if (lane < 8) cmd[(n_bar & 1u) * 8 + lane] = word;
      __syncwarp();
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (n_bar & 1u)) : "memory");
      ++n_bar;
    };
    Unit u;
    for (uint32_t nu = 0; ok && unit(nu, u); ++nu) {
      seen(nu);
      if (u.what & kDead) continue;
      const bool load_q = u.what & kLoadQ, load_k = u.what & kLoadK;
      const uint32_t slot = u.what >> 20;
      if (load_q && ring.other(slot)) ring.begin(slot);
      if (load_q) q0 = ring.at;
      if (load_k) kc += kChunks;
      const uint32_t flags = kGo | (u.what & kEnds ? kFreeK : 0u) |
                             (u.what & kDropQ ? kFreeQ : 0u) | ((u.what >> 16) & 15u) << 8 |
                             slot << 20 | (ns & 1u) << 16;
      if (!(ok = W.wait(s_empty(ns), ((ns >> 1) & 1u) ^ 1u))) break;
      ++ns;
      // lane c looks for chunk c's K, lane 8 + c for its Q
      const uint32_t c = lane & 7u, x = kc - kChunks + c, q = ring.slot(q0, c);
      const uint32_t bar = lane < 8 ? k_full(x % kKSlots) : q_full(q);
      const uint32_t par = lane < 8 ? (x / kKSlots) & 1u : ring.parity(q, c);
      const bool need = c < kChunks && (lane < 8 ? load_k : lane < 16 && load_q);
      const uint32_t word = flags | (c == 0 ? kFirst : 0u) | (c == kChunks - 1 ? kLast : 0u) |
                            (x % kKSlots) << 12 | q << 24;
      uint32_t done = 0;
      while (done < kChunks) {
        // (a slot's next use is not looked for before this one is here)
        const uint32_t upto = load_q ? min((uint32_t)kChunks, done + ring.count) : kChunks;
        const bool is = !need || (c >= done && c < upto && mbar_test(bar, par));
        const uint32_t m = __ballot_sync(0xffffffffu, is);
        uint32_t n = run_of(m & (m >> 8), done, upto);
        if (n == 0) {
          const uint32_t k_bar = __shfl_sync(0xffffffffu, bar, done);
          const uint32_t k_par = __shfl_sync(0xffffffffu, par, done);
          const uint32_t q_bar = __shfl_sync(0xffffffffu, bar, 8 + done);
          const uint32_t q_par = __shfl_sync(0xffffffffu, par, 8 + done);
          if (load_k) ok = W.wait(k_bar, k_par);
          if (load_q && ok) ok = W.wait(q_bar, q_par);
          if (!ok) break;
          n = 1;
        }
        const uint32_t w = __shfl_sync(0xffffffffu, word, done + c);
        let_in(c < n ? w : 0u);
        done += n;
      }
      if (load_q) ring.used(kChunks);
    }
    let_in(0u);
  } else if (warp == kMmaWarp && rank == 0) {
    // ========================================== MMA issuer (leader only)
    const uint32_t dK = (uint32_t)sdesc_sw128(sK, 16, 1024);
    const uint32_t dQ = (uint32_t)sdesc_sw128(sQ, 16, 1024);
    const uint32_t hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    bool any = false;
    for (uint32_t n_bar = 0;; ++n_bar) {
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (n_bar & 1u)) : "memory");
      const uint32_t mine = cmd[(n_bar & 1u) * 8 + (lane & 7)];
      uint32_t word = __shfl_sync(0xffffffffu, mine, 0);
      if (word == 0u) break;
      any = true;
      tc_fence_after();
#pragma unroll 1
      for (int i = 1; word; ++i) {
        if (elect_one()) {
          const uint32_t n = (word >> 8) & 15u, s = (word >> 12) & 15u, u = (word >> 16) & 1u;
          const uint32_t q = word >> 24, slot = (word >> 20) & 15u, d = tmem + u * kBlock;
          const uint32_t idesc = idesc_bf16(256, 0, 0, 0) | (64 * n) >> 3 << 17;
          const uint32_t da = dK + s * (kKBytes >> 4), db = dQ + q * slot * (kQBytes >> 4);
          tc_mma2(d, da, db, hi, idesc, word & kFirst ? 0u : 1u);
#pragma unroll
          for (uint32_t x = 1; x < 4; ++x) tc_mma2(d, da + 2 * x, db + 2 * x, hi, idesc, 1u);
          if (word & kFreeK) tc_commit2(k_empty(s));
          if (word & kFreeQ) tc_commit2(q_empty(q));
          if (word & kLast) tc_commit2(s_full(u));
        }
        __syncwarp();
        if (i == 8) break;
        word = __shfl_sync(0xffffffffu, mine, i);
      }
    }
    if (any) {
      if (elect_one()) tc_commit2(done_bar);
      __syncwarp();
      drain(done_bar, 0, a.timeout_ns);
    }
  } else if (warp < kEpiWarps) {
    // ======================================================== epilogue
    const int quad = warp & 3, g = warp >> 2;  // TMEM lanes, every second set of 32 columns
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint64_t scale2 = pair2(a.scale, a.scale), log2e2 = pair2(kLog2e, kLog2e);
    uint32_t ns = 0, n_sync = 0, n_tiles = 0;
    auto epi_sync = [&]() {  // all epilogue warps of this CTA
      __syncwarp();
      if (lane == 0) mbar_arrive(epi);
      return W.wait(epi, n_sync++ & 1u);
    };
    bool ok = true;
    uint64_t sum[2] = {0ull, 0ull};
    int64_t slot = -1;  // of this thread's key, or -1
    float old = 0.f;    // what it has received before (used last: the load is long)
    Unit u;
    for (uint32_t nu = 0; ok && unit(nu, u); ++nu) {
      const int32_t pos0 = u.pos + (int)rank * 128 + quad * 32, pos = pos0 + lane;
      if (u.what & kBegins) {
        sum[0] = sum[1] = 0ull;
        slot = -1;
        old = 0.f;
        if (g == 0 && pos < u.len) {
          const int32_t row = units[nu % kUnits].page_row[(quad * 32 + lane) >> a.page_log2];
          if (row != no_row) slot = (int64_t)row + (pos & (page - 1));
          if (slot >= 0 && pos < u.base)
            old = __int_as_float(ld_input(reinterpret_cast<const int32_t*>(a.w + slot)));
        }
      }
      if (!(u.what & kDead)) {
        const int32_t n = u.rows, at = u.at;
        const float* neg = neg_s + nu % kUnits * kBlock;
        if (!(ok = W.wait(s_full(ns), (ns >> 1) & 1u))) break;
        tc_fence_after();
        const int32_t first = pos - u.base;  // node, or first token that sees the key
        const bool all_see = pos0 + 31 < u.base || (!a.bits && pos0 + 31 <= u.base);
        const uint32_t tS = tmem + (ns & 1u) * kBlock + lane_base;
        const int sets = (n + 31) >> 5;
#pragma unroll 1
        for (int q = g; q < sets; q += 2) {
          uint32_t s[2][16];
          tmem_ld16(tS + 32 * q, s[0]);
          tmem_ld16(tS + 32 * q + 16, s[1]);
          uint32_t mask = live_s[nu % kUnits * 8 + q];
          if (!all_see) {
            const int32_t r0 = at + 32 * q;  // the set's first row, from the request's
            if (!a.bits) {
              // rows from (pos - base) H on
              const int64_t skip = (int64_t)first * a.H - r0;
              if (skip > 0) mask = skip >= 32 ? 0u : mask & (0xffffffffu << skip);
            } else {
              // lane l reads row r0 + l's bits of the warp's 32 keys; then the 32 x 32
              // bits are turned around
              const int32_t j0 = pos0 - u.base, w0 = j0 >> 5;
              uint32_t lo = 0u, hi = 0u;
              if (32 * q + lane < n &&
                  DSA_IN_BOUNDS((u.row0 - at + r0 + lane) / a.H < a.T, a.status)) {
                const int32_t* bits =
                    a.bits + (int64_t)((u.row0 - at + r0 + lane) / a.H) * a.words;
                if (w0 >= 0 && w0 < a.words) lo = (uint32_t)ld_input(bits + w0);
                if (w0 + 1 >= 0 && w0 + 1 < a.words) hi = (uint32_t)ld_input(bits + w0 + 1);
              }
              uint32_t x = __funnelshift_r(lo, hi, (uint32_t)j0 & 31u);
#pragma unroll
              for (int y = 16; y > 0; y >>= 1) {
                const uint32_t low = 0xffffffffu / ((1u << y) + 1u);
                const uint32_t o = __shfl_xor_sync(0xffffffffu, x, y);
                x = lane & y ? (x & ~low) | ((o & ~low) >> y) : (x & low) | ((o & low) << y);
              }
              if (first >= 0) mask &= x;
            }
          }
          const bool plain = __all_sync(0xffffffffu, mask == 0xffffffffu);
          const ulonglong2* neg2 = reinterpret_cast<const ulonglong2*>(neg + 32 * q);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_wait_ld_dep(s[h]);
            uint64_t y[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const ulonglong2 l = neg2[4 * h + e / 2];
              y[e] = fma2(pair2(__uint_as_float(s[h][2 * e]), __uint_as_float(s[h][2 * e + 1])),
                          scale2, l.x);
              y[e + 1] =
                  fma2(pair2(__uint_as_float(s[h][2 * e + 2]), __uint_as_float(s[h][2 * e + 3])),
                       scale2, l.y);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float p0, p1;
              unpair2(mul2(y[e], log2e2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              if (!plain) {
                if (!(mask >> (16 * h + 2 * e) & 1u)) p0 = 0.f;
                if (!(mask >> (16 * h + 2 * e + 1) & 1u)) p1 = 0.f;
              }
              sum[e & 1] = add2(sum[e & 1], pair2(p0, p1));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_signal(at_rank(s_empty(ns), 0));
        ++ns;
      }
      seen(nu);
      if (!(u.what & kEnds)) continue;
      // ---- this CTA's part of the tile is done
      float lo, hi, v;
      unpair2(add2(sum[0], sum[1]), lo, hi);
      v = lo + hi;
      float* red = red_s + (n_tiles++ & 1u) * 128;
      if (g == 1) red[quad * 32 + lane] = v;
      if (!(ok = epi_sync())) break;
      if (g == 0) v += red[quad * 32 + lane];
      bool mine = g == 0;
      if (!(u.what & kWhole)) {
        // the pairs that have a unit of the tile, and this one's sums for the others
        const int from = (int)(u.pairs & 255u), to = (int)(u.pairs >> 8);
        auto part = [&](int p) {
          return a.parts + (((int64_t)p * 2 + rank) * 2 + (p == from ? 1 : 0)) * 128 + quad * 32 +
                 lane;
        };
        if (g == 0) __stcg(part(pair), v);
        __threadfence();
        if (!(ok = epi_sync())) break;
        if (tid == 0) {
          const int at = from * 2 + (int)rank, shift = 8 * (at & 3);
          const uint32_t old = atomicAdd(a.counters + (at >> 2), 1u << shift);
          const bool last = ((old >> shift) & 255u) == (uint32_t)(to - from);
          if (last) atomicSub(a.counters + (at >> 2), (uint32_t)(to - from + 1) << shift);
          __threadfence();
          misc[2] = last ? 1u : 0u;
        }
        if (!(ok = epi_sync())) break;
        mine = mine && misc[2] != 0u;
        if (mine) {
          v = 0.f;
          for (int p = from; p <= to; ++p) v += __ldcg(part(p));
        }
      }
      if (mine && slot >= 0 && DSA_IN_BOUNDS(slot < a.n_pages << a.page_log2, a.status))
        a.w_out[slot] = a.decay * old + v;
      sum[0] = sum[1] = 0ull;
    }
  }

  // ---- teardown: after a wait that gave up, copies may be in flight to either CTA:
  // they get 2 ms to land before the CTAs go
  if (tid == 0 && *W.w.abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000u) __nanosleep(100000);
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
}

template <int D>
cudaError_t launch_t(const LaunchCtx& c, const CUtensorMap (&qm)[3], const CUtensorMap& km,
                     const Args& a) {
  static std::atomic<uint64_t> prepared{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        key_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  const int pairs = c.num_sms / 2 < kMaxPairs ? c.num_sms / 2 : kMaxPairs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<D>, qm[0], qm[1], qm[2], km, a);
}

}  // namespace

size_t key_weights_ws(const ServeShape&) { return (size_t)kMaxPairs * 2 * 2 * 128 * 4; }

cudaError_t launch_key_weights(const LaunchCtx& c, const ServeShape& s,
                               const CUtensorMap (&q_maps)[3], const CUtensorMap& k_map,
                               const float* lse, const int32_t* table, const int32_t* seq,
                               const int32_t* cu, const uint32_t* tree_bits, int words,
                               const float* w_pages, float decay, float* w_out, uint8_t* ws) {
  Args a;
  a.lse = lse;
  a.table = table;
  a.seq = seq;
  a.cu = cu;
  a.bits = reinterpret_cast<const int32_t*>(tree_bits);
  a.words = words;
  a.w = w_pages;
  a.w_out = w_out;
  a.parts = reinterpret_cast<float*>(ws + kHeader);
  a.counters = reinterpret_cast<uint32_t*>(ws + 64);
  a.decay = decay;
  a.scale = s.scale;
  a.B = s.B;
  a.H = s.H;
  a.max_blocks = s.max_blocks;
  a.page_log2 = s.page_log2;
  a.T = s.T;
  a.n_pages = s.n_pages;
  a.status = c.status;
  a.timeout_ns = c.timeout_ns;
  if (s.D == 128) return launch_t<128>(c, q_maps, k_map, a);
  if (s.D == 256) return launch_t<256>(c, q_maps, k_map, a);
  return launch_t<512>(c, q_maps, k_map, a);
}

}  // namespace dsa
