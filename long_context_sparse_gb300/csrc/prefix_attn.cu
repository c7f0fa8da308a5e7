// prefix_attn.cu -- attention of a batch of requests over one shared prefix
// and each request's own tokens, both in a paged cache, on 5th-generation
// tensor cores by pairs of SMs.
//
// Rows.  K and V are shared by all heads, so the (token, head) rows of every
// request form one tall operand against the prefix: 128 of them are a row
// block.  A unit is one row block against one list of keys: the prefix (row
// blocks over all rows) or a request's own tokens (row blocks over its rows).
//
// Products of a tile of 256 keys, by a cluster of two CTAs (cta_group::2, M =
// 256), with the keys or the value dims on the accumulators' lanes:
//   S^T[key, row]  = K_tile . Q^T     A: 128 keys of each CTA, B: 64 rows of Q each
//   O^T[dv, row]  += V_tile^T . P^T   A: 128 dv of each CTA,   B: 64 rows of P each
// Each CTA so reads half of the keys' K and half of the dims' V, and holds
// half of Q and of P: with 128 rows a pair each byte brought into shared memory
// feeds twice the products that one CTA with 64 rows would make of it, and an
// MMA of 256 x 128 x 16 reads 6 KB of shared memory per SM in its 64 cycles
// where 128 x 64 would read 6 KB in 32.  TMEM: two S^T buffers (2 x 128
// columns) and O^T (128 columns per 256 dv): all 512 at d = 512.
//
// Softmax.  A thread owns one key (a TMEM lane) and 64 rows:
//   P = 2^((s - m) c),  l += P,  O^T += V^T P^T   (O, l, m in fp32, P in bf16:
//   the tensor core's operand type, one rounding of each weight;
//   c = scale log2 e).
// m of a row is a reference near its maximum, shared by the pair: the maximum
// over 32 keys of the first tile, afterwards raised to a tile's maximum, only
// when a weight would pass 2^20.  (Any reference gives the same result as long
// as nothing overflows: the weights are floating point, and fp32 leaves 2^107
// above.)  It is a score as the products leave it, and is taken off before the
// multiplication by c: the difference of two scores is exact where they are
// close, whatever their size, where s c - m c in one fused operation would be
// off by the rounding of m c, which from 2^28 on is more than the slack.
// So the usual tile has no maxima to exchange.  A warp that meets
// a larger score raises a flag; the softmax warps of the pair meet once a tile,
// behind the tensor cores' work on the tile before, and where the flag is up
// they take the exact maxima and rescale l and O^T before they hand P over.
// P of rows 0-63 goes to CTA 0, of rows 64-127 to CTA 1, which is the B
// operand's split: what crosses goes by st.async, whose bytes the receiving
// CTA's barrier counts.  Signals between the CTAs on the usual path carry no
// cluster-scope fence (measured: a release.cluster arrival waits about 1500
// cycles under load, a plain one none): data that crosses is counted by a
// barrier (TMA, st.async), and what a CTA's own threads wrote to its own
// shared memory was handed to the relaying thread inside the CTA.  The relay's
// arrival at the leader so publishes nothing to the leader's threads.  It leans
// on the reader of that P being the tensor core of the SM that holds it, behind
// the writers' proxy fences there; the memory model does not spell that out.
//
// Work.  Units cost their tiles plus kUnitCost; the pairs share the sum
// evenly in unit order, so a long prefix is split over all of them and short
// requests are packed together.  A request's units all cost the tiles of its
// longest row, also those whose rows see fewer: the charge is even and the work
// is not where a prompt's own causal blocks are most of it (tiles of the busiest
// of 76 pairs against the mean: 2048 tokens of 64 heads alone 110 and 61, 4096 of
// 16 heads behind 4096 keys 217 and 165).  What a pair has of a unit is an item.  Every
// (unit, pair) that meet leaves O, m and l (fp32, not normalised) in a slot of
// the workspace, and a second kernel joins each row's slots:
// sum w_i O_i / sum w_i l_i with w_i = 2^((m_i - M) c).
//
// Bounds.  Many rows (64 requests of 64 heads of 512 behind 128k keys, 1107
// GFLOP): 720 us, 1538 TFLOP/s, 80% of the measured bf16 peak and 89% of the rate
// that the power limit sustains.  A tile of 256 keys takes about 4950 cycles, of
// which its products need 4096; the rest is the loads' way into the ring (issue
// to arrival under load about 1500 cycles, four stages of 32 KB on the way) and
// shared memory, which a stage writes once and reads one and a half times in its
// 512 cycles of products.  Two stages more would need the shared memory that Q
// takes; with stages of half the size the call took 17% longer.  Few rows
// behind 1M keys (8 requests of 16 heads): 237 us for 1.08 GB, 4.6 TB/s, the same
// ring with loads from HBM.  d = 256 (ragged drafts): 107 us, 1022 TFLOP/s: half the
// products a tile for the same softmax.  Small calls: 14 us on the GPU, a chain of
// lookups, loads and hand-overs; each further item of a pair about 10 us.
#include <atomic>
#include <type_traits>

#include "attn_common.cuh"
#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;           // rows of a unit
constexpr int kKeys = 256;           // keys of a tile
constexpr int kMaxPairs = 80;        // workspace bound on the pairs of a launch
// A unit's Q load and epilogue, in tiles: 3, and 2 where shares are short, so
// that a tile more or less for a pair weighs more than what it stands for.  us a
// call with 1, 2, 3, by the tiles of a share: 64 rows a request, d = 512, 222 (64
// requests behind 128k keys): 770 707 705; 40: 193 145 145; 32: 160 123 122; 24:
// 128 98.6 99.8; 20: 110 87.5 91.9; 16: 94.0 78.1 79.7; 12: 77.2 65.8 69.6; 8 (16
// requests behind 16k): 49.3 42.4 43.7.  Ragged prompts, 146: 527 454 450.  d = 256,
// 46 (drafts): 126 109 108; 36: 125 93.3 94.5; 28: 101 77.8 78.3; 12: 54.9 45.8
// 47.0.  The two are alike between 28 and 46, where the line is drawn.
constexpr int kUnitCost = 3, kShortCost = 2, kShortShare = 32;
constexpr int kSoftWarps = 8;        // 4 TMEM lane quadrants x 2 groups of rows
constexpr int kGroupRows = 64;
constexpr int kProdWarp = 8, kScoutWarp = 9, kMmaWarp = 10, kPassWarp = 11;
constexpr int kThreads = 32 * 12;
constexpr uint32_t kAtom = 16384;    // 128 rows of 128 bytes
constexpr uint32_t kStageBytes = 2 * kAtom;
constexpr int kSoftRegs = 216, kServiceRegs = 72;  // of the 168 that each thread starts with
static_assert(32 * (8 * kSoftRegs + 4 * kServiceRegs) <= kThreads * 168, "register split");
constexpr float kSlack = 20.0f;      // log2 headroom before a row's reference is raised
// -m of a row none of whose keys has scored above -inf so far: the least finite
// score, which any later one is compared with and raises, and under which -inf
// still has a weight of 0.
constexpr float kUnset = 3.402823466e38f;

// ------------------------------------------------------------------- plan
// The division of work: every CTA of the main kernel derives it from the
// lengths; CTA 0 writes it down for the joining kernel.
struct Plan {
  int64_t total;        // cost of all units; 0: nothing to do
  int64_t chunk;        // cost of a pair's share
  int64_t prefix_cost;  // of the prefix units, which come first
  int32_t prefix_tiles;
  int32_t unit_cost;
};
// ccum[b], ucum[b]: cost and unit number of request b's first unit (b = 0..B)

struct PlanView {
  Plan* p;
  int64_t* ccum;
  int32_t* ucum;
  float2* ml;  // [slots][2][128]: m, and l over each CTA's keys
  float* o;    // [slots][128][D]
};

size_t plan_bytes(int B) { return 256 + round_up((size_t)(B + 1) * 12, 256); }

// Units of the prefix, units of the requests that have rows (at most T), and
// a part more for each pair.
int64_t max_slots(const ServeShape& s) {
  const int64_t n = (s.T * s.H + kRows - 1) / kRows;
  return 2 * n + (s.B < s.T ? s.B : s.T) + kMaxPairs;
}

PlanView plan_view(const ServeShape& s, uint8_t* work) {
  PlanView v;
  v.p = reinterpret_cast<Plan*>(work);
  v.ccum = reinterpret_cast<int64_t*>(work + 256);
  v.ucum = reinterpret_cast<int32_t*>(work + 256 + (size_t)(s.B + 1) * 8);
  uint8_t* at = work + plan_bytes(s.B);
  v.ml = reinterpret_cast<float2*>(at);
  at += (size_t)max_slots(s) * 2 * kRows * sizeof(float2);
  v.o = reinterpret_cast<float*>(at);
  return v;
}

struct Lens {
  const int32_t *seq, *cu;
  int32_t cap;  // tokens that a table row holds
  int H;
};

struct ReqShape {
  int32_t row0;    // first row (token * H)
  int32_t n_rows;  // rows
  int32_t len;     // own tokens
  int32_t tiles;   // of its longest row
  int32_t n_new;   // query tokens
};

template <bool Ahead = false>
__device__ __forceinline__ ReqShape req_shape(const Lens& L, int b) {
  const int32_t c0 = ld_input<Ahead>(L.cu + b), c1 = ld_input<Ahead>(L.cu + b + 1);
  int32_t len = ld_input<Ahead>(L.seq + b);
  if (len < 0 || len > L.cap) len = 0;  // latched by CTA 0
  return {c0 * L.H, (c1 - c0) * L.H, len, (len + kKeys - 1) / kKeys, c1 - c0};
}

// Own tokens that row r (from the request's first) of a request sees.
__device__ __forceinline__ int32_t row_limit(const ReqShape& r, int H, int32_t row) {
  return max(0, r.len - r.n_new + row / H + 1);
}

__device__ __forceinline__ int32_t unit_count(const ReqShape& r) {
  return r.tiles ? (r.n_rows + kRows - 1) / kRows : 0;
}

// x / y for x >= 0, y > 0: by 32 bits where they do (64 take ten times as long)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// Tiles [a, z) of a unit of `tiles` tiles that starts at cost c0, for the
// pair whose share is [s, e).
__device__ __forceinline__ void share_of(int64_t c0, int32_t tiles, int32_t unit_cost,
                                         int64_t s, int64_t e, int32_t& a, int32_t& z) {
  const int64_t lo = s - c0 - unit_cost;
  const int64_t hi = min(e - c0, (int64_t)tiles + unit_cost) - unit_cost;
  a = lo > 0 ? (int32_t)lo : 0;
  z = hi > 0 ? (int32_t)hi : 0;
}

// The tiles of an item are taken in turn from `rot` on, wrapping around, so that
// the pairs, which walk other row blocks of the same prefix, are at the same
// tile at the same time (each tile then comes from HBM once, whatever the
// prefix's length): the tile at cost t of a share is t modulo the shorter of a
// share and a unit, where the item has it.
struct Item {
  int32_t tile0, n;       // its first tile, its tiles; n = 0: no more items
  int32_t rot;            // its first turn
  int32_t len;            // keys of the list
  int32_t lim_min;        // keys of it that every row of the block sees
  int32_t row0, n_rows;   // first row of the block, rows of it that count
  int32_t unit;
  int32_t b;              // request, or -1: the prefix
  int32_t rel0;           // row0 from the request's first row
};

// A pair's share and where it starts.
struct Share {
  int64_t start, end;    // the share, in cost
  int64_t prefix_cost;
  int64_t first_cost;    // cost before request first_b
  int32_t first_b;       // request at start, or the first one
  int32_t first_unit;    // its first unit
  int32_t prefix_tiles;
  int32_t rows_all;      // rows of all requests
  int32_t unit_cost;
};

// The tile of an item's turn j.
__device__ __forceinline__ int32_t tile_at(int32_t tile0, int32_t n, int32_t rot, int32_t j) {
  const int32_t x = j + rot;
  return tile0 + (x < n ? x : x - n);
}

// Walks the units of one pair's share, in order; a whole warp, in step.
struct Walk {
  Share sh;
  int64_t pos;
  int64_t cb;   // cost and units before request b, which is at or before pos
  int32_t ub, b;

  // the next item, or one of no tiles
  __device__ __forceinline__ void next(const Lens& L, int B, int32_t prefix_len, Item& it) {
    const int64_t start = sh.start, end = sh.end;
    const int32_t unit_cost = sh.unit_cost;
    it.n = 0;
    while (it.n <= 0 && pos < end) {
      int64_t c0;
      int32_t tiles, last;
      it.rot = 0;
      if (pos < sh.prefix_cost) {
        tiles = sh.prefix_tiles;
        const int32_t u = (int32_t)quotient(pos, tiles + unit_cost);
        c0 = (int64_t)u * (tiles + unit_cost);
        it.unit = u;
        it.row0 = it.rel0 = u * kRows;
        it.n_rows = min(kRows, sh.rows_all - it.row0);
        it.len = it.lim_min = prefix_len;
        it.b = -1;
        share_of(c0, tiles, unit_cost, start, end, it.tile0, last);
        const int64_t turn = min(end - start, (int64_t)tiles + unit_cost);
        const int64_t ahead = c0 + unit_cost - start;
        const int64_t x = ahead < 0 ? -ahead : ahead, y = x - quotient(x, turn) * turn;
        it.rot = (int32_t)(ahead < 0 && y ? turn - y : y);
        if (it.rot >= last - it.tile0) it.rot = 0;
      } else {
        ReqShape r = req_shape(L, b);
        for (;;) {
          const int32_t units = unit_count(r);
          const int64_t next_cb = cb + (int64_t)units * (r.tiles + unit_cost);
          if (pos < next_cb) break;
          cb = next_cb;
          ub += units;
          // the next request with units; the idle ones are passed 32 at a time
          uint32_t some = 0;
          while (!some && ++b < B) {
            const int x = b + (int)(threadIdx.x & 31);
            some = __ballot_sync(0xffffffffu, x < B && unit_count(req_shape(L, x)) > 0);
            b += some ? __ffs(some) - 1 : 31;
          }
          if (!some) {  // lengths that changed under the kernel
            pos = end;
            return;
          }
          r = req_shape(L, b);
        }
        tiles = r.tiles;
        const int32_t j = (int32_t)quotient(pos - cb, tiles + unit_cost);
        c0 = cb + (int64_t)j * (tiles + unit_cost);
        it.unit = ub + j;
        it.rel0 = j * kRows;
        it.row0 = r.row0 + it.rel0;
        it.n_rows = min(kRows, r.n_rows - it.rel0);
        // keys beyond the block's last row are seen by no row of it
        it.len = min(r.len, row_limit(r, L.H, it.rel0 + it.n_rows - 1));
        it.lim_min = row_limit(r, L.H, it.rel0);
        it.b = b;
        share_of(c0, tiles, unit_cost, start, end, it.tile0, last);
        last = min(last, (it.len + kKeys - 1) / kKeys);
      }
      pos = min(end, c0 + tiles + unit_cost);
      it.n = last - it.tile0;
    }
    if (it.n < 0) it.n = 0;
  }
};

// The share of pair `pair` of `pairs`; all threads of the CTA, `scratch` in
// shared memory.  The requests are summed once for the total and scanned for
// the one at the share's start (B <= kThreads: one step each).  `out`: CTA 0
// writes the plan down and latches what is wrong with the lengths.
__device__ __forceinline__ void divide(const Lens& L, int B, int64_t T, int32_t prefix_len,
                                       int64_t pair, int pairs, const PlanView* out,
                                       uint32_t* status, Share* share, int64_t* scratch) {
  constexpr int kWarps = kThreads / 32;
  int32_t* scratch_u = reinterpret_cast<int32_t*>(scratch + kWarps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t first = ld_input(L.cu), last = ld_input(L.cu + B);
  int bad = first < 0 || last > T;
  int64_t sum = 0;
  for (int b = tid; b < B; b += kThreads) {
    const ReqShape r = req_shape(L, b);
    bad |= r.n_new < 0;
    const int64_t units = unit_count(r);
    sum += units * r.tiles + (units << 40);  // tiles (below 2^39), units
    if (out) {
      const int32_t n = ld_input(L.seq + b);
      if (n < 0 || n > L.cap) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    }
  }
  sum = warp_sum(sum);
  if (lane == 0) scratch[warp] = sum;
  bad = __syncthreads_or(bad);
  const int32_t ptiles = (prefix_len + kKeys - 1) / kKeys;
  const int32_t np = ptiles ? (int32_t)(((int64_t)last * L.H + kRows - 1) / kRows) : 0;
  int64_t total = (int64_t)np * ptiles + ((int64_t)np << 40);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += scratch[w];
  if (bad) total = 0;  // offsets that do not ascend within [0, T]: nothing is computed
  const int64_t tiles = total & (((int64_t)1 << 40) - 1), units = total >> 40;
  const int32_t unit_cost =
      tiles + kUnitCost * units < (int64_t)kShortShare * pairs ? kShortCost : kUnitCost;
  total = tiles + unit_cost * units;
  const int64_t prefix_cost = (int64_t)np * (ptiles + unit_cost);
  const int64_t chunk = total > pairs ? quotient(total + pairs - 1, pairs) : 1;
  const int64_t start = min(total, pair * chunk);
  if (tid == 0) {
    share->start = start;
    share->end = min(total, start + chunk);
    share->prefix_cost = prefix_cost;
    share->prefix_tiles = ptiles;
    share->unit_cost = unit_cost;
    share->rows_all = last * L.H;
    share->first_b = 0;
    share->first_cost = prefix_cost;
    share->first_unit = np;
    if (out) {
      *out->p = Plan{total, chunk, prefix_cost, ptiles, unit_cost};
      if (bad) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    }
  }
  int64_t c = prefix_cost;
  int32_t u = np;
  // (the other CTAs stop at their own start, those with nothing at once)
  for (int b0 = 0; b0 < B && !bad && (out || (c <= start && start < total)); b0 += kThreads) {
    const int b = b0 + tid;
    int64_t mc = 0;
    int32_t mu = 0;
    if (b < B) {
      const ReqShape r = req_shape(L, b);
      mu = unit_count(r);
      mc = (int64_t)mu * (r.tiles + unit_cost);
    }
    int64_t ic = mc;
    int32_t iu = mu;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, ic, s);
      const int32_t y = __shfl_up_sync(0xffffffffu, iu, s);
      if (lane >= s) {
        ic += x;
        iu += y;
      }
    }
    __syncthreads();
    if (lane == 31) {
      scratch[warp] = ic;
      scratch_u[warp] = iu;
    }
    __syncthreads();
    int64_t tc = 0;
    int32_t tu = 0;
#pragma unroll 4
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        ic += tc;
        iu += tu;
      }
      tc += scratch[w];
      tu += scratch_u[w];
    }
    const int64_t c0 = c + ic - mc;
    const int32_t u0 = u + iu - mu;
    if (b < B && c0 <= start && start < c0 + mc) {
      share->first_b = b;
      share->first_cost = c0;
      share->first_unit = u0;
    }
    if (out && b < B) {
      out->ccum[b] = c0;
      out->ucum[b] = u0;
    }
    c += tc;
    u += tu;
  }
}

// --------------------------------------------------------------- warp PTX
// One lane of a converged warp, the same one every time.  The compiler knows
// this branch as one whose operands may stay in uniform registers, which it
// does not of `lane == 0`: eight MMAs and their commit then issue in 517 cycles
// instead of 649, and in 720 instead of 990 beside warps that keep the
// schedulers busy (MMAs and TMA alone; 512 is their rate).
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ uint32_t round16(int x) { return ((uint32_t)x + 15u) & ~15u; }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
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

// 32 columns of this thread's TMEM lane; the values are there after the wait,
// which the compiler sees as writing them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// ------------------------------------------------------------ main kernel
// Shared memory at D = 512: Q 64 KB, P 32 KB, four stages of 32 KB, 2 KB of row
// constants and barriers, 1 KB to align: all of the 227 KB; at 256 and 128 a
// second P.
constexpr int kStages = 4;
constexpr int kBars = 28;

template <int D>
struct PCfg {
  static constexpr int kKStages = D / 128;               // stages of a tile's K
  static constexpr int kBlocks = D > 256 ? D / 256 : 1;  // 256-dv blocks of O^T
  static constexpr int kVStages = 2 * kBlocks;           // 128 keys of a block each
  static constexpr uint32_t kQBytes = 64 * D * 2;        // this CTA's 64 rows
  static constexpr uint32_t kPBytes = kKeys * 128;       // 256 keys x 64 rows
  // P buffers: where two fit, a tile's P is written while the one before is read
  static constexpr uint32_t kPBufs = D == 512 ? 1 : 2;
  static constexpr uint32_t kTail = 2048;
  static constexpr uint32_t kSmem =
      1024 + kQBytes + kPBufs * kPBytes + kStages * kStageBytes + kTail;
  static_assert(kSmem <= 232448, "shared memory");
};

// Reduce 16 columns over the warp's lanes: lanes i and i + 16 end with column i
// (16 shuffles: each step halves the columns that a lane keeps).
template <bool MAX>
__device__ __forceinline__ float column_reduce(float (&x)[16], int lane) {
#pragma unroll
  for (int H = 8; H > 0; H >>= 1) {
    const bool up = (lane & H) != 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float keep = up ? x[i + H] : x[i], give = up ? x[i] : x[i + H];
      const float got = __shfl_xor_sync(0xffffffffu, give, H);
      x[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, x[0], 16);
  return MAX ? fmaxf(x[0], got) : x[0] + got;
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ CUtensorMap v8_map,
                       const __grid_constant__ CUtensorMap v1_map, PlanView view, Lens L,
                       const int32_t* __restrict__ prefix_table, int32_t prefix_len,
                       const int32_t* __restrict__ table, int B, int64_t T,
                       int max_blocks, int page_log2, int32_t n_pages, int64_t n_slots,
                       float scale_log2, uint32_t* status, uint64_t timeout_ns) {
  using C = PCfg<D>;
  constexpr uint32_t IDESC_S = idesc_bf16(256, 128, 0, 0);
  constexpr uint32_t IDESC_O = idesc_bf16(256, 128, 1, 1);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (base - raw);
  const uint32_t sQ = base;
  const uint32_t sP = sQ + C::kQBytes;
  const uint32_t sStage = sP + C::kPBufs * C::kPBytes;
  uint8_t* tail = gb + C::kQBytes + C::kPBufs * C::kPBytes + kStages * kStageBytes;
  float* nm2_s = reinterpret_cast<float*>(tail);          // [item & 1][row] -m
  float* fac_s = nm2_s + 2 * kRows;  // [row] what raising m makes of l and O
  uint8_t* lim_s = reinterpret_cast<uint8_t*>(fac_s + kRows);  // [row] keys past lim_min
  uint64_t* bars = reinterpret_cast<uint64_t*>(lim_s + kRows);
  // abort, tmem, beyond, issuer's tiles
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + kBars);
  Item* posts = reinterpret_cast<Item*>(misc + 4);             // [2]
  static_assert(3 * kRows * 4 + kRows + kBars * 8 + 16 + 2 * sizeof(Item) <= C::kTail, "tail");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  // scratch in the part of P that only this CTA's warps write: used while no
  // product reads P and before this CTA's warps write it again
  float* red = reinterpret_cast<float*>(gb + C::kQBytes + rank * 128 * 128);  // [8][row]
  float* lred = red + 8 * kRows;                                             // [4][row]
  Share* share = reinterpret_cast<Share*>(lred);  // until the first item is posted
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };              // leader: both landed
  auto empty = [&](uint32_t s) { return bar0 + 8u * (kStages + s); };  // stage read
  const uint32_t bx = bar0 + 8u * (2 * kStages);
  const uint32_t q_full = bx;                                     // leader
  const uint32_t q_empty = bx + 8;
  auto s_full = [&](uint32_t b) { return bx + 16 + 8 * b; };
  auto p_in = [&](uint32_t t) { return bx + 32 + 8 * (t & 1u); };     // own P is written
  auto p_full = [&](uint32_t t) { return bx + 48 + 8 * (t & 1u); };   // leader: both CTAs' are
  auto p_done = [&](uint32_t t) { return bx + 64 + 8 * (t & 1u); };   // and have been read
  const uint32_t o_empty = bx + 80;  // leader
  const uint32_t xs = bx + 88;       // the softmax warps of both CTAs
  const uint32_t grp = bx + 96;      // the softmax warps of this CTA
  const uint32_t done_bar = bx + 104;
  auto post_full = [&](uint32_t i) { return bx + 112 + 8 * (i & 1u); };
  auto post_free = [&](uint32_t i) { return bx + 128 + 8 * (i & 1u); };
  const uint32_t refs = bx + 144;    // an item's first references
  static_assert(2 * kStages + 19 <= kBars, "barriers");
  // phase parity of a barrier that serves every other tile, in tile t
  auto turn = [](uint32_t t) { return (t >> 1) & 1u; };
  // tile number + 1 of the last tile with a score beyond its reference
  volatile uint32_t* beyond_s = misc + 2;
  const PairWaiter W{misc, at_rank(smem_u32(misc), peer), status, timeout_ns};

  if (tid == 0) {
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_in(b), kSoftWarps / 2 + 1);
      mbar_init(p_full(b), 2);
      mbar_init(p_done(b), 1);
      mbar_init(post_full(b), 1);
      mbar_init(post_free(b), kSoftWarps + (rank == 0 ? 2 : 1));
    }
    mbar_init(o_empty, 2 * kSoftWarps);
    mbar_init(xs, 2 * kSoftWarps);
    mbar_init(grp, kSoftWarps);
    mbar_init(refs, rank == 0 ? kSoftWarps : 1);
    mbar_init(done_bar, 1);
    misc[0] = misc[2] = 0u;
    fence_mbar_init();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(misc + 1)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // the barriers and TMEM are ready: the CTAs meet while they divide the work
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  // the stream's work before; then the joining kernel may start, which reads the
  // lengths before it waits for this kernel's end
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t pair = blockIdx.x >> 1;
  divide(L, B, T, prefix_len, pair, gridDim.x >> 1, blockIdx.x == 0 ? &view : nullptr, status,
         share, reinterpret_cast<int64_t*>(red));
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  // item ni, as kPassWarp posted it, one ahead of its tiles
  uint32_t ni = 0;
  auto take = [&](Item& i) {
    if (!W.wait(post_full(ni), (ni >> 1) & 1u)) return false;
    i = posts[ni & 1u];
    return i.n > 0;
  };
  auto give_back = [&]() {  // the item's slot
    __syncwarp();
    if (lane == 0) mbar_arrive(post_free(ni));
    ++ni;
  };
  constexpr uint32_t tmem = 0;  // an allocation of all 512 columns starts at column 0
  constexpr uint32_t tO = tmem + 2 * kRows;
  Item it;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kServiceRegs));
    if (warp == kProdWarp) {
      // ==================================================== TMA producer
      // A stage is 128 keys by two 64-wide column blocks: of K this CTA's keys
      // and 128 dims, of V 128 keys of either CTA and this CTA's 128 dv.
      const int32_t n_rows_cache = n_pages << page_log2;  // out of range: zero rows
      const int nb = 128 >> page_log2;                    // page boxes of a column block
      const bool on = lane < 2 * nb;
      const int col = on ? (lane >> (7 - page_log2)) * 64 : 0;     // of this lane's box
      const int key0 = on ? (lane & (nb - 1)) << page_log2 : 0;    // its first key
      const uint32_t dst = sStage + (uint32_t)(col / 64) * kAtom + (uint32_t)key0 * 128;
      const bool arms = rank == 0 && lane == 0;
      const uint32_t lead_q = at_rank(q_full, 0), lead_full = at_rank(full(0), 0);
      uint32_t u = 0, nq = 0;  // stages, items so far
      const int page = 1 << page_log2;
      bool ok = true;
      const int32_t* pages = nullptr;
      int32_t tile = 0, turns = 0;  // this turn's tile, the item's turns so far
      int32_t ids[2] = {0, 0};      // its pages
      int32_t v_row[2] = {0, 0}, v_left = 0;  // the turn's before: V rows, keys from it on
      bool k_on = false, v_on = false;        // is there a K tile, a V tile this turn
      it.n = 0;
      // page of key `half * 128 + key0` of tile j (0 where nothing is read)
      auto page_at = [&](int32_t j, int half) {
        const int32_t pos = j * kKeys + half * 128 + key0;
        return pos < it.len ? ld_input(pages + (pos >> page_log2)) : 0;
      };
      // its first cache row, or out of range past the end
      auto row_of = [&](int32_t j, int half, int32_t p) {
        if (j * kKeys + half * 128 + key0 >= it.len) return n_rows_cache;
        if (p < 0 || p >= n_pages) {
          latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
          return n_rows_cache;
        }
        return p << page_log2;
      };
      // A turn: K of a tile and V of the tile before, across items
      do {
        if (turns == it.n) {
          turns = 0;
          k_on = take(it);
          if (k_on) {
            pages = it.b < 0 ? prefix_table : table + (int64_t)it.b * max_blocks;
            give_back();
            if (!(ok = W.wait(q_empty, (nq & 1u) ^ 1u))) break;
            if (arms) mbar_expect_tx(q_full, 2 * C::kQBytes);
            if (lane < D / 64)
              tma_load_pair(sQ + lane * 8192, &q_map, lane * 64, it.row0 + (int32_t)rank * 64,
                            lead_q);
            ++nq;
            tile = it.tile0 + it.rot;
            ids[0] = page_at(tile, 0);
            ids[1] = page_at(tile, 1);
          }
        }
        int32_t c_row[2] = {0, 0}, c_left = 0;
        if (k_on) {  // K of this turn's tile
          c_row[0] = row_of(tile, 0, ids[0]);
          c_row[1] = row_of(tile, 1, ids[1]);
          c_left = it.len - tile * kKeys;
          ++turns;
          tile = tile_at(it.tile0, it.n, it.rot, turns < it.n ? turns : 0);
          ids[0] = page_at(tile, 0);  // looked at in the next turn
          ids[1] = page_at(tile, 1);
          const int32_t row = rank ? c_row[1] : c_row[0];
#pragma unroll 1
          for (int a = 0; a < C::kKStages; ++a, ++u) {
            const uint32_t s = u % kStages;
            if (!(ok = W.wait(empty(s), ((u / kStages) & 1u) ^ 1u))) break;
            if (arms) mbar_expect_tx(full(s), 2 * kStageBytes);
            if (on)
              tma_load_pair(dst + s * kStageBytes, &k_map, a * 128 + col, row,
                            lead_full + 8u * s);
          }
        }
        if (v_on && ok) {  // V of the turn's before
#pragma unroll 1
          for (int x = 0; x < C::kVStages; ++x, ++u) {
            const uint32_t s = u % kStages;
            const int half = x & 1;
            if (!(ok = W.wait(empty(s), ((u / kStages) & 1u) ^ 1u))) break;
            const int keys = v_left - 128 * half;  // of this stage, that count
            const int32_t rows = half ? v_row[1] : v_row[0];
            const int x0 = (x >> 1) * 256 + (int)rank * 128;
            if (arms) mbar_expect_tx(full(s), 2 * kStageBytes);
            if (keys <= 0 || (keys & (page - 1)) == 0 || keys >= 128) {
              if (on)
                tma_load_pair(dst + s * kStageBytes, &v_map, x0 + col, rows,
                              lead_full + 8u * s);
              continue;
            }
            // The list ends inside a page.  The rows behind may hold NaN, which a
            // zero weight does not cancel, so none of them is loaded: eight rows
            // a lane, those around the end one by one, and zeros (out of range)
            // past it.
            const int end8 = keys & 7 ? keys >> 3 : 16;
            const int r = lane < 16 ? 8 * lane : 8 * end8 + (lane & 7);
            const int32_t from = __shfl_sync(0xffffffffu, rows, (r & 127) >> page_log2) +
                                 (r & (page - 1));
            if (lane < 16 ? lane != end8 : lane < 24 && end8 < 16)
              for (int a = 0; a < 2; ++a)
                tma_load_pair(sStage + s * kStageBytes + a * kAtom + r * 128,
                              lane < 16 ? &v8_map : &v1_map, x0 + a * 64,
                              r < keys ? from : n_rows_cache, lead_full + 8u * s);
          }
        }
        v_row[0] = c_row[0];
        v_row[1] = c_row[1];
        v_left = c_left;
        v_on = k_on;
      } while (ok && k_on);
      // the leader's last arrival here is done_bar's: the CTA outlives it
      if (ok && rank != 0 && u > 0) W.wait(done_bar, 0);
    } else if (warp == kScoutWarp && rank == 0) {
      // ================ scout (leader only): waits for the MMA issuer's operands
      // A wait on an mbarrier queues behind the MMAs that the same thread has
      // issued, and the tensor core idles until it returns: a loop that waits
      // and issues took 610 to 670 cycles a stage of 512 (MMAs and TMA alone),
      // one that is let in at a named barrier 530.  So this warp does the
      // waiting and meets the issuer at one barrier a stage.  When a wait gives
      // up it lets the issuer through what is left (on whatever shared memory
      // holds), so that no thread is left behind at a barrier.
      uint32_t u = 0, nt = 0, nq = 0, no = 0;  // stages, tiles, items by S^T and by O^T
      bool ok = true;
      auto let_in = [&]() {
        if (ok) ok = W.wait(full(u % kStages), (u / kStages) & 1u);
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (u & 1u)) : "memory");
        ++u;
      };
      int left = 0;  // tiles of the item whose S^T is to come
      bool s_on, o_on = false, o_first = false;
      do {
        const bool fresh = left == 0;
        if (fresh) {
          left = ok && take(it) ? it.n : 0;
          if (lane == 0) misc[3] = (uint32_t)left;  // the issuer takes the same turns
          asm volatile("bar.sync 3, 64;" ::: "memory");
          if (left > 0) {
            give_back();
            if (ok) ok = W.wait(q_full, nq & 1u);
            ++nq;
          }
        }
        s_on = left > 0;
        if (s_on) {
          --left;
          for (int c = 0; c < C::kKStages; ++c) let_in();
        }
        if (o_on) {
          if (ok) ok = W.wait(p_full(nt), turn(nt));
          if (o_first) {
            if (ok) ok = W.wait(o_empty, (no & 1u) ^ 1u);
            ++no;
          }
          for (int c = 0; c < C::kVStages; ++c) let_in();
          ++nt;
        }
        o_on = s_on;
        o_first = fresh;
      } while (s_on);
    } else if (warp == kPassWarp) {
      // ===== items to the softmax warps; this CTA's P complete -> the leader
      uint32_t nt = 0;
      bool ok = true;
      Walk walk{*share, share->start, share->first_cost, share->first_unit, share->first_b};
      __syncwarp();
      auto post = [&]() {  // the next item, one ahead of its tiles
        walk.next(L, B, prefix_len, it);
        if (!W.wait(post_free(ni), ((ni >> 1) & 1u) ^ 1u)) return false;
        if (lane == 0) {
          posts[ni & 1u] = it;
          mbar_arrive(post_full(ni));
        }
        __syncwarp();
        ++ni;
        return true;
      };
      ok = post();
      while (ok && it.n > 0) {
        const int32_t n = it.n, n_rows = it.n_rows;
        if (!(ok = post())) break;
        // bytes from the other CTA's keys, if this CTA's group has rows
        const uint32_t bytes =
            n_rows > kGroupRows * (int)rank ? 128 * kGroupRows * 2 : 0;
        for (int32_t j = 0; j < n; ++j, ++nt) {
          if (lane == 0) mbar_expect_tx(p_in(nt), bytes);
          if (!(ok = W.wait(p_in(nt), turn(nt)))) break;
          if (lane == 0) {
            fence_proxy_async();
            mbar_signal(at_rank(p_full(nt), 0));
          }
          __syncwarp();
        }
      }
    } else if (warp == kMmaWarp && rank == 0) {
      // ========================================== MMA issuer (leader only)
      // Descriptors: an address 16 bytes on is 1 more.
      uint32_t u = 0, nt = 0;
      const uint32_t dK = (uint32_t)sdesc_sw128(sStage, 16, 1024);
      const uint32_t dV = (uint32_t)sdesc_sw128(sStage, kAtom, 1024);
      const uint32_t dQ = (uint32_t)sdesc_sw128(sQ, 16, 1024);
      const uint32_t dP = (uint32_t)sdesc_sw128(sP, 16, 1024);
      const uint32_t hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
      // eight MMAs of a stage, let in by the scout: mma(descriptor offset, x)
      auto stage = [&](auto mma) {
        const uint32_t s = u % kStages;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (u & 1u)) : "memory");
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (uint32_t x = 0; x < 8; ++x) mma(s * (kStageBytes >> 4), x);
          tc_commit2(empty(s));
        }
        ++u;
      };
      int left = 0;
      bool s_on, o_on = false, o_first = false;
      do {  // a turn: S^T of a tile and O^T of the tile before, across items
        const bool fresh = left == 0;
        if (fresh) {
          asm volatile("bar.sync 3, 64;" ::: "memory");
          left = (int)*reinterpret_cast<volatile uint32_t*>(misc + 3);
        }
        s_on = left > 0;
        if (s_on) {
          // the softmax has read this S^T buffer's last tile: that tile's PV,
          // which waited for it, is ahead in this order
          const uint32_t b = (nt + (o_on ? 1u : 0u)) & 1u, d = tmem + b * kRows;
#pragma unroll 1
          for (uint32_t c = 0; c < C::kKStages; ++c)
            stage([&](uint32_t at, uint32_t x) {  // 64-dim atom x / 4, 16 dims each
              tc_mma2(d, dK + at + (x >> 2) * (kAtom >> 4) + (x & 3) * 2,
                      dQ + (2 * c + (x >> 2)) * 512 + (x & 3) * 2, hi, IDESC_S,
                      c + x != 0 ? 1u : 0u);
            });
          if (elect_one()) {
            if (left == 1) tc_commit2(q_empty);
            tc_commit2(s_full(b));
          }
          --left;
        }
        if (o_on) {
          const uint32_t db = dP + (nt & (C::kPBufs - 1)) * (C::kPBytes >> 4);
#pragma unroll 1
          for (uint32_t c = 0; c < C::kVStages; ++c)
            stage([&](uint32_t at, uint32_t x) {  // 16 keys each
              tc_mma2(tO + (c >> 1) * kRows, dV + at + x * 128, db + ((c & 1) * 8 + x) * 128,
                      hi, IDESC_O, !o_first || (c & 1) + x != 0 ? 1u : 0u);
            });
          if (elect_one()) tc_commit2(p_done(nt));
          ++nt;
        }
        o_on = s_on;
        o_first = fresh;
      } while (s_on);
      if (u > 0) {
        if (elect_one()) tc_commit2(done_bar);
        __syncwarp();
        drain(done_bar, 0, timeout_ns);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ================================================ softmax, epilogue
    const int quad = warp & 3, g = warp >> 2;  // TMEM lanes, rows 64 g .. 64 g + 63
    const int r0 = kGroupRows * g;
    const int key = (int)rank * 128 + quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t owner = (uint32_t)g;  // the CTA that holds P of these rows
    const uint32_t p_row = (owner == rank ? sP : at_rank(sP, peer)) + (uint32_t)key * 128u;
    const uint32_t p_sw = (uint32_t)(key & 7);
    const uint64_t scale2 = pair2(scale_log2, scale_log2);
    uint32_t nx = 0, nf = 0, ng = 0, nt = 0;
    // all softmax warps of the pair; `publish`: with this warp's writes to both
    // CTAs before it
    auto pair_sync = [&](bool publish) {
      __syncwarp();
      if (lane == 0) {
        if (publish) fence_cluster();
        mbar_signal(at_rank(xs, rank));
        mbar_signal(at_rank(xs, peer));
      }
      return W.wait(xs, nx++ & 1u);
    };
    auto group_sync = [&]() {  // all softmax warps of this CTA
      __syncwarp();
      if (lane == 0) mbar_arrive(grp);
      return W.wait(grp, ng++ & 1u);
    };
    bool ok = true;
    while (ok && W.wait(post_full(ni), (ni >> 1) & 1u)) {
      const volatile Item* post = posts + (ni & 1u);
      const int n = post->n;
      if (n == 0) break;
      const int32_t tile0 = post->tile0, rot = post->rot, lim_min = post->lim_min;
      const bool live = post->n_rows > r0;  // this group has rows that count
      const bool same = post->len == lim_min;  // every row sees as many keys
      // references in turns: the other CTA may still read the last item's when
      // this item's arrive there
      float* nm_s = nm2_s + (ni & 1u) * kRows;
      if (tid < kRows) {  // at most one key more a row
        const int32_t pb = post->b;
        lim_s[tid] = pb < 0 ? 0
                            : (uint8_t)(row_limit(req_shape(L, pb), L.H,
                                                  post->rel0 + min(tid, post->n_rows - 1)) -
                                        lim_min);
        // rows without a reference have no weights
        if (tid >= (int)round16(post->n_rows)) nm_s[tid] = -INFINITY;
      }
      if (!(ok = group_sync())) break;
      uint64_t l[32];  // this thread's row sums, in pairs
#pragma unroll
      for (int h = 0; h < 32; ++h) l[h] = 0ull;
      uint32_t pk[32];  // this thread's P, bf16 pairs

      // The first references, of 16 rows a warp of CTA 0: the maxima over the
      // 32 keys of its lanes in the item's first tile.  Where some row does not
      // see all of that tile, over its first 32 keys, by the first warp of the
      // group: every row that sees a key of the item sees one of those (the
      // requests' own tokens are taken in order).  CTA 1 counts theirs by bytes.
      auto first_refs = [&](int32_t tile, uint32_t b) {
        const int n_rows = post->n_rows;
        if (rank == 0) {
          const bool whole = (tile + 1) * kKeys <= lim_min;  // uniform
          const int32_t pos = tile * kKeys + quad * 32 + lane;
          const int h_end = min(n_rows, r0 + (whole ? 16 * (quad + 1) : quad ? 0 : kGroupRows));
#pragma unroll 1
          for (int h0 = r0 + (whole ? 16 * quad : 0); h0 < h_end; h0 += 16) {
            float x[16];
            uint32_t r[16];
            tmem_ld16(tmem + b * kRows + lane_base + h0, r);
            tmem_wait_ld_dep(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[e]);
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (pos >= lim_min + lim_s[h0 + e]) x[e] = -INFINITY;
            }
            // (scores that are not numbers raise no reference: they reach l)
            const float ref = -fmaxf(column_reduce<true>(x, lane), -kUnset);
            float* to = nm_s + h0 + (lane & 15);
            if (lane < 16) *to = ref;
            else st_async_f32(at_rank(smem_u32(to), 1), ref, at_rank(refs, 1));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(refs);
        } else if (tid == 0) {
          mbar_expect_tx(refs, 4 * round16(n_rows));
        }
        return W.wait(refs, nf++ & 1u);
      };
      // The references of the rows where a tile (S^T in buffer b) passes them by
      // more than the slack become its exact maxima
      auto raise = [&](int32_t tile, uint32_t b) {
        const int32_t pos = tile * kKeys + key;
#pragma unroll 1
        for (int h0 = r0; h0 < r0 + kGroupRows; h0 += 16) {
          float x[16];
          uint32_t r[16];
          if (live) {
            tmem_ld16(tmem + b * kRows + lane_base + h0, r);
            tmem_wait_ld_dep(r);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = live && pos < lim_min + lim_s[h0 + e] ? __uint_as_float(r[e]) : -INFINITY;
          const float t = column_reduce<true>(x, lane);
          const uint32_t at = (uint32_t)(((int)rank * 4 + quad) * kRows + h0 + lane);
          if (lane < 16) {
            st_cluster_u32(at_rank(sP + peer * 128 * 128, peer) + 4 * at, __float_as_uint(t));
            red[at] = t;
          }
        }
        if (!pair_sync(true)) return false;
        if (tid < kRows) {
          float top = red[tid];
#pragma unroll
          for (int w = 1; w < 8; ++w) top = fmaxf(top, red[w * kRows + tid]);
          const float nm = nm_s[tid];
          const bool up = (top + nm) * scale_log2 > kSlack;  // as weights() finds it
          fac_s[tid] = up ? ex2((-nm - top) * scale_log2) : 1.f;
          if (up) nm_s[tid] = -top;
        }
        return group_sync();
      };
      // P of a tile from S^T in buffer b, whether a score is beyond its
      // reference, and l.  The weights of 32 rows among which one is beyond are
      // left out of l, which so stays finite, and are added when the tile is
      // visited again (`revisit`) under references that hold them.  `Plain`: each
      // key is seen by all rows or by none, first visit; without branches, so that
      // the work on one half of the rows overlaps the other's loads.
      uint32_t left = 0;
      auto weights = [&](auto plain, int32_t tile, uint32_t b, bool revisit) {
        constexpr bool Plain = decltype(plain)::value;
        const int32_t pos = tile * kKeys + key;
        const bool masked = !Plain && (tile + 1) * kKeys > lim_min;  // uniform
        const bool seen = !Plain || pos < lim_min;
        uint32_t r[2][32];
        const uint32_t tS = tmem + b * kRows + lane_base + r0;
        const ulonglong2* refs2 = reinterpret_cast<const ulonglong2*>(nm_s + r0);
        tmem_ld32(tS, r[0]);
        bool any = false;
        const uint32_t out_before = left;
        left = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ulonglong2 c[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] = refs2[8 * h + e];
          tmem_wait_ld32(r[h]);
          if (h == 0) tmem_ld32(tS + 32, r[1]);
          float d[32];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            unpair2(mul2(add2(pair2(__uint_as_float(r[h][e]), __uint_as_float(r[h][e + 1])),
                              c[e / 4].x),
                         scale2),
                    d[e], d[e + 1]);
            unpair2(mul2(add2(pair2(__uint_as_float(r[h][e + 2]), __uint_as_float(r[h][e + 3])),
                              c[e / 4].y),
                         scale2),
                    d[e + 2], d[e + 3]);
          }
          if (!Plain && masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (pos >= lim_min + lim_s[r0 + 32 * h + e]) d[e] = -INFINITY;
          }
          float top[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = d[e];
#pragma unroll
          for (int e = 4; e < 32; e += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              top[y] = e + 4 < 32 ? fmaxf(top[y], fmaxf(d[e + y], d[e + 4 + y]))
                                  : fmaxf(top[y], d[e + y]);
          const bool beyond =
              fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kSlack && seen;
          any |= beyond;
          left |= beyond ? 1u << h : 0u;
          const bool add = !beyond && seen && (Plain || !revisit || (out_before >> h & 1u) != 0u);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2(d[e]), p1 = ex2(d[e + 1]);
            pk[16 * h + e / 2] = seen ? pack_bf16(p0, p1) : 0u;
            if (add) l[16 * h + e / 2] = add2(l[16 * h + e / 2], pair2(p0, p1));
          }
        }
        return any;
      };
      // P into the CTA that owns the rows.  What crosses is counted by its bytes
      // and goes 64 bytes of a key at a time: four lanes exchange their 16-byte
      // pieces so that they write one key's (lane by lane, 16 bytes of as many
      // keys, a call of 64 requests behind 128k took 8% longer and one of ragged
      // prompts 12%, the exchange aside).
      auto hand_over = [&]() {
        tc_fence_before();  // S^T has been read
        const uint32_t p_to = p_row + (nt & (C::kPBufs - 1)) * C::kPBytes;
        if (owner == rank) {
          if (live) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                               p_to + (((uint32_t)c ^ p_sw) << 4)),
                           "r"(pk[4 * c]), "r"(pk[4 * c + 1]), "r"(pk[4 * c + 2]),
                           "r"(pk[4 * c + 3])
                           : "memory");
          }
          fence_proxy_async();  // P -> the tensor core's reads
          __syncwarp();
          if (lane == 0) mbar_arrive(p_in(nt));
        } else if (live) {
          const uint32_t counts = at_rank(p_in(nt), peer);
          const uint32_t to = p_to - (uint32_t)(lane & 3) * (128 - 16);
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            uint32_t w[4][4];  // w[x]: piece 4 h + x of the key of lane ^ x
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[x][e] = __shfl_xor_sync(0xffffffffu, pk[4 * (4 * h + x) + e], x);
            // w[x]: of the group's key x, at place 4 h + (lane & 3) of its line
#pragma unroll
            for (int x = 0; x < 4; x += 2)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[x][e], b = w[x + 1][e];
                w[x][e] = lane & 1 ? b : a;
                w[x + 1][e] = lane & 1 ? a : b;
              }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[x][e], b = w[x + 2][e];
                w[x][e] = lane & 2 ? b : a;
                w[x + 2][e] = lane & 2 ? a : b;
              }
            const uint32_t half = (h << 6) ^ ((uint32_t)(lane & 4) << 4);
#pragma unroll
            for (int x = 0; x < 4; ++x) st_async_v4(to + 128 * x + half, w[x], counts);
          }
        }
      };
      // l and O^T times 2^((m_old - m_new) c)
      auto rescale = [&](bool o_too) {
        bool any = false;
#pragma unroll
        for (int h = 0; h < kGroupRows / 2; ++h) {
          const float a = fac_s[r0 + 2 * h], c = fac_s[r0 + 2 * h + 1];
          any |= a != 1.f || c != 1.f;
          l[h] = mul2(l[h], pair2(a, c));
        }
        if (!any || !live || !o_too) return;  // the same in every lane
#pragma unroll 1
        for (int c = 0; c < 4 * C::kBlocks; ++c) {
          uint32_t r[16];
          const int h0 = r0 + 16 * (c & 3);
          const uint32_t ta = tO + (c >> 2) * kRows + lane_base + h0;
          tmem_ld16(ta, r);
          tmem_wait_ld_dep(r);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            r[e] = __float_as_uint(__uint_as_float(r[e]) * fac_s[h0 + e]);
          tmem_st16(ta, r);
        }
        tmem_wait_st();
      };

      for (int j = 0; j < n; ++j, ++nt) {
        const uint32_t b = nt & 1u;
        const int32_t tile = tile_at(tile0, n, rot, j);
        if (!(ok = W.wait(s_full(b), turn(nt)))) break;
        tc_fence_after();
        if (j == 0 && !(ok = first_refs(tile, b))) break;
        for (bool revisit = false;; revisit = true) {
          bool beyond = false;
          if (live)
            beyond = !revisit && (same || (tile + 1) * kKeys <= lim_min)
                         ? weights(std::true_type{}, tile, b, false)
                         : weights(std::false_type{}, tile, b, revisit);
          if (revisit) break;
          beyond = __any_sync(0xffffffffu, beyond);
          if (beyond && lane == 0) {
            st_cluster_u32(at_rank(smem_u32(misc + 2), 0), nt + 1u);
            st_cluster_u32(at_rank(smem_u32(misc + 2), 1), nt + 1u);
          }
          if (!(ok = pair_sync(beyond))) break;
          if (*beyond_s != nt + 1u) break;
          // O^T holds every tile before this one
          if (j > 0 && !(ok = W.wait(p_done(nt - 1u), turn(nt - 1u)))) break;
          tc_fence_after();
          if (!(ok = raise(tile, b))) break;
          rescale(j > 0);
        }
        if (!ok) break;
        // the P buffer's last tile has been read (a group without rows writes none,
        // and nothing waits for it: it could come after the buffer's next tile)
        if (live && nt >= C::kPBufs &&
            !(ok = W.wait(p_done(nt - C::kPBufs), turn(nt - C::kPBufs))))
          break;
        hand_over();
      }
      if (!ok || !(ok = W.wait(p_done(nt - 1u), turn(nt - 1u)))) break;
      tc_fence_after();
      // ---- epilogue: m, l and O of this (unit, pair) to its slot
      const int n_rows = post->n_rows;
      const int64_t slot = (int64_t)post->unit + pair;
#pragma unroll
      for (int h0 = 0; h0 < kGroupRows; h0 += 16) {
        if (r0 + h0 >= n_rows) break;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) unpair2(l[(h0 + e) / 2], x[e], x[e + 1]);
        const float t = column_reduce<false>(x, lane);
        if (lane < 16) lred[quad * kRows + r0 + h0 + lane] = t;
      }
      if (!(ok = group_sync())) break;
      if (DSA_IN_BOUNDS(slot < n_slots, status)) {
        if (tid < n_rows) {
          const float sum = lred[tid] + lred[kRows + tid] + lred[2 * kRows + tid] +
                            lred[3 * kRows + tid];
          view.ml[(slot * 2 + rank) * kRows + tid] = make_float2(-nm_s[tid], sum);
        }
        float* out = view.o + slot * (int64_t)(kRows * D);
#pragma unroll 1
        for (int m = 0; m < C::kBlocks; ++m) {
          const int dv = m * 256 + (int)rank * 128 + quad * 32 + lane;
          if (dv >= D) break;  // D = 128: the second CTA's lanes are padding
#pragma unroll 1
          for (int h0 = r0; h0 < min(r0 + kGroupRows, n_rows); h0 += 16) {
            uint32_t r[16];
            tmem_ld16(tO + m * kRows + lane_base + h0, r);
            tmem_wait_ld_dep(r);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (h0 + e < n_rows) out[(int64_t)(h0 + e) * D + dv] = __uint_as_float(r[e]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_signal(at_rank(o_empty, 0));
      give_back();
    }
  }

  // ---- teardown: every role has left its loop.  After a wait that gave up,
  // copies may be in flight to either CTA: they get 2 ms to land before the
  // CTAs go.
  if (tid == 0 && *W.abort_flag) {
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

// ---------------------------------------------------------------- joining
// Row by row, Lanes threads each: the slots of the row's prefix unit and of its
// own unit, weighted by 2^((m_i - M) c).  A tile at cost c belongs to pair
// c / chunk, so a unit's slots are those of the pairs of its first tile to its
// last.  Each lane takes one slot's m and l; then every partial result is read
// once, kJoin of them in flight.  1024 rows of 512: 9.5 us, latency (lookups, m
// and l, partial results); 25600 rows, 190 MB: 25 us.
constexpr int kJoinBlocks = 8;  // of 128 threads on an SM

template <int D, int Lanes>
__global__ void __launch_bounds__(128, D == 16 * Lanes ? 6 : kJoinBlocks)
    join_kernel(PlanView view, Lens L, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                int B, int64_t n_rows, int64_t n_slots, float scale, uint32_t* status) {
  constexpr int kPer = 128 / Lanes;      // rows of a block
  constexpr int kVec = D / (4 * Lanes);  // float4 of a thread in a row
  constexpr int kJoin = 8 / kVec;        // partial results in flight
  asm volatile("griddepcontrol.launch_dependents;");  // a next call's kernel waits for the end
  const int sub = threadIdx.x / Lanes, th = threadIdx.x % Lanes;
  const int64_t row = blockIdx.x * (int64_t)kPer + sub;
  const int32_t t = (int32_t)row / L.H;  // n_rows <= 2^20
  // the row's request, from the call's inputs: before the main kernel's end (it
  // let this one start when it had waited for them itself)
  // the last b in [lo, lo + n) with cu[b] <= t, a 32nd at a time (a warp has one row)
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int n = row < n_rows ? B : 0; n > 1;) {
    const int step = (n + 31) >> 5, x = lane * step;
    const uint32_t le = __ballot_sync(
        0xffffffffu, x < n && ld_input<true>(L.cu + lo + min(x, n - 1)) <= t);
    const int at = (31 - __clz(le | 1u)) * step;
    lo += at;
    n = min(step, n - at);
  }
  ReqShape r{};
  if (row < n_rows) r = req_shape<true>(L, lo);
  const int32_t rel = (int32_t)row - r.row0, block = rel / kRows;
  const bool mine = rel >= 0 && rel < r.n_rows;  // no rows: none past the last either
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel's results
  if (!mine) return;
  const Plan plan = *view.p;
  const int64_t cost = view.ccum[lo];
  const int32_t first_unit = view.ucum[lo];
  // slots s[x] .. s[x] + n[x] - 1: of the prefix unit, of the request's own
  int32_t s[2] = {0, 0}, n[2] = {0, 0};
  const int32_t at[2] = {(int32_t)(row % kRows), rel % kRows};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int32_t tiles = x ? r.tiles : plan.prefix_tiles;
    // tiles that hold keys which some row of the block sees
    const int32_t used =
        x ? (min(r.len, row_limit(r, L.H, min((block + 1) * kRows, r.n_rows) - 1)) + kKeys - 1) /
                kKeys
          : tiles;
    if (plan.total == 0 || used == 0) continue;
    const int32_t u = x ? block : (int32_t)(row / kRows);
    const int64_t c =
        (x ? cost : 0) + (int64_t)u * (tiles + plan.unit_cost) + plan.unit_cost;
    const int32_t first = (int32_t)quotient(c, plan.chunk);
    n[x] = (int32_t)(quotient(c + used - 1, plan.chunk) - first) + 1;
    s[x] = (x ? first_unit : 0) + u + first;
  }
  const int count = n[0] + n[1];
  const float scale_log2 = scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  float4 acc[kVec], oi[kJoin][kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  // row of the partial results with slot number k of this row's
  auto part = [&](int k) { return (k < n[0] ? s[0] + k : s[1] + (k - n[0])) * (int64_t)kRows; };
  auto in_part = [&](int k) { return k < n[0] ? at[0] : at[1]; };
  auto load = [&](int k0) {
#pragma unroll
    for (int e = 0; e < kJoin; ++e)
      if (k0 + e < count && DSA_IN_BOUNDS(part(k0 + e) < n_slots * kRows, status))
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          oi[e][v] = reinterpret_cast<const float4*>(view.o + (part(k0 + e) + in_part(k0 + e)) *
                                                                  D)[v * Lanes + th];
  };
  for (int i = 0; i < count; i += 32) {
    load(i);  // on the way while the weights are worked out
    float mi = -INFINITY, li = 0.f;
    if (i + lane < count && DSA_IN_BOUNDS(part(i + lane) < n_slots * kRows, status)) {
      const float2* ml = view.ml + 2 * part(i + lane) + in_part(i + lane);
      const float2 a = ml[0], b = ml[kRows];
      li = a.y + b.y;  // 0: no key seen
      if (li != 0.f) mi = a.x;
    }
    float top = fmaxf(m, mi);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float keep = m == -INFINITY ? 0.f : ex2((m - top) * scale_log2);
    const float w = mi == -INFINITY ? 0.f : ex2((mi - top) * scale_log2);
    li *= w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) li += __shfl_xor_sync(0xffffffffu, li, x);
    l = fmaf(l, keep, li);
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      acc[v] = make_float4(acc[v].x * keep, acc[v].y * keep, acc[v].z * keep, acc[v].w * keep);
    m = top;
    for (int j = 0; j < 32 && i + j < count; j += kJoin) {
      if (j > 0) load(i + j);
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, j + e);  // 0 past the last slot
        if (we == 0.f) continue;  // what no key went into may be anything
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          acc[v].x = fmaf(we, oi[e][v].x, acc[v].x);
          acc[v].y = fmaf(we, oi[e][v].y, acc[v].y);
          acc[v].z = fmaf(we, oi[e][v].z, acc[v].z);
          acc[v].w = fmaf(we, oi[e][v].w, acc[v].w);
        }
      }
    }
  }
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / l;
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    reinterpret_cast<uint2*>(o + row * D)[v * Lanes + th] =
        make_uint2(pack_bf16(acc[v].x * inv, acc[v].y * inv),
                   pack_bf16(acc[v].z * inv, acc[v].w * inv));
  if (th == 0) lse[row] = none ? -INFINITY : fmaf(m, scale, log2f(l) * kLn2);
}

template <int D>
cudaError_t launch_t(const LaunchCtx& c, const ServeShape& s, const CUtensorMap& qm,
                     const CUtensorMap& km, const CUtensorMap (&vm)[3],
                     const int32_t* prefix_table, int32_t prefix_len, const int32_t* table,
                     const Lens& L, __nv_bfloat16* o, float* lse, uint8_t* work) {
  using C = PCfg<D>;
  const PlanView view = plan_view(s, work);
  cudaError_t e;
  static std::atomic<uint64_t> prepared{0};  // devices whose kernel has its attribute
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(prefix_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::kSmem);
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  const int pairs = c.num_sms / 2 < kMaxPairs ? c.num_sms / 2 : kMaxPairs;
  const int64_t slots = max_slots(s);
  // Both kernels are launched while what is before them in the stream runs, and
  // wait for its end on the device (one request behind 1021 keys, call after call:
  // 15.0 us, and 2.6 more with the first launched behind it).
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefix_attn_kernel<D>, qm, km, vm[0], vm[1], vm[2], view, L,
                         prefix_table, prefix_len, table, s.B, s.T, s.max_blocks, s.page_log2,
                         (int32_t)s.n_pages, slots, s.scale * kLog2e, c.status, c.timeout_ns);
  if (e != cudaSuccess) return e;
  const int64_t rows = s.T * s.H;
  // D / 4 threads a row while all rows are on the SMs at once (with a warp each a
  // call of 1024 rows of 512 took 3 us longer), else a warp each, which looks a row
  // up once (25600 rows: 24 us less a call)
  const bool wide = rows * (D / 4) <= (int64_t)c.num_sms * kJoinBlocks * 128;
  const int64_t per = wide ? 512 / D : 4;
  cfg.gridDim = dim3((unsigned)((rows + per - 1) / per));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, wide ? join_kernel<D, D / 4> : join_kernel<D, 32>, view, L, o,
                            lse, s.B, rows, slots, s.scale, c.status);
}

}  // namespace

size_t prefix_attn_ws(const ServeShape& s) {
  return plan_bytes(s.B) + (size_t)max_slots(s) * kRows * (2 * sizeof(float2) + (size_t)s.D * 4);
}

cudaError_t launch_prefix_attn(const LaunchCtx& c, const ServeShape& s,
                               const CUtensorMap& q_map, const CUtensorMap& k_map,
                               const CUtensorMap (&v_maps)[3], const int32_t* prefix_table,
                               int64_t prefix_len, const int32_t* table,
                               const int32_t* seq, const int32_t* cu, __nv_bfloat16* o,
                               float* lse, uint8_t* work) {
  const Lens L{seq, cu, s.max_blocks << s.page_log2, s.H};
  auto run = [&](auto launch) {
    return launch(c, s, q_map, k_map, v_maps, prefix_table, (int32_t)prefix_len, table, L, o,
                  lse, work);
  };
  if (s.D == 128) return run(launch_t<128>);
  if (s.D == 256) return run(launch_t<256>);
  return run(launch_t<512>);
}

}  // namespace dsa
