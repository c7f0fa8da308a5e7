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
// Softmax.  A thread owns one key (a TMEM lane) and 64 rows; the running
// maximum m of a row is shared by the pair and only raised when a tile beats
// it by more than 2^8, so that the usual tile needs one exchange of flags
// between the CTAs and no reduction:
//   P = 2^(s - m),  l += P,  O^T += V^T P^T      (O, l, m in fp32, P in bf16:
//   the tensor core's operand type, one rounding of 2^-9 for each weight).
// P of rows 0-63 goes to CTA 0, of rows 64-127 to CTA 1, which is the B
// operand's split: what crosses goes by st.async, whose bytes the receiving
// CTA's barrier counts.  Signals between the CTAs on the usual path carry no
// cluster-scope fence (measured: a release.cluster arrival waits about 1500
// cycles under load, a plain one none): data that crosses is counted by a
// barrier (TMA, st.async), and what a CTA's own threads wrote to its own
// shared memory was handed to the relaying thread inside the CTA.
//
// Work.  Units cost their tiles plus kUnitCost; the pairs share the sum
// evenly in unit order, so a long prefix is split over all of them and short
// requests are packed together.  Every (unit, pair) that meet leaves O, m and
// l (fp32, not normalised) in a slot of the workspace, and a second kernel
// joins each row's slots: sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
#include "attn_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kRows = 128;           // rows of a unit
constexpr int kKeys = 256;           // keys of a tile
constexpr int kMaxPairs = 80;        // workspace bound on the pairs of a launch
constexpr int kUnitCost = 2;         // a unit's Q load and epilogue, in tiles
constexpr int kSoftWarps = 16;       // 4 TMEM lane quadrants x 4 groups of rows
constexpr int kGroupRows = 32;
constexpr int kProdWarp = 16, kFixWarp = 17, kMmaWarp = 18, kPassWarp = 19;
constexpr int kThreads = 32 * 20;
constexpr uint32_t kStageBytes = 16384;
constexpr float kSlack = 8.0f;       // log2 headroom before a maximum is raised

// ------------------------------------------------------------------- plan
// The division of work, written by plan_kernel, read by the other two.
struct Plan {
  int64_t total;        // cost of all units; 0: nothing to do
  int64_t chunk;        // cost of a pair's share
  int64_t prefix_cost;  // of the prefix units, which come first
  int32_t n_prefix;     // prefix units
  int32_t prefix_tiles;
};
// ccum[b], ucum[b]: cost and unit number of request b's first unit (b = 0..B)

struct PlanView {
  Plan* p;
  int64_t* ccum;
  int32_t* ucum;
  float2* ml;  // [slots][2][128]: m, and l of each CTA's keys
  float* o;    // [slots][128][D]
};

size_t plan_bytes(int B) { return 256 + round_up((size_t)(B + 1) * 12, 256); }

int64_t max_slots(const ServeShape& s) {
  const int64_t n = (s.T * s.H + kRows - 1) / kRows;
  return 2 * n + s.B + kMaxPairs;
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

__device__ __forceinline__ ReqShape req_shape(const Lens& L, int b) {
  const int32_t c0 = __ldg(L.cu + b), c1 = __ldg(L.cu + b + 1);
  int32_t len = __ldg(L.seq + b);
  if (len < 0 || len > L.cap) len = 0;  // latched by the plan
  return {c0 * L.H, (c1 - c0) * L.H, len, (len + kKeys - 1) / kKeys, c1 - c0};
}

// Own tokens that row r (from the request's first) of a request sees.
__device__ __forceinline__ int32_t row_limit(const ReqShape& r, int H, int32_t row) {
  return max(0, r.len - r.n_new + row / H + 1);
}

__global__ void __launch_bounds__(1024) plan_kernel(Lens L, int B, int64_t T,
                                                    int32_t prefix_len, int pairs,
                                                    Plan* plan, int64_t* ccum,
                                                    int32_t* ucum, uint32_t* status) {
  __shared__ int64_t wc[32];
  __shared__ int32_t wu[32];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int32_t first = __ldg(L.cu), last = __ldg(L.cu + B);
  if (tid == 0 && (first < 0 || last > T)) bad = 1;
  for (int b = tid; b < B; b += 1024)
    if (__ldg(L.cu + b) > __ldg(L.cu + b + 1)) bad = 1;
  __syncthreads();
  if (bad) {  // offsets that do not ascend within [0, T]: nothing is computed
    if (tid == 0) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      plan->total = 0;
      plan->chunk = 1;
    }
    return;
  }
  const int32_t ptiles = (prefix_len + kKeys - 1) / kKeys;
  const int32_t np = ptiles ? (int32_t)(((int64_t)last * L.H + kRows - 1) / kRows) : 0;
  int64_t c = (int64_t)np * (ptiles + kUnitCost);
  int32_t u = np;
  if (tid == 0) {
    plan->prefix_cost = c;
    plan->n_prefix = np;
    plan->prefix_tiles = ptiles;
  }
  for (int b0 = 0; b0 < B; b0 += 1024) {
    const int b = b0 + tid;
    int64_t mc = 0;
    int32_t mu = 0;
    if (b < B) {
      const int32_t n = __ldg(L.seq + b);
      if (n < 0 || n > L.cap) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      const ReqShape r = req_shape(L, b);
      if (r.tiles) mu = (r.n_rows + kRows - 1) / kRows;
      mc = (int64_t)mu * (r.tiles + kUnitCost);
    }
    int64_t ic = mc;
    int32_t iu = mu;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, ic, s);
      const int32_t d = __shfl_up_sync(0xffffffffu, iu, s);
      if (lane >= s) {
        ic += a;
        iu += d;
      }
    }
    __syncthreads();
    if (lane == 31) {
      wc[warp] = ic;
      wu[warp] = iu;
    }
    __syncthreads();
    int64_t tc = 0;
    int32_t tu = 0;
    for (int w = 0; w < 32; ++w) {
      if (w == warp) {
        ic += tc;
        iu += tu;
      }
      tc += wc[w];
      tu += wu[w];
    }
    if (b < B) {
      ccum[b] = c + ic - mc;
      ucum[b] = u + iu - mu;
    }
    c += tc;
    u += tu;
  }
  if (tid == 0) {
    ccum[B] = c;
    ucum[B] = u;
    plan->total = c;
    plan->chunk = c > pairs ? (c + pairs - 1) / pairs : 1;
  }
}

// Tiles [a, z) of a unit of `tiles` tiles that starts at cost c0, for the
// pair whose share is [s, e).
__device__ __forceinline__ void share_of(int64_t c0, int32_t tiles, int64_t s, int64_t e,
                                         int32_t& a, int32_t& z) {
  const int64_t lo = s - c0 - kUnitCost;
  const int64_t hi = min(e - c0, (int64_t)tiles + kUnitCost) - kUnitCost;
  a = lo > 0 ? (int32_t)lo : 0;
  z = hi > 0 ? (int32_t)hi : 0;
}

struct Item {
  int32_t unit;
  int32_t tile0, tile1;   // tiles [tile0, tile1) of the unit
  int32_t row0, n_rows;   // first row of the block, rows of it that count
  int32_t len;            // keys of the list
  const int32_t* pages;   // its page list
  int32_t b;              // request, or -1: the prefix
  int32_t rel0;           // row0 from the request's first row
};

// Walks the units of one pair's share, in order.
struct Walk {
  const Plan* plan;
  const int64_t* ccum;
  const int32_t* ucum;
  Lens L;
  const int32_t* prefix_table;
  const int32_t* table;
  int32_t prefix_len, max_blocks, rows_all;
  int64_t pos, start, end;
  int b;  // request at or before pos, once pos is past the prefix units

  __device__ __forceinline__ bool next(Item& it) {
    while (pos < end) {
      int64_t c0;
      int32_t tiles;
      if (pos < plan->prefix_cost) {
        tiles = plan->prefix_tiles;
        const int32_t u = (int32_t)(pos / (tiles + kUnitCost));
        c0 = (int64_t)u * (tiles + kUnitCost);
        it.unit = u;
        it.row0 = it.rel0 = u * kRows;
        it.n_rows = min(kRows, rows_all - it.row0);
        it.len = prefix_len;
        it.pages = prefix_table;
        it.b = -1;
        share_of(c0, tiles, start, end, it.tile0, it.tile1);
      } else {
        while (__ldg(ccum + b + 1) <= pos) ++b;
        const ReqShape r = req_shape(L, b);
        const int64_t cb = __ldg(ccum + b);
        tiles = r.tiles;
        const int32_t j = (int32_t)((pos - cb) / (tiles + kUnitCost));
        c0 = cb + (int64_t)j * (tiles + kUnitCost);
        it.unit = __ldg(ucum + b) + j;
        it.rel0 = j * kRows;
        it.row0 = r.row0 + it.rel0;
        it.n_rows = min(kRows, r.n_rows - it.rel0);
        // keys beyond the block's last row are seen by no row of it
        it.len = min(r.len, row_limit(r, L.H, it.rel0 + it.n_rows - 1));
        it.pages = table + (int64_t)b * max_blocks;
        it.b = b;
        share_of(c0, tiles, start, end, it.tile0, it.tile1);
        it.tile1 = min(it.tile1, (it.len + kKeys - 1) / kKeys);
      }
      pos = min(end, c0 + tiles + kUnitCost);
      if (it.tile0 < it.tile1) return true;
    }
    return false;
  }
};

// ---------------------------------------------------- pair (cluster) PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// Arrivals at a barrier of either CTA: with a cluster-scope release of this
// thread's writes, and without.
__device__ __forceinline__ void mbar_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void mbar_signal(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity, uint32_t hint) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(hint)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// 16 bytes into either CTA's shared memory; its barrier `bar` counts them.
__device__ __forceinline__ void st_async_v4(uint32_t addr, const uint32_t (&v)[4],
                                            uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];"
      ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
      : "memory");
}
// TMA load into this CTA, its bytes counted by a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                              int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs when the MMAs so far are done.
__device__ __forceinline__ void tc_commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bounded waits of the pair: as Waiter, with cluster scope; a failure stops
// both CTAs.  wait() is for whole warps and gives every lane the same answer,
// so that no lane is left behind at a warp's barrier; wait1() is one thread's.
struct PairWaiter {
  volatile uint32_t* abort_flag;
  uint32_t peer_flag;  // cluster address of the other CTA's flag
  uint32_t* status;
  uint64_t timeout_ns;
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait1(bar, parity));
  }
  __device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity) const {
    if (mbar_try_cluster(bar, parity, 0u)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      if (mbar_try_cluster(bar, parity, 20000u)) return true;
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > timeout_ns) {
        latch_error(status, DSA_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1u;
        st_cluster_u32(peer_flag, 1u);
        return false;
      }
    }
  }
};

// Position in the ring of N stages: the stage and its phase's parity.
template <int N>
struct Ring {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// ------------------------------------------------------------ main kernel
template <int D>
struct PCfg {
  static constexpr int kAtoms = D / 64;               // K stages of a tile
  static constexpr int kBlocks = D > 256 ? D / 256 : 1;  // 256-dv blocks of O^T
  static constexpr uint32_t kQBytes = 64 * D * 2;     // this CTA's 64 rows
  static constexpr uint32_t kPBytes = kKeys * 128;    // 256 keys x 64 rows
  static constexpr int kStages = D == 512 ? 7 : 9;
  static constexpr uint32_t kTail = 16 * 1024;
  // stages between the second-next ragged V stages (see the producer)
  static_assert(2 * (kAtoms + 4 * kBlocks) >= kStages, "ragged stages in flight");
  static constexpr uint32_t kSmem = 1024 + kQBytes + kPBytes + kStages * kStageBytes + kTail;
  static_assert(kSmem <= 232448, "shared memory");
};

// One butterfly step of column_reduce: lanes keep half of the 2 * H columns.
template <int H, bool MAX>
__device__ __forceinline__ void column_step(float (&x)[32], int lane) {
  const bool up = (lane & H) != 0;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float keep = up ? x[i + H] : x[i], give = up ? x[i] : x[i + H];
    const float got = __shfl_xor_sync(0xffffffffu, give, H);
    x[i] = MAX ? fmaxf(keep, got) : keep + got;
  }
}
// Reduce 32 columns over the warp's lanes: lane i ends with column i in x[0]
// (31 shuffles: each step halves the columns that a lane keeps).
template <bool MAX>
__device__ __forceinline__ void column_reduce(float (&x)[32], int lane) {
  column_step<16, MAX>(x, lane);
  column_step<8, MAX>(x, lane);
  column_step<4, MAX>(x, lane);
  column_step<2, MAX>(x, lane);
  column_step<1, MAX>(x, lane);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, PlanView view, Lens L,
                       const int32_t* __restrict__ prefix_table, int32_t prefix_len,
                       const int32_t* __restrict__ table, int B, int max_blocks,
                       int page_log2, int32_t n_pages, int64_t n_slots, float scale_log2,
                       uint32_t* status, uint64_t timeout_ns) {
  using C = PCfg<D>;
  constexpr int kStages = C::kStages;
  constexpr uint32_t IDESC_S = idesc_bf16(256, 128, 0, 0);
  constexpr uint32_t IDESC_O = idesc_bf16(256, 128, 1, 1);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (base - raw);
  const uint32_t sQ = base;
  const uint32_t sP = sQ + C::kQBytes;
  const uint32_t sStage = sP + C::kPBytes;
  uint8_t* tail = gb + C::kQBytes + C::kPBytes + kStages * kStageBytes;
  float* red = carve<float>(tail, 8 * kRows);     // [rank * 4 + quadrant][row] maxima
  float* lred = carve<float>(tail, 4 * kRows);    // [quadrant][row] sums
  // per row: -m (0 while m = -inf), and -(m + slack), above which the maximum
  // is raised (inf while m = -inf)
  float* nm_s = carve<float>(tail, kRows);
  float* nt_s = carve<float>(tail, kRows);
  float* alpha_s = carve<float>(tail, kRows);
  int32_t* lim_s = carve<int32_t>(tail, kRows);   // keys that a row sees
  uint64_t* bars = carve<uint64_t>(tail, 2 * kStages + 20);
  uint32_t* misc = carve<uint32_t>(tail, 8);      // abort, tmem, flags[2], start request
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };               // leader: both landed
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };  // stage read
  const uint32_t bx = bar0 + 8u * (2 * kStages);
  const uint32_t q_full = bx;                                     // leader
  const uint32_t q_empty = bx + 8;
  auto s_full = [&](uint32_t b) { return bx + 16 + 8 * b; };
  auto s_free = [&](uint32_t b) { return bx + 32 + 8 * b; };      // leader
  const uint32_t p_in = bx + 48;     // this CTA's P is written
  const uint32_t p_full = bx + 56;   // leader: both CTAs' P are
  const uint32_t p_done = bx + 64;
  const uint32_t o_empty = bx + 72;  // leader
  const uint32_t xs = bx + 80;       // the softmax warps of both CTAs
  const uint32_t grp = bx + 88;      // the softmax warps of this CTA
  const uint32_t done_bar = bx + 96;
  auto rag = [&](uint32_t r) { return bx + 104 + 8 * (r & 1u); };  // own ragged V stage
  auto fixed = [&](uint32_t r) { return bx + 120 + 8 * (r & 1u); };  // leader: the other's is
  volatile uint32_t* flags = misc + 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const PairWaiter W{misc, at_rank(smem_u32(misc), peer), status, timeout_ns};

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_free(b), 2 * kSoftWarps);
      mbar_init(rag(b), 1);
      mbar_init(fixed(b), 1);
    }
    mbar_init(p_in, kSoftWarps / 2 + 1);
    mbar_init(p_full, 2);
    mbar_init(p_done, 1);
    mbar_init(o_empty, 2 * kSoftWarps);
    mbar_init(xs, 2 * kSoftWarps);
    mbar_init(grp, kSoftWarps);
    mbar_init(done_bar, 1);
    misc[0] = 0u;
    misc[2] = misc[3] = 0u;
    misc[4] = 0u;
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
  // the share of this pair and the request that it starts in
  const Plan* plan = view.p;
  Walk walk;
  walk.plan = plan;
  walk.ccum = view.ccum;
  walk.ucum = view.ucum;
  walk.L = L;
  walk.prefix_table = prefix_table;
  walk.table = table;
  walk.prefix_len = prefix_len;
  walk.max_blocks = max_blocks;
  walk.rows_all = __ldg(L.cu + B) * L.H;
  const int64_t pair = blockIdx.x >> 1;
  walk.start = walk.pos = min(plan->total, pair * plan->chunk);
  walk.end = min(plan->total, walk.start + plan->chunk);
  __syncthreads();
  if (walk.start < walk.end && walk.start >= plan->prefix_cost)
    for (int b = tid; b < B; b += kThreads)
      if (__ldg(view.ccum + b) <= walk.start && walk.start < __ldg(view.ccum + b + 1))
        misc[4] = (uint32_t)b;
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  walk.b = (int)misc[4];
  const uint32_t tmem = misc[1];
  const uint32_t tO = tmem + 2 * kRows;
  Item it;

  if (warp == kProdWarp) {
    // ====================================================== TMA producer
    const int page = 1 << page_log2, box = min(page, 64);
    const int32_t n_rows_cache = n_pages << page_log2;  // out of range: zero rows
    const int kb = 128 / box, vb = 64 / box;            // boxes of a K stage, a V atom
    Ring<kStages> ring;
    uint32_t nq = 0, nr = 0;
    bool ok = true;
    const uint32_t lead_q = at_rank(q_full, 0), lead_full = at_rank(full(0), 0);
    // lane's part: box i of a K stage, box i % vb of atom i / vb of a V stage
    const bool k_on = lane < kb, v_on = lane < 2 * vb;
    const int k_key = (int)rank * 128 + (k_on ? lane : 0) * box;
    const int v_atom = v_on ? lane / vb : 0, v_key = v_on ? (lane % vb) * box : 0;
    const uint32_t k_dst = sStage + (uint32_t)lane * box * 128;
    const uint32_t v_dst = sStage + v_atom * 8192 + v_key * 128;
    const int v_col = (int)rank * 128 + v_atom * 64;
    const bool arms = rank == 0 && lane == 0;
    while (ok && walk.next(it)) {
      if (!(ok = W.wait(q_empty, (nq & 1u) ^ 1u))) break;
      if (arms) mbar_expect_tx(q_full, 2 * C::kQBytes);
      if (lane < C::kAtoms)
        tma_load_pair(sQ + lane * 8192, &q_map, lane * 64, it.row0 + (int32_t)rank * 64, lead_q);
      ++nq;
      // first cache row of the page that holds key x of tile j, in lane x / page
      auto page_rows = [&](int32_t j) {
        const int32_t pos = j * kKeys + (lane << page_log2);
        if ((lane << page_log2) >= kKeys || j >= it.tile1 || pos >= it.len) return n_rows_cache;
        const int32_t p = __ldg(it.pages + (pos >> page_log2));
        if (p < 0 || p >= n_pages) {
          latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
          return n_rows_cache;
        }
        return p << page_log2;
      };
      auto key_row = [&](int32_t j, int32_t rows, int key) {
        const int32_t r = __shfl_sync(0xffffffffu, rows, key >> page_log2);
        return r == n_rows_cache || j * kKeys + key >= it.len ? n_rows_cache
                                                              : r + (key & (page - 1));
      };
      int32_t rows_k = page_rows(it.tile0);
      int32_t v_row[4] = {};  // of this lane's box in the four 64-key groups of V
      for (int32_t j = it.tile0; j <= it.tile1 && ok; ++j) {
        const int32_t rows_n = page_rows(j + 1);
        if (j < it.tile1) {  // K of tile j: this CTA's 128 keys, 64 dims a stage
          const int32_t row = key_row(j, rows_k, k_key);
#pragma unroll 1
          for (int a = 0; a < C::kAtoms; ++a) {
            if (!(ok = W.wait(empty(ring.s), ring.ph ^ 1u))) break;
            if (arms) mbar_expect_tx(full(ring.s), 2 * kStageBytes);
            if (k_on)
              tma_load_pair(k_dst + ring.s * kStageBytes, &k_map, a * 64, row,
                            lead_full + 8u * ring.s);
            ring.step();
          }
        }
        if (j > it.tile0 && ok) {  // V of tile j-1: 64 keys, this CTA's 128 dv a stage
          const int32_t left0 = it.len - (j - 1) * kKeys;
#pragma unroll 1
          for (int m = 0; m < C::kBlocks && ok; ++m)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (!(ok = W.wait(empty(ring.s), ring.ph ^ 1u))) break;
              const bool ragged = left0 > 64 * g && left0 < 64 * g + 64;
              uint32_t bar = lead_full + 8u * ring.s;
              if (ragged) {  // lands at this CTA's barrier: kFixWarp passes it on
                if (lane == 0) mbar_expect_tx(rag(nr), kStageBytes);
                __syncwarp();
                bar = at_rank(rag(nr), rank);
                ++nr;
              } else if (arms) {
                mbar_expect_tx(full(ring.s), 2 * kStageBytes);
              }
              if (v_on)
                tma_load_pair(v_dst + ring.s * kStageBytes, &v_map, m * 256 + v_col, v_row[g],
                              bar);
              ring.step();
            }
        }
        if (j < it.tile1)
#pragma unroll
          for (int g = 0; g < 4; ++g) v_row[g] = key_row(j, rows_k, g * 64 + v_key);
        rows_k = rows_n;
      }
    }
  } else if (warp == kFixWarp) {
    // ============================================= ragged stages of V
    // Rows of V past the list's end may hold NaN, which a zero weight does not
    // cancel: the stage that holds the end is cleared behind it in both CTAs,
    // and then handed to the leader's barrier.  (Stages wholly past the end
    // are zero by TMA's out-of-range fill.)
    uint32_t u = 0, nr = 0;  // stages before this item, ragged stages so far
    bool ok = true;
    while (ok && walk.next(it)) {
      const int32_t last = it.tile1 - 1;            // only the last tile can hold the end
      const int32_t end = it.len - last * kKeys;    // keys of it that count
      const int n = it.tile1 - it.tile0;
      if (end < kKeys && (end & 63) != 0) {
        // its V stages are the item's last 4 * kBlocks; the end is in group end / 64
        for (int m = 0; m < C::kBlocks && ok; ++m, ++nr) {
          const uint32_t at = u + (uint32_t)n * (C::kAtoms + 4 * C::kBlocks) -
                              4 * (C::kBlocks - m) + (uint32_t)(end >> 6);
          const uint32_t s = at % kStages;
          if (!(ok = W.wait(rag(nr), (nr >> 1) & 1u))) break;
          for (int x = (end & 63) * 8 + lane; x < 64 * 8; x += 32)
#pragma unroll
            for (int a = 0; a < 2; ++a)
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                               sStage + s * kStageBytes + a * 8192 + x * 16),
                           "r"(0u)
                           : "memory");
          fence_proxy_async();
          __syncwarp();
          if (rank != 0) {
            if (lane == 0) mbar_release_cluster(at_rank(fixed(nr), 0));
          } else {
            if (!(ok = W.wait(fixed(nr), (nr >> 1) & 1u))) break;
            if (lane == 0) mbar_arrive(full(s));
          }
        }
      }
      u += (uint32_t)n * (C::kAtoms + 4 * C::kBlocks);
    }
  } else if (warp == kPassWarp) {
    // ================= this CTA's P complete -> the leader's barrier
    uint32_t nt = 0;
    bool ok = true;
    const uint32_t lead_p = at_rank(p_full, 0);
    while (ok && walk.next(it)) {
      // bytes from the other CTA's keys, for this CTA's groups with rows
      const int mine = (it.n_rows - 64 * (int)rank + kGroupRows - 1) / kGroupRows;
      const uint32_t bytes = (uint32_t)max(0, min(2, mine)) * (128 * kGroupRows * 2);
      for (int32_t j = it.tile0; j < it.tile1; ++j, ++nt) {
        if (lane == 0) mbar_expect_tx(p_in, bytes);
        if (!(ok = W.wait(p_in, nt & 1u))) break;
        if (lane == 0) {
          fence_proxy_async();
          mbar_signal(lead_p);
        }
        __syncwarp();
      }
    }
  } else if (warp == kMmaWarp) {
    // ============================================ MMA issuer (leader only)
    if (rank == 0 && lane == 0) {
      Ring<kStages> ring;
      uint32_t nt = 0, nq = 0;
      bool issued = false, ok = true;
      // descriptors of stage 0, Q and P; an address 16 bytes on is 1 more
      const uint64_t dK = sdesc_sw128(sStage, 16, 1024), dV = sdesc_sw128(sStage, 8192, 1024);
      const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dP = sdesc_sw128(sP, 16, 1024);
      constexpr uint32_t kStep = kStageBytes >> 4;
      while (ok && walk.next(it)) {
        if (!(ok = W.wait1(q_full, nq & 1u))) break;
        const int n = it.tile1 - it.tile0;
        for (int j = 0; j <= n && ok; ++j) {
          if (j < n) {
            const uint32_t t = nt + (uint32_t)j, b = t & 1u;
            if (!(ok = W.wait1(s_free(b), ((t >> 1) & 1u) ^ 1u))) break;
            issued = true;
#pragma unroll 2
            for (int a = 0; a < C::kAtoms; ++a) {
              const uint64_t da = dK + ring.s * kStep, db = dQ + (uint32_t)a * 512u;
              if (!(ok = W.wait1(full(ring.s), ring.ph))) break;
              tc_fence_after();
#pragma unroll
              for (uint32_t kin = 0; kin < 4; ++kin)
                tc_mma2(tmem + b * kRows, da + 2 * kin, db + 2 * kin, IDESC_S,
                        (a | kin) != 0 ? 1u : 0u);
              tc_commit2(empty(ring.s));
              ring.step();
            }
            if (!ok) break;
            if (j == n - 1) tc_commit2(q_empty);
            tc_commit2(s_full(b));
          }
          if (j >= 1) {
            const uint32_t t = nt + (uint32_t)j - 1u;
            if (!(ok = W.wait1(p_full, t & 1u))) break;
            if (j == 1 && !(ok = W.wait1(o_empty, (nq & 1u) ^ 1u))) break;
#pragma unroll 1
            for (int m = 0; m < C::kBlocks && ok; ++m)
#pragma unroll
              for (uint32_t g = 0; g < 4; ++g) {
                const uint64_t da = dV + ring.s * kStep;
                if (!(ok = W.wait1(full(ring.s), ring.ph))) break;
                tc_fence_after();
#pragma unroll
                for (uint32_t ks = 0; ks < 4; ++ks)
                  tc_mma2(tO + m * kRows, da + 128 * ks, dP + 128 * (4 * g + ks), IDESC_O,
                          (j > 1 || (g | ks) != 0) ? 1u : 0u);
                tc_commit2(empty(ring.s));
                ring.step();
              }
            if (!ok) break;
            tc_commit2(p_done);
          }
        }
        nt += (uint32_t)n;
        ++nq;
      }
      if (issued) {
        tc_commit2(done_bar);
        drain(done_bar, 0, timeout_ns);
      }
    }
    __syncwarp();
  } else {
    // ================================================ softmax, epilogue
    const int quad = warp & 3, g = warp >> 2;  // TMEM lanes, rows 32 g .. 32 g + 31
    const int r0 = kGroupRows * g;
    const int key = (int)rank * 128 + quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t xs_peer = at_rank(xs, peer), xs_own = at_rank(xs, rank);
    const uint32_t flag_own = at_rank(smem_u32(misc + 2), rank);
    const uint32_t flag_peer = at_rank(smem_u32(misc + 2), peer);
    const uint32_t red_own = at_rank(smem_u32(red), rank), red_peer = at_rank(smem_u32(red), peer);
    const uint32_t l_s_free0 = at_rank(s_free(0), 0), l_o_empty = at_rank(o_empty, 0);
    const uint32_t owner = (uint32_t)g >> 1;  // the CTA that holds P of these rows
    const uint32_t p_row = (owner == rank ? sP : at_rank(sP, peer)) + (uint32_t)key * 128u;
    const uint32_t p_in_peer = at_rank(p_in, peer);
    const uint32_t p_c0 = (uint32_t)(g & 1) * 4u, p_sw = (uint32_t)(key & 7);
    uint32_t nx = 0, ng = 0, nt = 0;
    // all softmax warps of the pair; `publish`: with this warp's writes to both
    // CTAs before it
    auto pair_sync = [&](bool publish) {
      __syncwarp();
      if (lane == 0) {
        if (publish) {
          mbar_release_cluster(xs_own);
          mbar_release_cluster(xs_peer);
        } else {
          mbar_signal(xs_own);
          mbar_signal(xs_peer);
        }
      }
      return W.wait(xs, nx++ & 1u);
    };
    auto group_sync = [&]() {  // all softmax warps of this CTA
      __syncwarp();
      if (lane == 0) mbar_arrive(grp);
      return W.wait(grp, ng++ & 1u);
    };
    bool ok = true;
    while (ok && walk.next(it)) {
      const bool live = it.n_rows > r0;  // this group has rows that count
      int32_t lim_min = it.len;          // keys that every row of the block sees
      if (it.b >= 0) {
        const ReqShape r = req_shape(L, it.b);
        lim_min = row_limit(r, L.H, it.rel0);
        if (tid < kRows)
          lim_s[tid] = min(it.len, row_limit(r, L.H, it.rel0 + min(tid, it.n_rows - 1)));
      } else if (tid < kRows) {
        lim_s[tid] = it.len;
      }
      if (tid < kRows) {
        nm_s[tid] = 0.f;
        nt_s[tid] = INFINITY;
      }
      float l[32];
#pragma unroll
      for (int h = 0; h < 32; ++h) l[h] = 0.f;
      const int n = it.tile1 - it.tile0;
      for (int j = 0; j < n; ++j, ++nt) {
        const uint32_t b = nt & 1u;
        const uint32_t tS = tmem + b * kRows + lane_base + r0;
        if (!(ok = W.wait(s_full(b), (nt >> 1) & 1u))) break;
        tc_fence_after();
        const int32_t pos = (it.tile0 + j) * kKeys + key;
        const bool masked = (it.tile0 + j + 1) * kKeys > lim_min;  // uniform
        // ---- does a score beat its row's maximum by more than 2^8?  (Always
        // taken on a unit's first tile, whose maxima are not set yet.)
        bool need = j == 0;
        if (j > 0 && live) {
          float over = -INFINITY;
#pragma unroll
          for (int h0 = 0; h0 < 32; h0 += 16) {
            uint32_t r[16];
            tmem_ld16(tS + h0, r);
            tmem_wait_ld();
            const float4* nt4 = reinterpret_cast<const float4*>(nt_s + r0 + h0);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 c = nt4[e / 4];
              const float y[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float d = fmaf(__uint_as_float(r[e + x]), scale_log2, y[x]);
                if (!masked || pos < lim_s[r0 + h0 + e + x]) over = fmaxf(over, d);
              }
            }
          }
          need = over > 0.f;
        }
        need = __any_sync(0xffffffffu, need);
        // the flag carries the tile's number, so it never needs clearing
        if (need && lane == 0) {
          st_cluster_u32(flag_own + 4 * b, nt + 1u);
          st_cluster_u32(flag_peer + 4 * b, nt + 1u);
        }
        if (!(ok = pair_sync(need))) break;
        // the previous tile's PV is done: O^T is current and P free
        if (nt > 0 && !(ok = W.wait(p_done, (nt - 1u) & 1u))) break;
        tc_fence_after();
        if (flags[b] == nt + 1u) {
          // ---- exact maxima of the tile, over both CTAs' keys
          float x[32];
#pragma unroll
          for (int h0 = 0; h0 < 32; h0 += 16) {
            uint32_t r[16];
            tmem_ld16(tS + h0, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[h0 + e] = !masked || pos < lim_s[r0 + h0 + e]
                              ? __uint_as_float(r[e]) * scale_log2
                              : -INFINITY;
          }
          column_reduce<true>(x, lane);
          const uint32_t at = 4u * (uint32_t)(((int)rank * 4 + quad) * kRows + r0 + lane);
          st_cluster_u32(red_own + at, __float_as_uint(x[0]));
          st_cluster_u32(red_peer + at, __float_as_uint(x[0]));
          if (!(ok = pair_sync(true))) break;
          if (tid < kRows) {
            float t = red[tid];
#pragma unroll
            for (int w = 1; w < 8; ++w) t = fmaxf(t, red[w * kRows + tid]);
            const float nt_old = nt_s[tid];
            const bool first = nt_old == INFINITY;
            const bool raise = first ? t > -INFINITY : t + nt_old > 0.f;
            alpha_s[tid] = raise && !first ? ex2(-nm_s[tid] - t) : 1.f;
            if (raise) {
              nm_s[tid] = -t;
              nt_s[tid] = -(t + kSlack);
            }
          }
          if (!(ok = group_sync())) break;
          if (j > 0) {
            bool rescale = false;
#pragma unroll
            for (int h = 0; h < 32; ++h) {
              const float a = alpha_s[r0 + h];
              l[h] *= a;
              rescale |= a != 1.f;
            }
            if (rescale) {  // the same in every lane
#pragma unroll 1
              for (int m = 0; m < C::kBlocks; ++m)
#pragma unroll 1
                for (int h0 = 0; h0 < 32; h0 += 16) {
                  uint32_t r[16];
                  const uint32_t ta = tO + m * kRows + lane_base + r0 + h0;
                  tmem_ld16(ta, r);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha_s[r0 + h0 + e]);
                  tmem_st16(ta, r);
                }
              tmem_wait_st();
            }
          }
        }
        // ---- P = 2^(s - m): row sums, and bf16 P into the CTA that owns the rows
        if (live) {
#pragma unroll
          for (int h0 = 0; h0 < 32; h0 += 16) {
            uint32_t r[16];
            tmem_ld16(tS + h0, r);
            tmem_wait_ld();
            if (h0 == 16) {  // the last read of this S^T buffer
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_signal(l_s_free0 + 8 * b);
            }
            float p[16];
            const float4* nm4 = reinterpret_cast<const float4*>(nm_s + r0 + h0);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 c = nm4[e / 4];
              p[e] = ex2(fmaf(__uint_as_float(r[e]), scale_log2, c.x));
              p[e + 1] = ex2(fmaf(__uint_as_float(r[e + 1]), scale_log2, c.y));
              p[e + 2] = ex2(fmaf(__uint_as_float(r[e + 2]), scale_log2, c.z));
              p[e + 3] = ex2(fmaf(__uint_as_float(r[e + 3]), scale_log2, c.w));
            }
            if (masked) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (pos >= lim_s[r0 + h0 + e]) p[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) l[h0 + e] += p[e];
#pragma unroll
            for (int c8 = 0; c8 < 2; ++c8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(p[8 * c8 + 2 * e], p[8 * c8 + 2 * e + 1]);
              const uint32_t a = p_row + (((p_c0 + (uint32_t)(h0 / 8 + c8)) ^ p_sw) << 4);
              if (owner == rank)
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[0]),
                             "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
              else
                st_async_v4(a, w, p_in_peer);
            }
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_signal(l_s_free0 + 8 * b);
        }
        if (owner == rank) {  // what crosses is counted by its bytes
          fence_proxy_async();  // P -> the tensor core's reads
          __syncwarp();
          if (lane == 0) mbar_arrive(p_in);
        }
      }
      if (!ok) break;
      // ---- epilogue: m, l and O of this (unit, pair) to its slot
      const int64_t slot = (int64_t)it.unit + pair;
      if (!(ok = W.wait(p_done, (nt - 1u) & 1u))) break;
      tc_fence_after();
      column_reduce<false>(l, lane);
      lred[quad * kRows + r0 + lane] = l[0];
      if (!(ok = group_sync())) break;
      if (DSA_IN_BOUNDS(slot < n_slots, status)) {
        if (tid < it.n_rows) {
          const float sum = lred[tid] + lred[kRows + tid] + lred[2 * kRows + tid] +
                            lred[3 * kRows + tid];
          view.ml[(slot * 2 + rank) * kRows + tid] =
              make_float2(nt_s[tid] == INFINITY ? -INFINITY : -nm_s[tid], sum);
        }
        float* out = view.o + slot * (int64_t)(kRows * D);
#pragma unroll 1
        for (int m = 0; m < C::kBlocks; ++m) {
          const int dv = m * 256 + (int)rank * 128 + quad * 32 + lane;
          if (dv >= D) break;  // D = 128: the second CTA's lanes are padding
#pragma unroll 1
          for (int h0 = r0; h0 < min(r0 + kGroupRows, it.n_rows); h0 += 16) {
            uint32_t r[16];
            tmem_ld16(tO + m * kRows + lane_base + h0, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (h0 + e < it.n_rows) out[(int64_t)(h0 + e) * D + dv] = __uint_as_float(r[e]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_signal(l_o_empty);
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
  cluster_sync_all();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
}

// ---------------------------------------------------------------- joining
// Row by row, D / 4 threads each: the slots of the row's prefix unit and of
// its own unit, weighted by 2^(m_i - M).  Reads each partial result once;
// kJoin of them in flight.
constexpr int kJoin = 8;

template <int D>
__global__ void __launch_bounds__(128) join_kernel(PlanView view, Lens L,
                                                   __nv_bfloat16* __restrict__ o,
                                                   float* __restrict__ lse, int B,
                                                   int64_t n_rows, int64_t n_slots,
                                                   uint32_t* status) {
  constexpr int kPer = 512 / D, kLanes = D / 4;  // rows of a block, threads of a row
  const int sub = threadIdx.x / kLanes, th = threadIdx.x % kLanes;
  const int64_t row = blockIdx.x * (int64_t)kPer + sub;
  if (row >= n_rows) return;
  const Plan* plan = view.p;
  const int64_t t = row / L.H, chunk = plan->chunk, total = plan->total;
  if (t < __ldg(L.cu) || t >= __ldg(L.cu + B)) return;
  int lo = 0, hi = B;  // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(L.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const ReqShape r = req_shape(L, lo);
  // the two units: first cost, tiles, tiles that hold keys, number, row in it
  int64_t c0[2];
  int32_t tiles[2], used[2], unit[2], at[2];
  int n_units = 0;
  if (plan->prefix_cost > 0 && total > 0) {
    tiles[0] = used[0] = plan->prefix_tiles;
    unit[0] = (int32_t)(row / kRows);
    at[0] = (int32_t)(row % kRows);
    c0[0] = (int64_t)unit[0] * (tiles[0] + kUnitCost);
    n_units = 1;
  }
  if (r.tiles && total > 0) {
    const int32_t rel = (int32_t)row - r.row0, j = rel / kRows;
    const int32_t last = min((j + 1) * kRows, r.n_rows) - 1;
    tiles[n_units] = r.tiles;
    used[n_units] = (min(r.len, row_limit(r, L.H, last)) + kKeys - 1) / kKeys;
    unit[n_units] = __ldg(view.ucum + lo) + j;
    at[n_units] = rel % kRows;
    c0[n_units] = __ldg(view.ccum + lo) + (int64_t)j * (r.tiles + kUnitCost);
    ++n_units;
  }
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x = 0; x < n_units; ++x) {
    const int64_t i0 = c0[x] / chunk, i1 = (c0[x] + tiles[x] + kUnitCost - 1) / chunk;
    for (int64_t i = i0; i <= i1; i += kJoin) {
      float mi[kJoin], li[kJoin];
      float4 oi[kJoin];
      float top = m;
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        mi[e] = -INFINITY;
        li[e] = 0.f;
        oi[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + e > i1) continue;
        int32_t a, z;
        share_of(c0[x], tiles[x], (i + e) * chunk, min(total, (i + e + 1) * chunk), a, z);
        if (a >= min(z, used[x])) continue;
        const int64_t slot = unit[x] + i + e;
        if (!DSA_IN_BOUNDS(slot < n_slots, status)) continue;
        const float2 p0 = view.ml[(slot * 2) * kRows + at[x]];
        const float2 p1 = view.ml[(slot * 2 + 1) * kRows + at[x]];
        mi[e] = p0.x;
        li[e] = p0.y + p1.y;
        oi[e] = reinterpret_cast<const float4*>(view.o + (slot * kRows + at[x]) * D)[th];
      }
#pragma unroll
      for (int e = 0; e < kJoin; ++e) top = fmaxf(top, mi[e]);
      const float keep = top == -INFINITY ? 1.f : ex2(m - top);
      l *= keep;
      acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
      m = top;
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        if (mi[e] == -INFINITY) continue;  // nothing there, or no key seen
        const float w = ex2(mi[e] - top);
        l = fmaf(w, li[e], l);
        acc.x = fmaf(w, oi[e].x, acc.x);
        acc.y = fmaf(w, oi[e].y, acc.y);
        acc.z = fmaf(w, oi[e].z, acc.z);
        acc.w = fmaf(w, oi[e].w, acc.w);
      }
    }
  }
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(o + row * D)[th] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (th == 0) lse[row] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
cudaError_t launch_t(const LaunchCtx& c, const ServeShape& s, const CUtensorMap& qm,
                     const CUtensorMap& km, const CUtensorMap& vm,
                     const int32_t* prefix_table, int32_t prefix_len, const int32_t* table,
                     const Lens& L, __nv_bfloat16* o, float* lse, uint8_t* work) {
  using C = PCfg<D>;
  const PlanView view = plan_view(s, work);
  cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)C::kSmem);
  if (e != cudaSuccess) return e;
  const int pairs = c.num_sms / 2 < kMaxPairs ? c.num_sms / 2 : kMaxPairs;
  plan_kernel<<<1, 1024, 0, c.stream>>>(L, s.B, s.T, prefix_len, pairs, view.p, view.ccum,
                                        view.ucum, c.status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t slots = max_slots(s);
  prefix_attn_kernel<D><<<2 * pairs, kThreads, C::kSmem, c.stream>>>(
      qm, km, vm, view, L, prefix_table, prefix_len, table, s.B, s.max_blocks, s.page_log2,
      (int32_t)s.n_pages, slots, s.scale * kLog2e, c.status, c.timeout_ns);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = s.T * s.H;
  constexpr int per = 512 / D;
  join_kernel<D><<<(unsigned)((rows + per - 1) / per), 128, 0, c.stream>>>(
      view, L, o, lse, s.B, rows, slots, c.status);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_attn_ws(const ServeShape& s) {
  return plan_bytes(s.B) + (size_t)max_slots(s) * kRows * (2 * sizeof(float2) + (size_t)s.D * 4);
}

cudaError_t launch_prefix_attn(const LaunchCtx& c, const ServeShape& s,
                               const CUtensorMap& q_map, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const int32_t* prefix_table,
                               int64_t prefix_len, const int32_t* table,
                               const int32_t* seq, const int32_t* cu, __nv_bfloat16* o,
                               float* lse, uint8_t* work) {
  const Lens L{seq, cu, s.max_blocks << s.page_log2, s.H};
  auto run = [&](auto launch) {
    return launch(c, s, q_map, k_map, v_map, prefix_table, (int32_t)prefix_len, table, L, o,
                  lse, work);
  };
  if (s.D == 128) return run(launch_t<128>);
  if (s.D == 256) return run(launch_t<256>);
  return run(launch_t<512>);
}

}  // namespace dsa
