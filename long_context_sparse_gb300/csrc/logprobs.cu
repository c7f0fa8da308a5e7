// logprobs.cu -- log probabilities of given tokens, entropy and the best
// alternatives from a row of logits, and their gradient: both stream the logits
// once, with fp32 arithmetic.
//
// Forward.  Of a row x (raw logits), with c = scale log2 e and a reference r near
// the maximum so far:  y = (x - r) c,  s = sum 2^y,  t = sum 2^y y.
//   lse = scale r + ln s,   logp = scale (x_tok - r) - ln s,   H = ln s - ln 2 t / s
// (no term of H cancels another: y <= 0 but for the first batch's own rounding).
// The reference is taken off before the scale, so that large logits lose nothing.
//
// Bounds (in a graph).  4095 rows of 100277 fp32 with 5 alternatives: 246 to 249 us, 6.6 TB/s,
// as a plain copy.  64 rows of 131072 bf16 with 20: 12.4 us, of which the pass 6.1 and six
// short steps of the alternatives, each behind a barrier, the rest; the eager call 22 to 26,
// 15 where the caller has its results (`out`).  4096 rows of 131072 bf16 with 0, 1, 5, 20, 32,
// 48, 64 alternatives: 158 188 192 209 227 262 288.
#include <cuda_fp16.h>
#include <math.h>

#include "attn_common.cuh"
#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kUnroll = 4;      // 16-byte vectors of a thread in flight: a batch
constexpr int kMaxTop = 64;
constexpr int kKept = 4;        // batches that a thread remembers
constexpr int kBuf = 512;       // candidates of a CTA; its cluster's alternatives
constexpr int kMaxCluster = 8;  // CTAs of a row
static_assert(kMaxTop * kMaxCluster <= kBuf, "the leader's buffer");
constexpr float kUnset = -3.402823466e38f;  // reference of nothing but -inf
constexpr float kNever = -16384.f;          // 2^ of it is 0

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// What the stream's work before has left, read once.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_f(const float* p) {
  return __int_as_float(ld_input(reinterpret_cast<const int32_t*>(p)));
}
// A 32-bit word of logits as floats, their maximum, and back.
template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNone = 0xff80ff80u;  // -inf
  __device__ static void get(uint32_t w, float (&x)[2]) {
    x[0] = bf16_lo(w);
    x[1] = bf16_hi(w);
  }
  __device__ static uint32_t put(const float (&x)[2]) { return pack_bf16(x[0], x[1]); }
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
template <>
struct Word<__half> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  __device__ static void get(uint32_t w, float (&x)[2]) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
    x[0] = f.x;
    x[1] = f.y;
  }
  __device__ static uint32_t put(const float (&x)[2]) {
    const __half2 h = __floats2half2_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    const __half2 m =
        __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
template <>
struct Word<float> {
  static constexpr int kPer = 1;
  static constexpr uint32_t kNone = 0xff800000u;
  __device__ static void get(uint32_t w, float (&x)[1]) { x[0] = __uint_as_float(w); }
  __device__ static uint32_t put(const float (&x)[1]) { return __float_as_uint(x[0]); }
  __device__ static uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1(const float* p) {
  return ld_f(p);
}
template <>
__device__ __forceinline__ float load1(const __nv_bfloat16* p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return __uint_as_float((uint32_t)v << 16);
}
template <>
__device__ __forceinline__ float load1(const __half* p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return __half2float(__ushort_as_half(v));
}
template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ float to_type(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 to_type(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half to_type(float x) {
  return __float2half_rn(x);
}

// A logit as an integer in the same order, above 0 (which stands for none): the two
// zeros alike, NaN with -inf, which also fills up a batch.  With its id behind it,
// larger for lower ids.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0x007fffffu : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t full_key(float x, uint32_t id) {
  return ((uint64_t)order_key(x) << 32) | (0xffffffffu - id);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ int32_t key_id(uint64_t k) {
  return (int32_t)(0xffffffffu - (uint32_t)k);
}

// A row: single elements up to the first 16-byte boundary, vectors, single ones.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / (int)sizeof(T);
  const T* at;
  int32_t head, n_vec, vocab;

  __device__ __forceinline__ Row(const T* p, int32_t v) : at(p), vocab(v) {
    head = (int32_t)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    if (head > vocab) head = vocab;
    n_vec = (vocab - head) / kVec;
  }
  __device__ __forceinline__ int32_t n_single() const { return vocab - n_vec * kVec; }
  __device__ __forceinline__ int32_t single(int i) const {  // its id
    return i < head ? i : n_vec * kVec + i;
  }
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(at + head);
  }
  __device__ __forceinline__ int32_t id(int32_t v) const { return head + v * kVec; }
};

struct Stat {
  float r, s, t;
};
// b's sums under a common reference added to a's
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  const float r = fmaxf(a.r, b.r);
  const float da = max_nan((a.r - r) * c, kNever), db = max_nan((b.r - r) * c, kNever);
  const float fa = ex2(da), fb = ex2(db);
  return {r, fa * a.s + fb * b.s, fa * (a.t + da * a.s) + fb * (b.t + db * b.s)};
}

__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A cluster of CTAs has a row, each a share of its vectors.
//
// Alternatives, exactly and in the same pass: each thread remembers its kKept
// batches with the largest maxima.  A value that n of the threads' best elements
// reach is a bound for the n best of the share: here the n-th largest of what the k
// best threads of each warp have, two more than n in all need.  Only the batches whose
// maximum reaches it are looked at again, in L2, an element a lane and eight batches
// on their way at a time, and few elements of those pass.  A thread of which more
// batches than it remembers may reach the bound sends the share through a second look
// at all of it.  Where more elements pass than the buffer holds (rows of many equal
// values), ids break the ties already in the bound; and should that not do either, `n`
// passes each look for the largest below the last.
// Wide: the rows are few and have a cluster each; what is looked at again is found in
// L1 (64 rows of 131072 bf16 with 20 alternatives: 1.2 us less; with a row a CTA, 4% more).
template <typename T, bool Top, bool Wide, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprobs_kernel(
    const T* logits, int64_t ld, int32_t vocab, const int32_t* tokens, int n_top, float scale,
    float* logp, float* lse, float* entropy, int32_t* top_ids, float* top_logp,
    uint32_t* status) {
  constexpr int kWarps = kThreads / 32, kWords = 4 * kUnroll, kStep = kUnroll * kThreads;
  using W = Word<T>;
  __shared__ Stat stats[kWarps];
  __shared__ Stat total;
  __shared__ alignas(16) uint64_t best[Top ? kThreads : 1];
  __shared__ alignas(16) uint64_t buf[Top ? kBuf : 2];
  __shared__ uint64_t top[Top ? kMaxTop : 1];
  // the leader's: what the cluster's CTAs have found
  __shared__ Stat from[kMaxCluster];
  __shared__ alignas(16) uint64_t from_top[Wide && Top ? kMaxTop * kMaxCluster : 2];
  __shared__ uint32_t warp_best[96];
  // [warp][lanes and numbers of the batches that are looked at again]
  __shared__ uint32_t again_list[Top ? kWarps : 1][Top ? 32 * kKept : 1];
  __shared__ uint32_t n_buf, again, tok_at, tok_word;
  __shared__ int32_t token;
  __shared__ uint64_t bound;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  if (Wide) cluster_arrive();  // the leader has begun: waited for before it is written to
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x / size;
  const Row<T> row(logits + r * ld, vocab);
  const float c = scale * kLog2e;
  const uint64_t c2 = pair2(c, c);
  const int32_t per = (row.n_vec + (int)size - 1) / (int)size;
  const int32_t v0 = min(row.n_vec, (int)rank * per), v1 = min(row.n_vec, v0 + per);
  const int n_single = rank == 0 ? row.n_single() : 0;
  const uint4* vec = row.vec();
  const bool has_token = rank == 0 && tid == kThreads - 1;  // the thread that sees to it

  float ref = kUnset;
  uint64_t s2 = 0ull, t2 = 0ull;
  uint32_t kept[kKept];  // order keys of the remembered batches' maxima, largest first
  int32_t which[kKept];  // their numbers; -1: this thread's single element
#pragma unroll
  for (int q = 0; q < kKept; ++q) {
    kept[q] = 0u;
    which[q] = 0;
  }
  auto remember = [&](float m, int32_t i) {
    uint32_t k = order_key(m);
    if (k > kept[kKept - 1]) {
#pragma unroll
      for (int q = 0; q < kKept; ++q) {
        const bool up = k > kept[q];
        const uint32_t k1 = kept[q];
        const int32_t i1 = which[q];
        kept[q] = up ? k : k1;
        which[q] = up ? i : i1;
        k = up ? k1 : k;
        i = up ? i1 : i;
      }
    }
  };
  auto raise = [&](float m) {
    if (m > ref) {
      const float d = max_nan((ref - m) * c, kNever), f = ex2(d);
      t2 = mul2(pair2(f, f), fma2(pair2(d, d), s2, t2));
      s2 = mul2(pair2(f, f), s2);
      ref = m;
    }
  };
  // two elements (of one alone: with -inf beside it)
  auto add = [&](float a, float b, uint64_t minus_ref) {
    float y0, y1;
    unpair2(mul2(add2(pair2(a, b), minus_ref), c2), y0, y1);
    y0 = max_nan(y0, kNever);
    y1 = max_nan(y1, kNever);
    const uint64_t e = pair2(ex2(y0), ex2(y1));
    s2 = add2(s2, e);
    t2 = fma2(e, pair2(y0, y1), t2);
  };
  auto load = [&](int32_t v, uint32_t (&w)[kWords]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint4 x = make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
      if (v + u * kThreads < v1)
        x = Wide && Top ? ld_input(vec + v + u * kThreads) : ld_stream(vec + v + u * kThreads);
      w[4 * u] = x.x;
      w[4 * u + 1] = x.y;
      w[4 * u + 2] = x.z;
      w[4 * u + 3] = x.w;
    }
  };
  auto largest = [&](const uint32_t (&w)[kWords]) {
    uint32_t m[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
    for (int i = 4; i < kWords; ++i) m[i & 3] = W::max(m[i & 3], w[i]);
    float x[W::kPer];
    W::get(W::max(W::max(m[0], m[1]), W::max(m[2], m[3])), x);
    return W::kPer == 2 ? fmaxf(x[0], x[W::kPer - 1]) : x[0];
  };
  int32_t batches = 0;
  auto take_in = [&](const uint32_t (&w)[kWords]) {
    const float m = largest(w);
    if (Top) remember(m, batches);
    ++batches;
    raise(m);
    const uint64_t minus_ref = pair2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < kWords; i += 3 - W::kPer) {
      float x[2];
      if constexpr (W::kPer == 2) {
        W::get(w[i], x);
      } else {
        x[0] = __uint_as_float(w[i]);
        x[1] = __uint_as_float(w[i + 1]);
      }
      add(x[0], x[1], minus_ref);
    }
  };
  {
    // a batch is on its way while the one before it is worked on
    uint32_t w[2][kWords];
    int32_t v = v0 + tid;
    if (v < v1) load(v, w[0]);
    if (has_token)  // on its way to shared memory beside the row
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&token)),
                   "l"(tokens + r)
                   : "memory");
    if (tid < n_single) {
      const float x = load1(row.at + row.single(tid));
      if (Top) remember(x, -1);
      raise(x);
      add(x, -INFINITY, pair2(-ref, -ref));
    }
    for (; v < v1; v += 2 * kStep) {
      if (v + kStep < v1) load(v + kStep, w[1]);
      take_in(w[0]);
      if (v + kStep >= v1) break;
      if (v + 2 * kStep < v1) load(v + 2 * kStep, w[0]);
      take_in(w[1]);
    }
  }
  // ---- the share's sums
  Stat all;
  {
    float a, b;
    all.r = ref;
    unpair2(s2, a, b);
    all.s = a + b;
    unpair2(t2, a, b);
    all.t = a + b;
  }
  auto merge_lanes = [&](int from) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      if (s > from) continue;
      const Stat o{__shfl_xor_sync(0xffffffffu, all.r, s), __shfl_xor_sync(0xffffffffu, all.s, s),
                   __shfl_xor_sync(0xffffffffu, all.t, s)};
      all = lane & s ? merge(o, all, c) : merge(all, o, c);
    }
  };
  if (has_token) {  // and the word that holds its logit beside what follows
    asm volatile("cp.async.wait_all;" ::: "memory");
    int32_t tok = token;
    if (tok >= vocab) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      tok = -1;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(row.at + (tok < 0 ? 0 : tok));
    tok_at = tok < 0 ? ~0u : (uint32_t)(at & 3u);
    if (tok >= 0)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&tok_word)),
                   "l"(at & ~(uintptr_t)3)
                   : "memory");
  }
  merge_lanes(16);
  if (lane == 0) stats[warp] = all;
  if (tid == 0) n_buf = again = 0u;
  // the elements of the thread's share, at least of the vectors whose largest order
  // key reaches floor(): f(value, id)
  auto visit_all = [&](auto floor, auto f) {
    if (tid < n_single) f(load1(row.at + row.single(tid)), (uint32_t)row.single(tid));
    for (int32_t v = v0 + tid; v < v1; v += kStep) {
      uint32_t w[kWords];
      load(v, w);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (v + u * kThreads >= v1) break;
        float x[W::kPer];
        W::get(W::max(W::max(w[4 * u], w[4 * u + 1]), W::max(w[4 * u + 2], w[4 * u + 3])), x);
        if (order_key(W::kPer == 2 ? fmaxf(x[0], x[W::kPer - 1]) : x[0]) < floor()) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          W::get(w[4 * u + i], x);
#pragma unroll
          for (int e = 0; e < W::kPer; ++e)
            f(x[e], (uint32_t)(row.id(v + u * kThreads) + i * W::kPer + e));
        }
      }
    }
  };
  // the n keys of `list` in order: f(key, place); all threads
  auto in_order = [&](const uint64_t* list, int n, auto f) {
    const int even = n & ~1;
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = list[i];
      int place = 0;
#pragma unroll 8
      for (int j = 0; j < even; j += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(list + j);
        place += (o.x > key) + (o.y > key);
      }
      if (even < n) place += list[even] > key;
      f(key, place);
    }
  };
  // ---- the share's alternatives, in order, into top[]
  if (Top) {
    // the threads that have vectors come first; whole warps of them have k each
    const int full = min(kThreads, v1 - v0) >> 5;
    const int k = full ? min((n_top + full - 1) / full + (n_top > 24 ? 2 : 1), 96 / full) : 33;
    if (k <= 32 && warp < full) {
      uint32_t mine = kept[0];
      for (int i = 0; i < k; ++i) {
        const uint32_t reached = __reduce_max_sync(0xffffffffu, mine);
        const uint32_t who = __ballot_sync(0xffffffffu, mine == reached);
        if (lane == __ffs(who) - 1) mine = 0u;
        if (lane == 0) warp_best[warp * k + i] = reached;
      }
    }
    for (int i = tid; i < kMaxTop; i += kThreads) top[i] = 0ull;
    __syncthreads();
    uint32_t least = 0u;
    if (k <= 32) {  // full * k values, n_top or more: from the nearer end
      const int list = full * k;
      uint32_t x[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) x[i] = lane + 32 * i < list ? warp_best[lane + 32 * i] : 0u;
      // counted from above 0 stands for none, from below (of what is left of ~0) too
      const bool up = n_top > list - n_top;
#pragma unroll
      for (int i = 0; i < 3; ++i) x[i] = up && x[i] ? ~x[i] : x[i];
      for (int i = up ? list - n_top + 1 : n_top; i > 0; --i) {
        least = __reduce_max_sync(0xffffffffu, max(max(x[0], x[1]), x[2]));
        const uint32_t who =
            __ballot_sync(0xffffffffu, x[0] == least || x[1] == least || x[2] == least);
        if (lane == __ffs(who) - 1) {
          if (x[0] == least) x[0] = 0u;
          else if (x[1] == least) x[1] = 0u;
          else x[2] = 0u;
        }
      }
      if (up) least = ~least;
    }
    uint64_t at_least = (uint64_t)least << 32;
    auto reach = [&] { return (uint32_t)(at_least >> 32); };
    auto push = [&](float x, uint32_t id) {
      const uint64_t key = full_key(x, id);
      if (key < at_least) return;
      const uint32_t i = atomicAdd(&n_buf, 1u);
      if (i < kBuf) buf[i] = key;
    };
    if (kept[kKept - 1] && kept[kKept - 1] >= least && batches + (tid < n_single) > kKept)
      again = 1u;
    constexpr int kElems = kUnroll * Row<T>::kVec, kPerLoad = 32 / kElems, kLoads = 8;
    int listed = 0;
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const uint32_t who = __ballot_sync(0xffffffffu, kept[q] && kept[q] >= least);
      if (who >> lane & 1u)
        again_list[warp][listed + __popc(who & ((1u << lane) - 1u))] =
            (uint32_t)lane | (uint32_t)(which[q] + 1) << 5;
      listed += __popc(who);
    }
    __syncwarp();
    for (int i0 = 0; i0 < listed; i0 += kLoads * kPerLoad) {
      float x[kLoads];
      uint32_t id[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = i0 + i * kPerLoad + lane / kElems, e = lane % kElems;
        id[i] = ~0u;
        if (at < listed) {
          const uint32_t entry = again_list[warp][at];
          const int t = (warp << 5) + (int)(entry & 31u), number = (int)(entry >> 5) - 1;
          if (number < 0) {
            if (e == 0) id[i] = (uint32_t)row.single(t);
          } else {
            const int32_t v = v0 + t + number * kStep + e / Row<T>::kVec * kThreads;
            if (v < v1) id[i] = (uint32_t)(row.id(v) + e % Row<T>::kVec);
          }
        }
        if (id[i] != ~0u) x[i] = load1(row.at + id[i]);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (id[i] != ~0u) push(x[i], id[i]);
    }
    __syncthreads();
    if (again) {
      __syncthreads();
      if (tid == 0) n_buf = 0u;
      __syncthreads();
      visit_all(reach, push);
      __syncthreads();
    }
    if (n_buf > kBuf) {
      // the n-th largest of the threads' best elements, by value and id
      uint64_t mine = 0ull;
      visit_all([&] { return (uint32_t)(mine >> 32); }, [&](float x, uint32_t id) {
        const uint64_t f = full_key(x, id);
        mine = f > mine ? f : mine;
      });
      best[tid] = mine;
      if (tid == 0) bound = 0ull;
      __syncthreads();
      int above = 0;
      for (int i = 0; i < kThreads; i += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(best + i);
        above += (o.x > mine) + (o.y > mine);
      }
      if (mine && above == n_top - 1) bound = mine;
      if (tid == 0) n_buf = 0u;
      __syncthreads();
      at_least = bound;
      if (mine >= at_least) visit_all(reach, push);
      __syncthreads();
    }
    if (n_buf > kBuf) {
      uint64_t last = ~0ull;
      for (int i = 0; i < n_top; ++i) {
        uint64_t most = 0ull;
        visit_all([&] { return (uint32_t)(most >> 32); }, [&](float x, uint32_t id) {
          const uint64_t f = full_key(x, id);
          if (f < last && f > most) most = f;
        });
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, most, s);
          most = o > most ? o : most;
        }
        if (lane == 0) best[warp] = most;
        __syncthreads();
        for (int x = 0; x < kWarps; ++x) most = best[x] > most ? best[x] : most;
        if (tid == 0) top[i] = most;
        last = most;
        __syncthreads();
      }
    } else {
      in_order(buf, (int)n_buf, [&](uint64_t key, int place) {
        if (place < n_top) top[place] = key;
      });
    }
  }
  __syncthreads();
  if (warp == 0) {
    all = lane < kWarps ? stats[lane] : Stat{kUnset, 0.f, 0.f};
    merge_lanes(kWarps / 2);
    if (lane == 0) total = all;
  }
  // ---- the row's: the others write to the leader, and go
  if (Wide) {
    cluster_wait();
    __syncthreads();
    if (tid < 3) {
      const float x = tid == 0 ? total.r : tid == 1 ? total.s : total.t;
      st_cluster_u32(at_rank(smem_u32(&from[rank]) + 4 * tid, 0), __float_as_uint(x));
    }
    if (Top && rank != 0)
      for (int i = tid; i < 2 * n_top; i += kThreads)
        st_cluster_u32(at_rank(smem_u32(from_top + rank * n_top) + 4 * i, 0),
                       reinterpret_cast<const uint32_t*>(top)[i]);
    if (Top && rank == 0 && tid < n_top) from_top[tid] = top[tid];
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) {
      all = lane < (int)size ? from[lane] : Stat{kUnset, 0.f, 0.f};
      merge_lanes(kMaxCluster / 2);
      if (lane == 0) total = all;
    }
    if (Top) {
      // none below the largest of the CTAs' n-th ones is among the row's n
      uint64_t least = 0ull;
      for (uint32_t g = 0; g < size; ++g) {
        const uint64_t last = from_top[(g + 1) * n_top - 1];
        least = last > least ? last : least;
      }
      if (tid == 0) n_buf = 0u;
      __syncthreads();
      for (int i = tid; i < (int)size * n_top; i += kThreads)
        if (from_top[i] && from_top[i] >= least) buf[atomicAdd(&n_buf, 1u)] = from_top[i];
      __syncthreads();
      in_order(buf, (int)n_buf, [&](uint64_t key, int place) {
        if (place < n_top) top[place] = key;
      });
    }
  }
  if (has_token) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const Stat s = total;
  const bool none = s.s == 0.f;  // nothing but -inf
  const float ln = logf(s.s);
  if (tid == 0) {
    lse[r] = none ? -INFINITY : fmaf(s.r, scale, ln);
    entropy[r] = none ? 0.f : ln - kLn2 * (s.t / s.s);
    float x[W::kPer];
    W::get(tok_word, x);
    logp[r] = tok_at == ~0u ? 0.f
              : none        ? -INFINITY
                            : (x[W::kPer == 2 && tok_at ? 1 : 0] - s.r) * scale - ln;
  }
  if (Top)
    for (int i = tid; i < n_top; i += kThreads) {
      const uint64_t key = top[i];
      if (!DSA_IN_BOUNDS((uint32_t)key_id(key) < (uint32_t)vocab, status)) continue;
      top_ids[r * n_top + i] = key_id(key);
      top_logp[r * n_top + i] = none ? -INFINITY : (key_value(key) - s.r) * scale - ln;
    }
}

// Backward.  With l = log p = scale x - lse:  dx = 2^(l log2 e) (A + B l) + 1[tok] G,
//   A = -scale (g + h H),  B = -scale h,  G = scale g.
// 8192 rows of 131072 bf16: 607 us, 7.1 TB/s (as long where half of them have no gradient:
// their logits are read all the same); 301 of 50257 fp16 10 us (in a graph; eager 15).
// A block takes kUnroll vectors a thread of one row, as the gradient lies in its 16
// bytes.  Where the logits lie differently, a vector of them is put together from the
// two that hold it: the neighbour's second is this one's first, and comes from L1
// (2048 rows of 131071: 178 us, 6 TB/s; element by element 689).
constexpr int kBwdThreads = 256;

// 16 bytes from byte 4 * words + 2 * half on of the 32 in lo, hi
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, uint32_t words,
                                         uint32_t half) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 7; ++i) w[i] = words & 1u ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = words & 2u ? w[i + 2] : w[i];
  const uint32_t s = 16u * half;
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                    __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

// Alike: every row's logits lie as its gradient does (the path aside costs 12 registers
// and 6% of 8192 rows of 131072).
template <typename T, bool Alike>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(
    const T* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t segs,
    const int32_t* tokens, const float* lse, const float* entropy, const float* g_logp,
    const float* g_entropy, float scale, T* dlogits, int64_t ld_grad, uint32_t* status) {
  using W = Word<T>;
  constexpr int kSeg = kUnroll * kBwdThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  for (int64_t item = blockIdx.x; item < rows * segs; item += gridDim.x) {
    const int64_t r = item / segs;
    const int32_t seg = (int32_t)(item - r * segs);
    const T* x_row = logits + r * ld;
    T* out = dlogits + r * ld_grad;
    const Row<T> row(out, vocab);  // divided as the gradient lies
    const T* first = x_row + row.head;
    const uint32_t off =
        Alike ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(first) & 15u);
    const uint4* vec = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(first) - off) +
                       (int64_t)seg * kSeg + tid;
    const int32_t v0 = seg * kSeg + tid;
    uint4 in[kUnroll];
    if (Alike || off == 0u) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * kBwdThreads < row.n_vec) in[u] = ld_stream(vec + u * kBwdThreads);
    } else {  // (each of the two vectors holds some of the row)
      uint4 hi[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * kBwdThreads < row.n_vec) {
          in[u] = ld_input(vec + u * kBwdThreads);
          hi[u] = ld_input(vec + u * kBwdThreads + 1);
        }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * kBwdThreads < row.n_vec)
          in[u] = shifted(in[u], hi[u], off >> 2, (off >> 1) & 1u);
    }
    int32_t tok = ld_input(tokens + r);
    if (tok >= vocab) {
      if (tid == 0 && seg == 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      tok = -1;
    }
    const float l0 = ld_f(lse + r);
    const float g = g_logp && tok >= 0 ? ld_f(g_logp + r) : 0.f;
    const float h = g_entropy ? ld_f(g_entropy + r) : 0.f;
    const float A = -scale * (g_entropy ? fmaf(h, ld_f(entropy + r), g) : g);
    const float B = -scale * h, G = scale * g;
    // a padding row's logits may be anything.  (They are on their way by now: looking
    // before they are asked for costs all other rows, 667 us at 606 for 8192 of 131072.)
    if (l0 == -INFINITY || (g == 0.f && h == 0.f)) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * kBwdThreads < row.n_vec)
          reinterpret_cast<uint4*>(out + row.head)[v0 + u * kBwdThreads] =
              make_uint4(0u, 0u, 0u, 0u);
      if (seg == 0 && tid < row.n_single()) out[row.single(tid)] = to_type<T>(0.f);
      continue;
    }
    auto grad = [&](float x, int32_t id) {
      const float l = max_nan(fmaf(x, scale, -l0), kNever);
      float d = ex2(l * kLog2e) * fmaf(B, l, A);
      if (id == tok) d += G;
      return d;
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t v = v0 + u * kBwdThreads;
      if (v >= row.n_vec) break;
      uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[W::kPer];
        W::get(w[i], x);
#pragma unroll
        for (int e = 0; e < W::kPer; ++e) x[e] = grad(x[e], row.id(v) + i * W::kPer + e);
        w[i] = W::put(x);
      }
      reinterpret_cast<uint4*>(out + row.head)[v] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (seg == 0 && tid < row.n_single()) {
      const int32_t id = row.single(tid);
      out[id] = to_type<T>(grad(load1(x_row + id), id));
    }
  }
}

// Rows that no address space holds.
dsa_status_t check_ld(const dsa_logprobs_config_t* c, int64_t ld) {
  return ld >= (int64_t)1 << 40 || c->rows > ((int64_t)1 << 45) / ld ? DSA_ERR_UNSUPPORTED_SHAPE
                                                                    : DSA_OK;
}

dsa_status_t check_logprobs(const dsa_logprobs_config_t* c) {
  if (!c) return DSA_ERR_INVALID_ARG;
  if (c->rows < 1 || c->vocab < 1 || c->ld < c->vocab || c->dtype < DSA_BF16 ||
      c->dtype > DSA_FP32 || c->n_top < 0 || c->n_top > c->vocab || !(c->scale > 0.f) ||
      isinf(c->scale * kLog2e) || c->reserved != 0)
    return DSA_ERR_INVALID_ARG;
  if (c->rows >= (int64_t)1 << 31 || c->vocab >= (int64_t)1 << 30 || c->n_top > kMaxTop)
    return DSA_ERR_UNSUPPORTED_SHAPE;
  return check_ld(c, c->ld);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t elem_bytes(const dsa_logprobs_config_t* c) { return c->dtype == DSA_FP32 ? 4 : 2; }

size_t span_bytes(const dsa_logprobs_config_t* c, int64_t ld) {
  return ((size_t)(c->rows - 1) * (size_t)ld + (size_t)c->vocab) * elem_bytes(c);
}

dsa_status_t check_ws256(void* ws, size_t ws_bytes) {
  if (!ws) return DSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DSA_ERR_MISALIGNED;
  return ws_bytes < kHeader ? DSA_ERR_WORKSPACE_TOO_SMALL : DSA_OK;
}

// A launch that may begin while what is before it in the stream runs.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Launch(const LaunchCtx& c, unsigned grid, int threads, int cluster) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
};

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status_t dsa_token_logprobs(const dsa_logprobs_config_t* cfg, const void* logits,
                                const int32_t* tokens, float* logp, float* lse, float* entropy,
                                int32_t* top_ids, float* top_logp, void* ws, size_t ws_bytes,
                                void* stream) {
  dsa_status_t st = check_logprobs(cfg);
  if (st != DSA_OK) return st;
  if (!logits || !tokens || !logp || !lse || !entropy || !top_ids != (cfg->n_top == 0) ||
      !top_logp != (cfg->n_top == 0))
    return DSA_ERR_INVALID_ARG;
  if ((st = check_ws256(ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {tokens, logp, lse, entropy, top_ids, top_logp};
  for (const void* p : ptrs)
    if (!aligned4(p)) return DSA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(cfg)) return DSA_ERR_MISALIGNED;
  const size_t R = (size_t)cfg->rows, tops = R * (size_t)cfg->n_top * 4;
  const Span reads[] = {{logits, span_bytes(cfg, cfg->ld)}, {tokens, R * 4}};
  const Span writes[] = {{logp, R * 4},     {lse, R * 4},       {entropy, R * 4},
                         {top_ids, tops}, {top_logp, tops}, {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  // A row to as many CTAs as two an SM allow, each with a batch of every thread at
  // least.  us in a graph with 1, 2, 4, 8 CTAs a row of 131072 bf16, 20 alternatives: 16
  // rows 16.7 14.0 12.3 11.0; 64 rows 17.5 15.3 13.5 14.9; 150 rows 18 16.9 22.3 30.7; 300
  // rows 23.4 24.8 35.8 53.8.
  int size = 1;
  const int64_t one = kUnroll * (16 / (int64_t)elem_bytes(cfg)), batch = 256 * one;
  while (size < kMaxCluster && cfg->rows * size <= ctx.num_sms &&
         cfg->vocab >= 2 * size * batch)
    size *= 2;
  if (cfg->rows * size >= (int64_t)1 << 31) return DSA_ERR_UNSUPPORTED_SHAPE;
  // Many rows: the steps behind a row's last logit are waits more than work, so that
  // short rows want few threads and many CTAs an SM; where a thread's batches are many
  // the second looks take over.  us with 32, 128, 256 threads, 20 alternatives, bf16: 8192
  // rows of 1000 28 67 119; 4000 of 4096 27 35 55; 2000 of 16384 54 31 38; 4000 of 32000 -
  // 90 89; 4096 of 131072 - 230 208; with 64 alternatives 8192 of 1000 500 127 215.
  int threads = 256;
  if (cfg->rows > ctx.num_sms && cfg->vocab <= 16 * 32 * one) threads = 128;
  if (cfg->rows > ctx.num_sms && cfg->vocab <= 4 * 32 * one && cfg->n_top <= 24) threads = 32;
  Launch l(ctx, (unsigned)(cfg->rows * size), threads, size);
  auto run = [&](auto zero) {
    using T = decltype(zero);
    const bool top = cfg->n_top > 0;
    auto kern = size > 1         ? (top ? logprobs_kernel<T, true, true, 256>
                                        : logprobs_kernel<T, false, true, 256>)
                : threads == 32  ? (top ? logprobs_kernel<T, true, false, 32>
                                        : logprobs_kernel<T, false, false, 32>)
                : threads == 128 ? (top ? logprobs_kernel<T, true, false, 128>
                                        : logprobs_kernel<T, false, false, 128>)
                                 : (top ? logprobs_kernel<T, true, false, 256>
                                        : logprobs_kernel<T, false, false, 256>);
    return cuda_status(cudaLaunchKernelEx(&l.cfg, kern, static_cast<const T*>(logits), cfg->ld,
                                          (int32_t)cfg->vocab, tokens, (int)cfg->n_top,
                                          cfg->scale, logp, lse, entropy, top_ids, top_logp,
                                          ctx.status));
  };
  if (cfg->dtype == DSA_BF16) return run(__nv_bfloat16());
  if (cfg->dtype == DSA_FP16) return run(__half());
  return run(float());
}

dsa_status_t dsa_token_logprobs_bwd(const dsa_logprobs_config_t* cfg, const void* logits,
                                    const int32_t* tokens, const float* lse,
                                    const float* entropy, const float* g_logp,
                                    const float* g_entropy, void* dlogits, int64_t ld_grad,
                                    void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t st = check_logprobs(cfg);
  if (st != DSA_OK) return st;
  if (!logits || !tokens || !lse || (g_entropy && !entropy) || !dlogits ||
      ld_grad < cfg->vocab)
    return DSA_ERR_INVALID_ARG;
  if ((st = check_ld(cfg, ld_grad)) != DSA_OK) return st;
  if ((st = check_ws256(ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {tokens, lse, entropy, g_logp, g_entropy};
  for (const void* p : ptrs)
    if (!aligned4(p)) return DSA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(cfg) ||
      reinterpret_cast<uintptr_t>(dlogits) % elem_bytes(cfg))
    return DSA_ERR_MISALIGNED;
  const size_t R = (size_t)cfg->rows;
  const bool same = dlogits == logits && ld_grad == cfg->ld;
  const Span reads[] = {{same ? nullptr : logits, span_bytes(cfg, cfg->ld)},
                        {tokens, R * 4},
                        {lse, R * 4},
                        {entropy, R * 4},
                        {g_logp, R * 4},
                        {g_entropy, R * 4}};
  const Span writes[] = {{dlogits, span_bytes(cfg, ld_grad)}, {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  const int64_t per = (int64_t)kBwdThreads * kUnroll * (16 / (int64_t)elem_bytes(cfg));
  const int32_t segs = (int32_t)((cfg->vocab + per - 1) / per);
  const int64_t items = cfg->rows * segs, most = ((int64_t)1 << 31) - 1;
  Launch l(ctx, (unsigned)(items < most ? items : most), kBwdThreads, 1);
  const size_t e = elem_bytes(cfg);
  const bool alike =
      ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15u) == 0 &&
      (cfg->rows == 1 || ((size_t)(cfg->ld - ld_grad) * e & 15u) == 0);
  auto run = [&](auto zero) {
    using T = decltype(zero);
    return cuda_status(cudaLaunchKernelEx(
        &l.cfg, alike ? logprobs_bwd_kernel<T, true> : logprobs_bwd_kernel<T, false>,
        static_cast<const T*>(logits), cfg->ld, cfg->rows, (int32_t)cfg->vocab, segs, tokens, lse,
        entropy, g_logp, g_entropy, cfg->scale, static_cast<T*>(dlogits), ld_grad, ctx.status));
  };
  if (cfg->dtype == DSA_BF16) return run(__nv_bfloat16());
  if (cfg->dtype == DSA_FP16) return run(__half());
  return run(float());
}

}  // extern "C"
