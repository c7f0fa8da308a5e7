// logprobs.cu -- log probabilities of given tokens, entropy and the best
// alternatives from a row of logits, and their gradient: both stream the logits
// once, with fp32 arithmetic.
//
// Forward.  Of a row x (raw logits), with c = scale log2 e and a reference r near
// the maximum so far:  y = (x - r) c,  s = sum 2^y,  t = sum 2^y y.
//   lse = scale r + ln s,   logp = scale (x_tok - r) - ln s,   H = ln s - ln 2 t / s
// (no term of H cancels another: y <= 0 but for the first batch's own rounding).
// The reference is taken off before the scale, so that large logits lose nothing.
#include <cuda_fp16.h>
#include <math.h>

#include "attn_common.cuh"
#include "dsa_internal.h"
#include "pair_common.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;      // 16-byte vectors of a thread in flight: a batch
constexpr int kMaxTop = 64;
constexpr int kKept = 4;        // batches that a thread remembers
constexpr int kBuf = 512;       // candidates of a CTA; alternatives of a cluster
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
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
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

// A logit as an integer in the same order (the two zeros alike, NaN below -inf and
// above 0, which stands for none); with its id behind it, larger for lower ids.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 1u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
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

// A cluster of CTAs has a row, each a share of its vectors.
//
// Alternatives, exactly and in the same pass: each thread remembers its kKept
// batches with the largest maxima.  The n-th largest of the threads' best elements
// is a bound that the n-th largest of the share reaches, so that only batches whose
// maximum reaches it are looked at again (they are in L2).  A thread of which more
// batches than it remembers may reach it, or a full buffer, sends the share through
// `slow`: n passes, each for the largest below the one before.
template <typename T, bool Top>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(
    const T* logits, int64_t ld, int32_t vocab, const int32_t* tokens, int n_top, float scale,
    float* logp, float* lse, float* entropy, int32_t* top_ids, float* top_logp,
    uint32_t* status) {
  constexpr int kWords = 4 * kUnroll;
  using W = Word<T>;
  __shared__ Stat stats[kWarps];
  __shared__ Stat total;
  __shared__ alignas(16) uint64_t best[Top ? kThreads : 1];
  __shared__ uint64_t buf[Top ? kBuf : 1];
  __shared__ uint64_t top[Top ? kMaxTop : 1];
  __shared__ uint32_t n_buf, again;
  __shared__ uint64_t bound;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x / size;
  const Row<T> row(logits + r * ld, vocab);
  const float c = scale * kLog2e;
  const int32_t per = (row.n_vec + (int)size - 1) / (int)size;
  const int32_t v0 = min(row.n_vec, (int)rank * per), v1 = min(row.n_vec, v0 + per);
  const int n_single = rank == 0 ? row.n_single() : 0;

  Stat a{kUnset, 0.f, 0.f};
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
    if (m > a.r) {
      const float d = max_nan((a.r - m) * c, kNever), f = ex2(d);
      a.t = f * (a.t + d * a.s);
      a.s *= f;
      a.r = m;
    }
  };
  auto add = [&](float x) {
    const float y = max_nan((x - a.r) * c, kNever), e = ex2(y);
    a.s += e;
    a.t += e * y;
  };
  if (tid < n_single) {
    const float x = load1(row.at + row.single(tid));
    if (Top) remember(x, -1);
    raise(x);
    add(x);
  }
  const uint4* vec = row.vec();
  int32_t batches = 0;
  for (int32_t v = v0 + tid; v < v1; v += kUnroll * kThreads, ++batches) {
    uint32_t w[kWords];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint4 x = make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
      if (v + u * kThreads < v1) x = ld_stream(vec + v + u * kThreads);
      w[4 * u] = x.x;
      w[4 * u + 1] = x.y;
      w[4 * u + 2] = x.z;
      w[4 * u + 3] = x.w;
    }
    uint32_t m[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
    for (int i = 4; i < kWords; ++i) m[i & 3] = W::max(m[i & 3], w[i]);
    float x[W::kPer];
    W::get(W::max(W::max(m[0], m[1]), W::max(m[2], m[3])), x);
    const float top_x = W::kPer == 2 ? fmaxf(x[0], x[W::kPer - 1]) : x[0];
    if (Top) remember(top_x, batches);
    raise(top_x);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      W::get(w[i], x);
#pragma unroll
      for (int e = 0; e < W::kPer; ++e) add(x[e]);
    }
  }
  // ---- the share's sums
  Stat all = a;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const Stat o{__shfl_xor_sync(0xffffffffu, all.r, s), __shfl_xor_sync(0xffffffffu, all.s, s),
                 __shfl_xor_sync(0xffffffffu, all.t, s)};
    all = lane & s ? merge(o, all, c) : merge(all, o, c);
  }
  if (lane == 0) stats[warp] = all;
  if (tid == 0) {
    n_buf = again = 0u;
    bound = 0ull;
  }
  // each candidate of the thread's remembered batch q: f(value, id)
  auto visit = [&](int32_t number, auto f) {
    if (number < 0) {
      f(load1(row.at + row.single(tid)), (uint32_t)row.single(tid));
      return;
    }
    const int32_t v = v0 + tid + number * kUnroll * kThreads;
#pragma unroll 1
    for (int u = 0; u < kUnroll && v + u * kThreads < v1; ++u) {
      const uint4 q = ld_input(vec + v + u * kThreads);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[W::kPer];
        W::get(w[i], x);
#pragma unroll
        for (int e = 0; e < W::kPer; ++e)
          f(x[e], (uint32_t)(row.id(v + u * kThreads) + i * W::kPer + e));
      }
    }
  };
  // ---- the share's alternatives, in order, into top[]
  if (Top) {
    uint64_t mine = 0ull;
    if (kept[0])
      visit(which[0], [&](float x, uint32_t id) {
        const uint64_t k = full_key(x, id);
        mine = k > mine ? k : mine;
      });
    best[tid] = mine;
    if (tid < kMaxTop) top[tid] = 0ull;
    __syncthreads();
    int above = 0;
    for (int i = 0; i < kThreads; i += 2) {
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(best + i);
      above += (k.x > mine) + (k.y > mine);
    }
    if (mine && above == n_top - 1) bound = mine;
    __syncthreads();
    const uint64_t at_least = bound;
    const uint32_t least = (uint32_t)(at_least >> 32);
    if (kept[0] && kept[0] >= least) {
      if (kept[kKept - 1] >= least && batches + (tid < n_single) > kKept) again = 1u;
#pragma unroll 1
      for (int q = 0; q < kKept; ++q) {
        const uint32_t kq = q == 0 ? kept[0] : q == 1 ? kept[1] : q == 2 ? kept[2] : kept[3];
        const int32_t wq = q == 0 ? which[0] : q == 1 ? which[1] : q == 2 ? which[2] : which[3];
        if (kq == 0u || kq < least) break;
        visit(wq, [&](float x, uint32_t id) {
          const uint64_t k = full_key(x, id);
          if (k < at_least) return;
          const uint32_t i = atomicAdd(&n_buf, 1u);
          if (i < kBuf) buf[i] = k;
        });
      }
    }
    __syncthreads();
    if (again || n_buf > kBuf) {
      uint64_t last = ~0ull;
      for (int i = 0; i < n_top; ++i) {
        uint64_t k = 0ull;
        auto take = [&](float x, uint32_t id) {
          const uint64_t f = full_key(x, id);
          if (f < last && f > k) k = f;
        };
        if (tid < n_single) visit(-1, take);
        for (int32_t q = 0; q < batches; ++q) visit(q, take);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, k, s);
          k = o > k ? o : k;
        }
        if (lane == 0) best[warp] = k;
        __syncthreads();
        for (int x = 0; x < kWarps; ++x) k = best[x] > k ? best[x] : k;
        if (tid == 0) top[i] = k;
        last = k;
        __syncthreads();
      }
    } else {
      const int n = (int)n_buf;
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = buf[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += buf[j] > k;
        if (place < n_top) top[place] = k;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    Stat s = stats[0];
    for (int x = 1; x < kWarps; ++x) s = merge(s, stats[x], c);
    total = s;
  }
  __syncthreads();
  // ---- the row's
  if (size > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank == 0) {
      if (tid == 0) {
        Stat s = total;
        for (uint32_t g = 1; g < size; ++g) {
          const uint32_t at = at_rank(smem_u32(&total), g);
          const Stat o{__uint_as_float(ld_cluster(at)), __uint_as_float(ld_cluster(at + 4)),
                       __uint_as_float(ld_cluster(at + 8))};
          s = merge(s, o, c);
        }
        total = s;
      }
      if (Top) {
        const int n = (int)size * n_top;
        for (int i = tid; i < n; i += kThreads) {
          const uint32_t at = at_rank(smem_u32(top + i % n_top), i / n_top);
          buf[i] = ld_cluster(at) | ((uint64_t)ld_cluster(at + 4) << 32);
        }
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
          const uint64_t k = buf[i];
          int place = 0;
          for (int j = 0; j < n; ++j) place += buf[j] > k;
          if (k && place < n_top) top[place] = k;
        }
      }
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  if (rank != 0) return;
  const Stat s = total;
  const bool none = s.s == 0.f;  // nothing but -inf
  const float ln = logf(s.s);
  if (tid == 0) {
    int32_t tok = ld_input(tokens + r);
    if (tok >= vocab) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      tok = -1;
    }
    lse[r] = none ? -INFINITY : fmaf(s.r, scale, ln);
    entropy[r] = none ? 0.f : ln - kLn2 * (s.t / s.s);
    logp[r] = tok < 0 ? 0.f : none ? -INFINITY : (load1(row.at + tok) - s.r) * scale - ln;
  }
  if (Top && tid < n_top) {
    const uint64_t k = top[tid];
    top_ids[r * n_top + tid] = key_id(k);
    top_logp[r * n_top + tid] = none ? -INFINITY : (key_value(k) - s.r) * scale - ln;
  }
}

// Backward.  With l = log p = scale x - lse:  dx = 2^(l log2 e) (A + B l) + 1[tok] G,
//   A = -scale (g + h H),  B = -scale h,  G = scale g.
// A block takes kUnroll vectors a thread of one row; a row whose logits and
// gradients lie differently in their 16 bytes goes element by element.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(
    const T* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t segs,
    const int32_t* tokens, const float* lse, const float* entropy, const float* g_logp,
    const float* g_entropy, float scale, T* dlogits, int64_t ld_grad, uint32_t* status) {
  using W = Word<T>;
  constexpr int kVec = Row<T>::kVec, kSeg = kUnroll * kThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  for (int64_t item = blockIdx.x; item < rows * segs; item += gridDim.x) {
    const int64_t r = item / segs;
    const int32_t seg = (int32_t)(item - r * segs);
    const Row<T> row(logits + r * ld, vocab);
    T* out = dlogits + r * ld_grad;
    const bool alike =
        ((reinterpret_cast<uintptr_t>(row.at) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    const uint4* vec = row.vec() + (int64_t)seg * kSeg + tid;
    const int32_t v0 = seg * kSeg + tid;
    uint4 in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (alike && v0 + u * kThreads < row.n_vec) in[u] = ld_stream(vec + u * kThreads);
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
    const bool none = l0 == -INFINITY;
    auto grad = [&](float x, int32_t id) {
      const float l = max_nan(fmaf(x, scale, -l0), kNever);
      float d = ex2(l * kLog2e) * fmaf(B, l, A);
      if (id == tok) d += G;
      return none ? 0.f : d;
    };
    if (alike) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int32_t v = v0 + u * kThreads;
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
        out[id] = to_type<T>(grad(load1(row.at + id), id));
      }
    } else {
      const int32_t end = min((int64_t)vocab, ((int64_t)seg + 1) * kSeg * kVec);
      for (int32_t id = seg * kSeg * kVec + tid; id < end; id += kThreads)
        out[id] = to_type<T>(grad(load1(row.at + id), id));
    }
  }
}

dsa_status_t check_logprobs(const dsa_logprobs_config_t* c) {
  if (!c) return DSA_ERR_INVALID_ARG;
  if (c->rows < 1 || c->vocab < 1 || c->ld < c->vocab || c->dtype < DSA_BF16 ||
      c->dtype > DSA_FP32 || c->n_top < 0 || c->n_top > c->vocab || !(c->scale > 0.f) ||
      isinf(c->scale * kLog2e) || c->reserved != 0)
    return DSA_ERR_INVALID_ARG;
  if (c->rows >= (int64_t)1 << 31 || c->vocab >= (int64_t)1 << 30 ||
      c->ld >= (int64_t)1 << 40 || c->n_top > kMaxTop)
    return DSA_ERR_UNSUPPORTED_SHAPE;
  return DSA_OK;
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
  Launch(const LaunchCtx& c, unsigned grid, int cluster) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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
  // a row to a CTA where that fills the GPU, else to as many as that takes, each
  // with a batch of every thread at least
  int size = 1;
  const int64_t batch = (int64_t)kThreads * kUnroll * (16 / (int64_t)elem_bytes(cfg));
  while (size < kMaxCluster && cfg->rows * size < 4 * (int64_t)ctx.num_sms &&
         cfg->vocab >= 2 * size * batch)
    size *= 2;
  if (cfg->rows * size >= (int64_t)1 << 31) return DSA_ERR_UNSUPPORTED_SHAPE;
  Launch l(ctx, (unsigned)(cfg->rows * size), size);
  auto run = [&](auto zero, auto with, auto without) {
    using T = decltype(zero);
    return cuda_status(cudaLaunchKernelEx(&l.cfg, cfg->n_top ? with : without,
                                          static_cast<const T*>(logits), cfg->ld,
                                          (int32_t)cfg->vocab, tokens, (int)cfg->n_top,
                                          cfg->scale, logp, lse, entropy, top_ids, top_logp,
                                          ctx.status));
  };
  if (cfg->dtype == DSA_BF16)
    return run(__nv_bfloat16(), logprobs_kernel<__nv_bfloat16, true>,
               logprobs_kernel<__nv_bfloat16, false>);
  if (cfg->dtype == DSA_FP16)
    return run(__half(), logprobs_kernel<__half, true>, logprobs_kernel<__half, false>);
  return run(float(), logprobs_kernel<float, true>, logprobs_kernel<float, false>);
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
  if (ld_grad >= (int64_t)1 << 40) return DSA_ERR_UNSUPPORTED_SHAPE;
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
  const int64_t per = (int64_t)kThreads * kUnroll * (16 / (int64_t)elem_bytes(cfg));
  const int32_t segs = (int32_t)((cfg->vocab + per - 1) / per);
  const int64_t items = cfg->rows * segs, most = ((int64_t)1 << 31) - 1;
  Launch l(ctx, (unsigned)(items < most ? items : most), 1);
  auto run = [&](auto zero, auto kern) {
    using T = decltype(zero);
    return cuda_status(cudaLaunchKernelEx(
        &l.cfg, kern, static_cast<const T*>(logits), cfg->ld, cfg->rows, (int32_t)cfg->vocab,
        segs, tokens, lse, entropy, g_logp, g_entropy, cfg->scale, static_cast<T*>(dlogits),
        ld_grad, ctx.status));
  };
  if (cfg->dtype == DSA_BF16) return run(__nv_bfloat16(), logprobs_bwd_kernel<__nv_bfloat16>);
  if (cfg->dtype == DSA_FP16) return run(__half(), logprobs_bwd_kernel<__half>);
  return run(float(), logprobs_bwd_kernel<float>);
}

}  // extern "C"
