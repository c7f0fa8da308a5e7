// serve_tables.cu -- the paged cache around the shared-prefix attention: page
// tables and slots from request lengths, the append of new rows, the masks of
// drafted trees, and the pages that an eviction leaves free.
#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

// ------------------------------------------------------------ page tables
// Two exclusive sums over the requests (pages to add, tokens to add) say
// where each request's share of the free list and of the slot map begins.
// A block owns kReq consecutive requests and adds up the requests before
// them itself (coalesced reads that hit L2; at B = 65536 the last block
// reads 512 KB), so no block waits for another and one launch does it all.
// Blocks of one column (gridDim.y) share the owned requests' pages and
// tokens.  64 requests of one token: 2.9 us, latency (one read of the lengths,
// one reduction, one scan, a search, a page id and a write).  2047 requests of
// 1.05M slots (4.8 MB, 0.7 us of HBM): 8.8 us, of which 5.9 are the slots: each
// has its own search of eight steps, page id and 4-byte store, where those of a
// page could share all but the store.
constexpr int kReq = 256;

struct ReqLens {
  int32_t cached, fresh;
};

__device__ __forceinline__ ReqLens req_lens(const int32_t* cached, const int32_t* fresh,
                                            int b, int32_t cap, uint32_t* status) {
  ReqLens r{__ldg(cached + b), __ldg(fresh + b)};
  if (r.cached < 0 || r.fresh < 0 || r.cached > cap || r.fresh > cap - r.cached) {
    latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    r.cached = r.fresh = 0;
  }
  return r;
}

__global__ void __launch_bounds__(kReq) page_tables_kernel(
    const int32_t* __restrict__ cached, const int32_t* __restrict__ fresh,
    const int32_t* __restrict__ free_pages, int64_t n_free, int32_t* __restrict__ table,
    int32_t* __restrict__ slots, int32_t* __restrict__ cu, int32_t* __restrict__ seq,
    int32_t* __restrict__ taken, int B, int max_blocks, int page_log2, int64_t n_pages,
    int64_t T, uint32_t* status) {
  __shared__ int64_t s_pages[kReq + 1], s_tokens[kReq + 1];  // first page / token
  __shared__ int32_t s_cached[kReq];
  __shared__ int64_t red[2][kReq / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << page_log2;
  const int32_t cap = max_blocks << page_log2;
  const int b0 = blockIdx.x * kReq;
  const bool last = blockIdx.x == gridDim.x - 1;
  auto pages_of = [&](const ReqLens& r) {
    return ((r.cached + r.fresh + page - 1) >> page_log2) - ((r.cached + page - 1) >> page_log2);
  };
  // ---- the requests before this block's
  int64_t np = 0, nt = 0;
  for (int b = tid; b < b0; b += kReq) {
    const ReqLens r = req_lens(cached, fresh, b, cap, status);
    np += pages_of(r);
    nt += r.fresh;
  }
  np = warp_sum(np);
  nt = warp_sum(nt);
  if (lane == 0) {
    red[0][warp] = np;
    red[1][warp] = nt;
  }
  // ---- this block's own: an exclusive scan
  ReqLens r{0, 0};
  if (b0 + tid < B) r = req_lens(cached, fresh, b0 + tid, cap, status);
  const int64_t my_p = pages_of(r), my_t = r.fresh;
  int64_t ip = my_p, it = my_t;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, ip, s);
    const int64_t c = __shfl_up_sync(0xffffffffu, it, s);
    if (lane >= s) {
      ip += a;
      it += c;
    }
  }
  __shared__ int64_t wtot[2][kReq / 32];
  if (lane == 31) {
    wtot[0][warp] = ip;
    wtot[1][warp] = it;
  }
  __syncthreads();
  int64_t base_p = 0, base_t = 0;
#pragma unroll
  for (int w = 0; w < kReq / 32; ++w) {
    base_p += red[0][w];
    base_t += red[1][w];
    if (w < warp) {
      ip += wtot[0][w];
      it += wtot[1][w];
    }
  }
  s_pages[tid] = base_p + ip - my_p;
  s_tokens[tid] = base_t + it - my_t;
  s_cached[tid] = r.cached;
  if (tid == kReq - 1) {
    s_pages[kReq] = base_p + ip;
    s_tokens[kReq] = base_t + it;
  }
  __syncthreads();
  if (blockIdx.y == 0 && b0 + tid < B) {
    cu[b0 + tid] = (int32_t)min(s_tokens[tid], T);
    seq[b0 + tid] = r.cached + r.fresh;
  }
  if (blockIdx.y == 0 && last && tid == 0) {
    cu[B] = (int32_t)min(s_tokens[kReq], T);
    taken[0] = (int32_t)min(s_pages[kReq], (int64_t)INT32_MAX);
    if (s_tokens[kReq] > T) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
  }
  // the request of element x: the last whose first element is <= x (requests
  // without elements share their successor's first)
  auto find = [&](const int64_t* first, int64_t x) {
    int lo = 0;
#pragma unroll
    for (int s = kReq / 2; s > 0; s >>= 1)
      if (first[lo + s] <= x) lo += s;
    return lo;
  };
  // entry i of the free list, or -1
  auto take = [&](int64_t i) -> int32_t {
    if (i >= n_free) {
      latch_error(status, DSA_ERR_DEVICE_NO_PAGES);
      return -1;
    }
    const int32_t p = __ldg(free_pages + i);
    if (p < 0 || p >= n_pages) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      return -1;
    }
    return p;
  };
  const int64_t step = (int64_t)gridDim.y * kReq, me = (int64_t)blockIdx.y * kReq + tid;
  for (int64_t x = s_pages[0] + me; x < s_pages[kReq]; x += step) {
    const int i = find(s_pages, x);
    const int have = (s_cached[i] + page - 1) >> page_log2;
    table[(int64_t)(b0 + i) * max_blocks + have + (x - s_pages[i])] = take(x);
  }
  const int64_t t_end = min(s_tokens[kReq], T);
  for (int64_t x = s_tokens[0] + me; x < t_end; x += step) {
    const int i = find(s_tokens, x);
    const int32_t pos = s_cached[i] + (int32_t)(x - s_tokens[i]);
    const int have = (s_cached[i] + page - 1) >> page_log2, blk = pos >> page_log2;
    int32_t p;
    if (blk >= have) {
      p = take(s_pages[i] + (blk - have));
    } else {  // the open page that the request holds already
      p = table[(int64_t)(b0 + i) * max_blocks + blk];
      if (p < 0 || p >= n_pages) {
        latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
        p = -1;
      }
    }
    slots[x] = p < 0 ? -1 : (p << page_log2) + (pos & (page - 1));
  }
  if (last)
    for (int64_t x = t_end + me; x < T; x += step) slots[x] = -1;
}

// ---------------------------------------------------------------- append
// One 16-byte piece of a row per thread and tensor, kUnroll rows' pieces in
// flight: a copy, bound by HBM (each row read once and written once).
// 131071 rows of K and V, d = 512 (537 MB): 80.7 us, 6.7 TB/s, 98% of a plain
// copy's rate; 64 rows of one tensor: 1.2 us.
constexpr int kUnroll = 4;

template <int D>
__global__ void __launch_bounds__(256) append_kernel(
    const int32_t* __restrict__ slots, const uint4* __restrict__ k_new,
    const uint4* __restrict__ v_new, uint4* __restrict__ k_pages, uint4* __restrict__ v_pages,
    int64_t T, int64_t n_slots, uint32_t* status) {
  constexpr int kPieces = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the stream's work before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t n = T * kPieces, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t x0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x0 < n;
       x0 += kUnroll * step) {
    int64_t dst[kUnroll];
    uint4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t x = x0 + u * step;
      dst[u] = -1;
      if (x >= n) continue;
      const int32_t s = ld_input(slots + x / kPieces);
      if (s >= n_slots) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      if (s < 0 || s >= n_slots) continue;
      dst[u] = (int64_t)s * kPieces + x % kPieces;
      a[u] = ld_input(k_new + x);
      if (v_new) b[u] = ld_input(v_new + x);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (dst[u] < 0) continue;
      k_pages[dst[u]] = a[u];
      if (v_new) v_pages[dst[u]] = b[u];
    }
  }
}

// ----------------------------------------------------------- released pages
// The other way round: what each request gives back begins behind what the
// requests before it do, whose sum each block works out itself, as above.  64
// requests of up to 64 pages: 4 us, the chain of lengths, scan, page id and store.
__global__ void __launch_bounds__(kReq) release_kernel(
    const int32_t* seq, const int32_t* keep,
    const int32_t* table, int32_t* __restrict__ new_lens,
    int32_t* __restrict__ pages, int64_t n_max, int32_t* __restrict__ n_released, int B,
    int max_blocks, int page_log2, uint32_t* status) {
  __shared__ int64_t s_first[kReq + 1];
  __shared__ int32_t s_left[kReq];  // pages that the request keeps
  __shared__ int64_t red[kReq / 32], wtot[kReq / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << page_log2;
  const int32_t cap = max_blocks << page_log2;
  const int b0 = blockIdx.x * kReq;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the stream's work before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto lens = [&](int b, int32_t& n, int32_t& left) {
    n = ld_input(seq + b);
    const int32_t k = ld_input(keep + b);
    if (n < 0 || n > cap || k < 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    left = k < 0 || n < 0 || n > cap ? n : min(n, k);
    return n < 0 || n > cap
               ? 0
               : (int32_t)(((n + page - 1) >> page_log2) - ((left + page - 1) >> page_log2));
  };
  int32_t n, left = 0;
  int64_t before = 0;
  for (int b = tid; b < b0; b += kReq) before += lens(b, n, left);
  before = warp_sum(before);
  if (lane == 0) red[warp] = before;
  left = 0;
  const int64_t mine = b0 + tid < B ? lens(b0 + tid, n, left) : 0;
  int64_t incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += a;
  }
  if (lane == 31) wtot[warp] = incl;
  __syncthreads();
  int64_t base = 0;
#pragma unroll
  for (int w = 0; w < kReq / 32; ++w) {
    base += red[w];
    if (w < warp) incl += wtot[w];
  }
  s_first[tid] = base + incl - mine;
  s_left[tid] = (left + page - 1) >> page_log2;
  if (tid == kReq - 1) s_first[kReq] = base + incl;
  __syncthreads();
  if (blockIdx.y == 0 && b0 + tid < B) new_lens[b0 + tid] = left;
  if (blockIdx.y == 0 && blockIdx.x == gridDim.x - 1 && tid == 0) {
    n_released[0] = (int32_t)min(s_first[kReq], (int64_t)INT32_MAX);
    if (s_first[kReq] > n_max) latch_error(status, DSA_ERR_DEVICE_NO_PAGES);
  }
  const int64_t end = min(s_first[kReq], n_max);
  const int64_t step = (int64_t)gridDim.y * kReq;
  for (int64_t x = s_first[0] + (int64_t)blockIdx.y * kReq + tid; x < end; x += step) {
    int lo = 0;
#pragma unroll
    for (int s = kReq / 2; s > 0; s >>= 1)
      if (s_first[lo + s] <= x) lo += s;
    pages[x] = ld_input(table + (int64_t)(b0 + lo) * max_blocks + s_left[lo] + (x - s_first[lo]));
  }
}

// ------------------------------------------------------------- tree masks
// A thread for each word of a row's mask walks up from the row's node; numbers
// fall on the way, so it may stop below its word: at most 32 * words steps,
// whatever the parents hold.  In a graph: 7 nodes 1.6 us, 24 random trees of up to 64 2 to 4,
// latency (offsets, then a parent from L1 for each step).  Long chains are slow, since each
// word of a row walks for itself: 64 nodes (2 words) 4.9 us, 256 (8) 65, 1024 (32) 3540.
__global__ void __launch_bounds__(256) tree_kernel(const int32_t* parents,
                                                   const int32_t* cu, int words,
                                                   uint32_t* __restrict__ bits, int B, int64_t T,
                                                   uint32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    const int32_t c0 = ld_input(cu + b), c1 = ld_input(cu + b + 1);
    if (c0 < 0 || c1 < c0 || c1 > T) {
      if (threadIdx.x == 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      continue;
    }
    const int32_t n = c1 - c0;
    if (n > 32 * words) {
      if (threadIdx.x == 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      continue;
    }
    const int32_t* up = parents + c0;
    for (int64_t x = threadIdx.x; x < (int64_t)n * words; x += blockDim.x) {
      const int32_t i = (int32_t)(x / words), lo = (int32_t)(x % words) * 32;
      uint32_t m = 0u;
      for (int32_t j = i; j >= lo;) {
        if (j < lo + 32) m |= 1u << (j - lo);
        const int32_t p = ld_input(up + j);
        if (p < -1 || p >= j) {
          latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
          break;
        }
        j = p;
      }
      bits[(int64_t)c0 * words + x] = m;
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const LaunchCtx& c, const ServeShape& s,
                               const int32_t* cached, const int32_t* fresh,
                               const int32_t* free_pages, int64_t n_free, int32_t* table,
                               int32_t* slots, int32_t* cu, int32_t* seq, int32_t* taken) {
  const int chunks = (s.B + kReq - 1) / kReq;
  // about 4 slots a thread, at most four blocks an SM (2047 requests, 1.05M slots:
  // with two or eight 2 us longer: each adds up the requests before it)
  int64_t y = (s.T + 4 * kReq - 1) / (4 * kReq);
  const int64_t most = 4 * (int64_t)c.num_sms / chunks;
  if (y > most) y = most;
  if (y < 1) y = 1;
  page_tables_kernel<<<dim3(chunks, (unsigned)y), kReq, 0, c.stream>>>(
      cached, fresh, free_pages, n_free, table, slots, cu, seq, taken, s.B, s.max_blocks,
      s.page_log2, s.n_pages, s.T, c.status);
  return cudaGetLastError();
}

cudaError_t launch_append(const LaunchCtx& c, const ServeShape& s, const int32_t* slots,
                          const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                          __nv_bfloat16* k_pages, __nv_bfloat16* v_pages) {
  const int64_t n = s.T * (s.D / 8);
  int64_t g = (n + 255) / 256;
  const int64_t cap = (int64_t)c.num_sms * 8;
  if (g > cap) g = cap;
  // Launched while what is before it in the stream runs, which it waits for on the
  // device, as the attention behind it is (an append of 64 rows and the smallest
  // attention, call after call: 1.4 us less).  The page tables are not: their
  // largest case took 1 us longer so.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)g);
  cfg.blockDim = dim3(256);
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    return cudaLaunchKernelEx(&cfg, kern, slots, reinterpret_cast<const uint4*>(k_new),
                              reinterpret_cast<const uint4*>(v_new),
                              reinterpret_cast<uint4*>(k_pages),
                              reinterpret_cast<uint4*>(v_pages), s.T,
                              (int64_t)(s.n_pages * s.page), c.status);
  };
  if (s.D == 128) return run(append_kernel<128>);
  if (s.D == 256) return run(append_kernel<256>);
  return run(append_kernel<512>);
}

// A launch that may begin while what is before it in the stream runs: the kernels
// wait for its end on the device.
template <typename... P, typename... A>
static cudaError_t launch_early(const LaunchCtx& c, dim3 grid, int threads, void (*kern)(P...),
                                A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_build_tree(const LaunchCtx& c, const ServeShape& s, const int32_t* parents,
                              const int32_t* cu, int words, uint32_t* tree_bits) {
  const int most = c.num_sms * 8;
  return launch_early(c, dim3(s.B < most ? s.B : most), 256, tree_kernel, parents, cu, words,
                      tree_bits, s.B, s.T, c.status);
}

cudaError_t launch_release_pages(const LaunchCtx& c, const ServeShape& s, const int32_t* seq,
                                 const int32_t* keep, const int32_t* table,
                                 int32_t* new_lens, int32_t* pages, int64_t n_max,
                                 int32_t* n_released) {
  // a column for each 8 page ids a thread that the block's requests can have
  const int chunks = (s.B + kReq - 1) / kReq;
  const int64_t ids = (int64_t)(s.B < kReq ? s.B : kReq) * s.max_blocks;
  int64_t y = (ids + 8 * kReq - 1) / (8 * kReq);
  const int64_t most = 4 * (int64_t)c.num_sms / chunks;
  if (y > most) y = most;
  if (y < 1) y = 1;
  return launch_early(c, dim3(chunks, (unsigned)y), kReq, release_kernel, seq, keep, table,
                      new_lens, pages, n_max, n_released, s.B, s.max_blocks, s.page_log2,
                      c.status);
}

}  // namespace dsa
