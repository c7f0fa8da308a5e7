// prefix_attn.cu -- attention of a batch of requests over one shared prefix
// and each request's own tokens, both in a paged cache.
//
// One warp per (token, head) row walks the prefix's keys, then the request's
// own up to the token's place, with the running maximum m and sum l of the
// softmax and O in registers (fp32):
//   m' = max(m, s),  O' = O 2^(m - m') + 2^(s - m') v,  l' likewise.
#include "attn_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

template <int D>
__global__ void __launch_bounds__(256) prefix_attn_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ prefix_table,
    int32_t prefix_len, const int32_t* __restrict__ table, const int32_t* __restrict__ seq,
    const int32_t* __restrict__ cu, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
    int64_t T, int B, int H, int max_blocks, int page_log2, int64_t n_pages,
    float scale_log2, uint32_t* status) {
  constexpr int P = D / 64;  // bf16 pairs of a lane: 2 * lane + 64 * p
  const int lane = threadIdx.x & 31;
  const int64_t row = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  if (row >= T * H) return;
  const int64_t t = row / H;
  int lo = 0, hi = B;  // the request: the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int32_t c0 = __ldg(cu + lo), c1 = __ldg(cu + lo + 1);
  if (c0 < 0 || c1 > T) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
  if (t < c0 || t >= c1) return;
  int32_t len = __ldg(seq + lo);
  if (len < 0 || len > (max_blocks << page_log2)) {
    latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    len = 0;
  }
  const int32_t own = max(0, len - (c1 - c0) + (int32_t)(t - c0) + 1);
  float qv[2 * P], acc[2 * P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t x = reinterpret_cast<const uint32_t*>(q + row * D)[lane + 32 * p];
    qv[2 * p] = bf16_lo(x) * scale_log2;
    qv[2 * p + 1] = bf16_hi(x) * scale_log2;
    acc[2 * p] = acc[2 * p + 1] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int part = 0; part < 2; ++part) {
    const int32_t* pages = part ? table + (int64_t)lo * max_blocks : prefix_table;
    const int32_t n = part ? own : prefix_len;
    for (int32_t j = 0; j < n; ++j) {
      const int32_t pg = __ldg(pages + (j >> page_log2));
      if (pg < 0 || pg >= n_pages) {
        latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
        continue;
      }
      const int64_t r = ((int64_t)pg << page_log2) + (j & ((1 << page_log2) - 1));
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(k + r * D) + lane + 32 * p);
        s = fmaf(qv[2 * p], bf16_lo(x), s);
        s = fmaf(qv[2 * p + 1], bf16_hi(x), s);
      }
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
      const float mn = fmaxf(m, s);
      const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
      const float e = mn == -INFINITY ? 0.f : exp2f(s - mn);
      m = mn;
      l = l * a + e;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(v + r * D) + lane + 32 * p);
        acc[2 * p] = fmaf(e, bf16_lo(x), acc[2 * p] * a);
        acc[2 * p + 1] = fmaf(e, bf16_hi(x), acc[2 * p + 1] * a);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
    reinterpret_cast<uint32_t*>(o + row * D)[lane + 32 * p] =
        pack_bf16(acc[2 * p] * inv, acc[2 * p + 1] * inv);
  if (lane == 0) lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t prefix_attn_ws(const ServeShape&) { return 0; }

cudaError_t launch_prefix_attn(const LaunchCtx& c, const ServeShape& s,
                               const __nv_bfloat16* q, const __nv_bfloat16* k,
                               const __nv_bfloat16* v, const int32_t* prefix_table,
                               int64_t prefix_len, const int32_t* table,
                               const int32_t* seq, const int32_t* cu, __nv_bfloat16* o,
                               float* lse, uint8_t*) {
  const int64_t rows = s.T * s.H;
  auto run = [&](auto kern) {
    kern<<<(unsigned)((rows + 7) / 8), 256, 0, c.stream>>>(
        q, k, v, prefix_table, (int32_t)prefix_len, table, seq, cu, o, lse, s.T, s.B, s.H,
        s.max_blocks, s.page_log2, s.n_pages, s.scale * kLog2e, c.status);
  };
  if (s.D == 128) run(prefix_attn_kernel<128>);
  else if (s.D == 256) run(prefix_attn_kernel<256>);
  else run(prefix_attn_kernel<512>);
  return cudaGetLastError();
}

}  // namespace dsa
