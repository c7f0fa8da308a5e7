// key_weights.cu -- what the cached tokens of each request receive of its rows'
// attention: sums of weights over the rows, one for each key.
#include "attn_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kKeys = 32;  // of a block: a warp has four

template <int D>
__global__ void __launch_bounds__(256) key_weights_kernel(
    const __nv_bfloat16* q, const float* lse, const __nv_bfloat16* k, const int32_t* table,
    const int32_t* seq, const int32_t* cu, const int32_t* tree_bits, int words, const float* w,
    float decay, float* w_out, int H, int64_t T, int max_blocks, int page_log2, int64_t n_pages,
    int tiles, float scale, uint32_t* status) {
  constexpr int kPer = D / 32;
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c0 = cu[b], c1 = cu[b + 1], n = seq[b], cap = max_blocks << page_log2;
  if (c0 < 0 || c1 < c0 || c1 > T || n < 0 || n > cap) {
    if (threadIdx.x == 0) latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
    return;
  }
  const int32_t n_new = c1 - c0, base = n - n_new;
  if (n_new == 0) return;
  for (int x = 0; x < kKeys / 8; ++x) {
    const int32_t j = tile * kKeys + warp * (kKeys / 8) + x;
    if (j >= n) return;
    const int32_t p = table[(int64_t)b * max_blocks + (j >> page_log2)];
    if (p < 0 || p >= n_pages) {
      latch_error(status, DSA_ERR_DEVICE_BAD_INDEX);
      continue;
    }
    const int64_t slot = ((int64_t)p << page_log2) + (j & ((1 << page_log2) - 1));
    float key[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) key[e] = __bfloat162float(k[slot * D + e * 32 + lane]);
    float sum = 0.f;
    for (int32_t i = 0; i < n_new; ++i) {
      const int32_t node = j - base;
      const bool sees =
          node < 0 ||
          (tree_bits ? node < 32 * words &&
                           (tree_bits[(int64_t)(c0 + i) * words + (node >> 5)] >> (node & 31) & 1)
                     : node <= i);
      if (!sees) continue;
      for (int h = 0; h < H; ++h) {
        const int64_t r = (int64_t)(c0 + i) * H + h;
        const float l = lse[r];
        if (l == -INFINITY) continue;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          s = fmaf(key[e], __bfloat162float(q[r * D + e * 32 + lane]), s);
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
        sum += expf(s * scale - l);
      }
    }
    if (lane == 0) w_out[slot] = (j < base ? decay * w[slot] : 0.f) + sum;
  }
}

}  // namespace

size_t key_weights_ws(const ServeShape&) { return 0; }

cudaError_t launch_key_weights(const LaunchCtx& c, const ServeShape& s, const CUtensorMap&,
                               const CUtensorMap&, const __nv_bfloat16* q, const float* lse,
                               const __nv_bfloat16* k_pages, const int32_t* table,
                               const int32_t* seq, const int32_t* cu,
                               const uint32_t* tree_bits, int words, const float* w_pages,
                               float decay, float* w_out, uint8_t*) {
  const int tiles = (s.max_blocks * s.page + kKeys - 1) / kKeys;
  auto run = [&](auto kern) {
    kern<<<(unsigned)(s.B * tiles), 256, 0, c.stream>>>(
        q, lse, k_pages, table, seq, cu, reinterpret_cast<const int32_t*>(tree_bits), words,
        w_pages, decay, w_out, s.H, s.T, s.max_blocks, s.page_log2, s.n_pages, tiles, s.scale,
        c.status);
    return cudaGetLastError();
  };
  if (s.D == 128) return run(key_weights_kernel<128>);
  if (s.D == 256) return run(key_weights_kernel<256>);
  return run(key_weights_kernel<512>);
}

}  // namespace dsa
