// serve_api.cu -- the serving entry points of include/dsa.h: argument
// checks, workspace sizes and launches.  Host code only.
#include <math.h>

#include "attn_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 20;  // T * H of dsa_prefix_attn

dsa_status_t check_serve(const dsa_serve_config_t* c, int which) {
  if (!c) return DSA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->max_tokens < 1 || c->page_size < 1 || c->batch < 1 ||
      c->max_blocks < 1 || c->attn_heads < 1 || c->d_qk < 1 || c->d_v < 1 ||
      !(c->sm_scale >= 0.f) || isinf(c->sm_scale * kLog2e))
    return DSA_ERR_INVALID_ARG;
  const int p = c->page_size;
  if (p != 16 && p != 32 && p != 64 && p != 128) return DSA_ERR_UNSUPPORTED_SHAPE;
  // slots and TMA row coordinates are int32
  if (c->n_pages > (((int64_t)1 << 31) - 257) / p) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (c->max_tokens >= (int64_t)1 << 30) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (c->batch > 65536) return DSA_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)c->max_blocks * p >= (int64_t)1 << 30) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (which != DSA_SERVE_WS_TABLES) {
    if (c->d_qk != 128 && c->d_qk != 256 && c->d_qk != 512) return DSA_ERR_UNSUPPORTED_SHAPE;
    if (c->d_v != c->d_qk) return DSA_ERR_UNSUPPORTED_SHAPE;
  }
  if (which == DSA_SERVE_WS_PREFIX) {
    if (c->attn_heads > 128) return DSA_ERR_UNSUPPORTED_SHAPE;
    if (c->max_tokens * c->attn_heads > kMaxRows) return DSA_ERR_UNSUPPORTED_SHAPE;
  }
  return DSA_OK;
}

ServeShape serve_shape(const dsa_serve_config_t* c) {
  ServeShape s;
  s.n_pages = c->n_pages;
  s.T = c->max_tokens;
  s.page = c->page_size;
  s.page_log2 = 0;
  while ((1 << s.page_log2) < s.page) ++s.page_log2;
  s.B = c->batch;
  s.max_blocks = c->max_blocks;
  s.H = c->attn_heads;
  s.D = c->d_qk;
  s.scale = c->sm_scale > 0.f ? c->sm_scale : 1.0f / sqrtf((float)c->d_qk);
  return s;
}

size_t serve_ws_bytes(const dsa_serve_config_t* c, int which) {
  return kHeader + (which == DSA_SERVE_WS_PREFIX ? prefix_attn_ws(serve_shape(c)) : 0);
}

dsa_status_t check_serve_ws(const dsa_serve_config_t* c, int which, void* ws,
                            size_t ws_bytes) {
  if (!ws) return DSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DSA_ERR_MISALIGNED;
  if (ws_bytes < serve_ws_bytes(c, which)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  return DSA_OK;
}

struct Span {
  const void* at;
  size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x && y && a.bytes && b.bytes && (x <= y ? y - x < a.bytes : x - y < b.bytes);
}

// Whether what a call writes meets what it reads, or itself: its blocks read
// and write in no order.
template <int W, int R>
bool written_meets(const Span (&w)[W], const Span (&r)[R]) {
  for (int i = 0; i < W; ++i) {
    for (int j = 0; j < R; ++j)
      if (overlap(w[i], r[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(w[i], w[j])) return true;
  }
  return false;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status_t dsa_serve_workspace_size(const dsa_serve_config_t* cfg, int32_t which,
                                      size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  if (which < DSA_SERVE_WS_TABLES || which > DSA_SERVE_WS_PREFIX) return DSA_ERR_INVALID_ARG;
  const dsa_status_t st = check_serve(cfg, which);
  if (st != DSA_OK) return st;
  *bytes = serve_ws_bytes(cfg, which);
  return DSA_OK;
}

dsa_status_t dsa_build_page_tables(const dsa_serve_config_t* cfg, const int32_t* cached_lens,
                                   const int32_t* new_lens, const int32_t* free_pages,
                                   int64_t n_free, int32_t* block_table, int32_t* slot_map,
                                   int32_t* cu_tokens, int32_t* seq_lens,
                                   int32_t* pages_taken, void* ws, size_t ws_bytes,
                                   void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_TABLES);
  if (st != DSA_OK) return st;
  if (!cached_lens || !new_lens || n_free < 0 || (n_free > 0 && !free_pages) ||
      !block_table || !slot_map || !cu_tokens || !seq_lens || !pages_taken)
    return DSA_ERR_INVALID_ARG;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_TABLES, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {cached_lens, new_lens, block_table, slot_map,
                        cu_tokens,   seq_lens, pages_taken};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(free_pages) & 3u) != 0) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch;
  const size_t frees = n_free < (int64_t)1 << 40 ? n_free : (int64_t)1 << 40;
  const Span reads[] = {{cached_lens, B * 4}, {new_lens, B * 4}, {free_pages, frees * 4}};
  const Span writes[] = {{block_table, B * (size_t)cfg->max_blocks * 4},
                         {slot_map, (size_t)cfg->max_tokens * 4},
                         {cu_tokens, (B + 1) * 4},
                         {seq_lens, B * 4},
                         {pages_taken, 4},
                         {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  return cuda_status(launch_page_tables(ctx, serve_shape(cfg), cached_lens, new_lens,
                                        free_pages, n_free, block_table, slot_map,
                                        cu_tokens, seq_lens, pages_taken));
}

dsa_status_t dsa_append_cache(const dsa_serve_config_t* cfg, const int32_t* slot_map,
                              const void* k_new, const void* v_new, void* k_pages,
                              void* v_pages, void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_APPEND);
  if (st != DSA_OK) return st;
  if (!slot_map || !k_new || !k_pages || !v_new != !v_pages) return DSA_ERR_INVALID_ARG;
  if (v_pages == k_pages) return DSA_ERR_INVALID_ARG;  // K = V: both v pointers null
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_APPEND, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {slot_map, k_new, v_new, k_pages, v_pages};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  const size_t T = (size_t)cfg->max_tokens, row = (size_t)cfg->d_qk * 2;
  const size_t cache = (size_t)cfg->n_pages * cfg->page_size * row;
  const Span reads[] = {{slot_map, T * 4}, {k_new, T * row}, {v_new, T * row}};
  const Span writes[] = {{k_pages, cache}, {v_pages, cache}, {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  return cuda_status(launch_append(ctx, serve_shape(cfg), slot_map,
                                   static_cast<const __nv_bfloat16*>(k_new),
                                   static_cast<const __nv_bfloat16*>(v_new),
                                   static_cast<__nv_bfloat16*>(k_pages),
                                   static_cast<__nv_bfloat16*>(v_pages)));
}

dsa_status_t dsa_prefix_attn(const dsa_serve_config_t* cfg, const void* q,
                             const void* k_pages, const void* v_pages,
                             const int32_t* prefix_table, int64_t prefix_len,
                             const int32_t* block_table, const int32_t* seq_lens,
                             const int32_t* cu_tokens, void* o, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_PREFIX);
  if (st != DSA_OK) return st;
  if (!q || !k_pages || prefix_len < 0 || (prefix_len > 0 && !prefix_table) ||
      !block_table || !seq_lens || !cu_tokens || !o || !lse)
    return DSA_ERR_INVALID_ARG;
  if (prefix_len >= (int64_t)1 << 30) return DSA_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_PREFIX, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {q, k_pages, v_pages, prefix_table, block_table,
                        seq_lens, cu_tokens, o, lse};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch, page = (size_t)cfg->page_size;
  const size_t rows = (size_t)cfg->max_tokens * cfg->attn_heads, row = (size_t)cfg->d_qk * 2;
  const size_t cache = (size_t)cfg->n_pages * page * row;
  // o and lse are written by the joining kernel, which reads the lengths and the
  // workspace but not q
  const Span reads[] = {{k_pages, cache},
                        {v_pages, cache},
                        {prefix_table, ((size_t)prefix_len + page - 1) / page * 4},
                        {block_table, B * (size_t)cfg->max_blocks * 4},
                        {seq_lens, B * 4},
                        {cu_tokens, (B + 1) * 4}};
  const Span work = {ws, serve_ws_bytes(cfg, DSA_SERVE_WS_PREFIX)};
  const Span writes[] = {{o, rows * row}, {lse, rows * 4}, work};
  if (written_meets(writes, reads) || overlap(work, {q, rows * row})) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  const ServeShape sh = serve_shape(cfg);
  CUtensorMap qm, km, vm[3];
  const uint64_t cache_rows = (uint64_t)sh.n_pages * sh.page, d = (uint64_t)sh.D;
  const uint32_t box = (uint32_t)sh.page;
  if ((st = encode_2d(&qm, q, (uint64_t)(sh.T * sh.H), d, 64)) != DSA_OK) return st;
  if ((st = encode_2d(&km, k_pages, cache_rows, d, box)) != DSA_OK) return st;
  vm[0] = km;
  const void* v = v_pages ? v_pages : k_pages;
  if (v != k_pages && (st = encode_2d(&vm[0], v, cache_rows, d, box)) != DSA_OK) return st;
  if ((st = encode_2d(&vm[1], v, cache_rows, d, 8)) != DSA_OK) return st;
  if ((st = encode_2d(&vm[2], v, cache_rows, d, 1)) != DSA_OK) return st;
  return cuda_status(launch_prefix_attn(ctx, sh, qm, km, vm, prefix_table, prefix_len,
                                        block_table, seq_lens, cu_tokens,
                                        static_cast<__nv_bfloat16*>(o), lse,
                                        static_cast<uint8_t*>(ws) + kHeader));
}

}  // extern "C"
