// serve_api.cu -- the serving entry points of include/dsa.h: argument
// checks, workspace sizes and launches.  Host code only.
#include <math.h>

#include "attn_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 20;  // T * H of the attention calls
constexpr int kMaxWords = 32;                   // of a row of tree_bits

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
  if (which != DSA_SERVE_WS_TABLES && which != DSA_SERVE_WS_TREE) {
    if (c->d_qk != 128 && c->d_qk != 256 && c->d_qk != 512) return DSA_ERR_UNSUPPORTED_SHAPE;
    if (c->d_v != c->d_qk) return DSA_ERR_UNSUPPORTED_SHAPE;
  }
  if (which == DSA_SERVE_WS_EVICT && (int64_t)c->max_blocks * p > (int64_t)1 << 22)
    return DSA_ERR_UNSUPPORTED_SHAPE;
  if (which == DSA_SERVE_WS_PREFIX || which == DSA_SERVE_WS_WEIGHTS) {
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
  switch (which) {
    case DSA_SERVE_WS_PREFIX: return kHeader + prefix_attn_ws(serve_shape(c));
    case DSA_SERVE_WS_WEIGHTS: return kHeader + key_weights_ws(serve_shape(c));
    case DSA_SERVE_WS_EVICT: return kHeader + evict_ws(serve_shape(c));
    default: return kHeader;
  }
}

dsa_status_t check_serve_ws(const dsa_serve_config_t* c, int which, void* ws,
                            size_t ws_bytes) {
  if (!ws) return DSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DSA_ERR_MISALIGNED;
  if (ws_bytes < serve_ws_bytes(c, which)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  return DSA_OK;
}

// Both attention calls; tree_bits NULL: the rows of a request see its tokens in order.
dsa_status_t attend(const dsa_serve_config_t* cfg, const void* q, const void* k_pages,
                    const void* v_pages, const int32_t* prefix_table, int64_t prefix_len,
                    const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* cu_tokens, const uint32_t* tree_bits, int words, void* o,
                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_PREFIX);
  if (st != DSA_OK) return st;
  if (!q || !k_pages || prefix_len < 0 || (prefix_len > 0 && !prefix_table) ||
      !block_table || !seq_lens || !cu_tokens || !o || !lse)
    return DSA_ERR_INVALID_ARG;
  if (prefix_len >= (int64_t)1 << 30) return DSA_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_PREFIX, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {q, k_pages, v_pages, prefix_table, block_table,
                        seq_lens, cu_tokens, tree_bits, o, lse};
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
                        {cu_tokens, (B + 1) * 4},
                        {tree_bits, (size_t)cfg->max_tokens * words * 4}};
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
                                        block_table, seq_lens, cu_tokens, tree_bits, words,
                                        static_cast<__nv_bfloat16*>(o), lse,
                                        static_cast<uint8_t*>(ws) + kHeader));
}

// Both evictions; pos_pages and next_pos NULL: the first and last tokens by place.
dsa_status_t evict(const dsa_serve_config_t* cfg, const float* w_pages, const float* rank_pages,
                   int32_t* pos_pages, const int32_t* next_pos, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* keep_lens, int64_t n_first,
                   int64_t n_last, void* k_pages, void* v_pages, float* w_out, void* ws,
                   size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_EVICT);
  if (st != DSA_OK) return st;
  if (!w_pages || !block_table || !seq_lens || !keep_lens || n_first < 0 || n_last < 0 ||
      !k_pages || !w_out || v_pages == k_pages)  // K = V: v_pages null
    return DSA_ERR_INVALID_ARG;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_EVICT, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {w_pages,  rank_pages, pos_pages, next_pos, block_table,
                        seq_lens, keep_lens,  k_pages,   v_pages,  w_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch, slots = (size_t)cfg->n_pages * cfg->page_size;
  const size_t cache = slots * cfg->d_qk * 2;
  if (rank_pages == w_pages) rank_pages = nullptr;
  const Span reads[] = {{w_pages == w_out ? nullptr : w_pages, slots * 4},
                        {rank_pages, slots * 4},
                        {next_pos, B * 4},
                        {block_table, B * (size_t)cfg->max_blocks * 4},
                        {seq_lens, B * 4},
                        {keep_lens, B * 4}};
  const Span writes[] = {{k_pages, cache},
                         {v_pages, cache},
                         {pos_pages, slots * 4},
                         {w_out, slots * 4},
                         {ws, serve_ws_bytes(cfg, DSA_SERVE_WS_EVICT)}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  return cuda_status(launch_evict(
      ctx, serve_shape(cfg), w_pages, rank_pages ? rank_pages : w_pages, pos_pages, next_pos,
      block_table, seq_lens, keep_lens, n_first, n_last, static_cast<__nv_bfloat16*>(k_pages),
      static_cast<__nv_bfloat16*>(v_pages), w_out, static_cast<uint8_t*>(ws)));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status_t dsa_serve_workspace_size(const dsa_serve_config_t* cfg, int32_t which,
                                      size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  if ((which < DSA_SERVE_WS_TABLES || which > DSA_SERVE_WS_PREFIX) &&
      (which < DSA_SERVE_WS_TREE || which > DSA_SERVE_WS_EVICT))
    return DSA_ERR_INVALID_ARG;
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
  return attend(cfg, q, k_pages, v_pages, prefix_table, prefix_len, block_table, seq_lens,
                cu_tokens, nullptr, 0, o, lse, ws, ws_bytes, stream);
}

dsa_status_t dsa_tree_attn(const dsa_serve_config_t* cfg, const void* q, const void* k_pages,
                           const void* v_pages, const int32_t* prefix_table,
                           int64_t prefix_len, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* cu_tokens,
                           const uint32_t* tree_bits, int32_t words, void* o, float* lse,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!tree_bits || words < 1 || words > kMaxWords) return DSA_ERR_INVALID_ARG;
  return attend(cfg, q, k_pages, v_pages, prefix_table, prefix_len, block_table, seq_lens,
                cu_tokens, tree_bits, words, o, lse, ws, ws_bytes, stream);
}

dsa_status_t dsa_build_tree(const dsa_serve_config_t* cfg, const int32_t* parents,
                            const int32_t* cu_tokens, int32_t words, uint32_t* tree_bits,
                            void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_TREE);
  if (st != DSA_OK) return st;
  if (!parents || !cu_tokens || !tree_bits || words < 1 || words > kMaxWords)
    return DSA_ERR_INVALID_ARG;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_TREE, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {parents, cu_tokens, tree_bits};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch, T = (size_t)cfg->max_tokens;
  const Span reads[] = {{parents, T * 4}, {cu_tokens, (B + 1) * 4}};
  const Span writes[] = {{tree_bits, T * words * 4}, {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  return cuda_status(
      launch_build_tree(ctx, serve_shape(cfg), parents, cu_tokens, words, tree_bits));
}

dsa_status_t dsa_key_weights(const dsa_serve_config_t* cfg, const void* q, const float* lse,
                             const void* k_pages, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* cu_tokens,
                             const uint32_t* tree_bits, int32_t words, const float* w_pages,
                             float decay, float* w_out, void* ws, size_t ws_bytes,
                             void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_WEIGHTS);
  if (st != DSA_OK) return st;
  if (!q || !lse || !k_pages || !block_table || !seq_lens || !cu_tokens || !w_pages ||
      !w_out || !(decay >= 0.f && decay <= 1.f) ||
      (tree_bits && (words < 1 || words > kMaxWords)))
    return DSA_ERR_INVALID_ARG;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_WEIGHTS, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {q,         lse,       k_pages, block_table, seq_lens,
                        cu_tokens, tree_bits, w_pages, w_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch, slots = (size_t)cfg->n_pages * cfg->page_size;
  const size_t rows = (size_t)cfg->max_tokens * cfg->attn_heads, row = (size_t)cfg->d_qk * 2;
  const Span reads[] = {{q, rows * row},
                        {lse, rows * 4},
                        {k_pages, slots * row},
                        {block_table, B * (size_t)cfg->max_blocks * 4},
                        {seq_lens, B * 4},
                        {cu_tokens, (B + 1) * 4},
                        {tree_bits, tree_bits ? (size_t)cfg->max_tokens * words * 4 : 0},
                        {w_pages == w_out ? nullptr : w_pages, slots * 4}};
  const Span writes[] = {{w_out, slots * 4}, {ws, serve_ws_bytes(cfg, DSA_SERVE_WS_WEIGHTS)}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  const ServeShape sh = serve_shape(cfg);
  CUtensorMap qm[3], km;
  const uint64_t d = (uint64_t)sh.D;
  for (int i = 0; i < 3; ++i)
    if ((st = encode_2d(&qm[i], q, (uint64_t)rows, d, 32u << i)) != DSA_OK) return st;
  if ((st = encode_2d(&km, k_pages, (uint64_t)slots, d, (uint32_t)sh.page)) != DSA_OK) return st;
  return cuda_status(launch_key_weights(ctx, sh, qm, km, lse, block_table, seq_lens, cu_tokens,
                                        tree_bits, words, w_pages, decay, w_out,
                                        static_cast<uint8_t*>(ws)));
}

dsa_status_t dsa_evict_cache(const dsa_serve_config_t* cfg, const float* w_pages,
                             const float* rank_pages, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* keep_lens, int64_t n_first,
                             int64_t n_last, void* k_pages, void* v_pages, float* w_out,
                             void* ws, size_t ws_bytes, void* stream) {
  return evict(cfg, w_pages, rank_pages, nullptr, nullptr, block_table, seq_lens, keep_lens,
               n_first, n_last, k_pages, v_pages, w_out, ws, ws_bytes, stream);
}

dsa_status_t dsa_evict_cache_aged(const dsa_serve_config_t* cfg, const float* w_pages,
                                  const float* rank_pages, int32_t* pos_pages,
                                  const int32_t* next_pos, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* keep_lens,
                                  int64_t n_first, int64_t n_last, void* k_pages,
                                  void* v_pages, float* w_out, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (!pos_pages || !next_pos) return DSA_ERR_INVALID_ARG;
  return evict(cfg, w_pages, rank_pages, pos_pages, next_pos, block_table, seq_lens, keep_lens,
               n_first, n_last, k_pages, v_pages, w_out, ws, ws_bytes, stream);
}

dsa_status_t dsa_release_pages(const dsa_serve_config_t* cfg, const int32_t* seq_lens,
                               const int32_t* keep_lens, const int32_t* block_table,
                               int32_t* new_lens, int32_t* pages, int64_t n_max,
                               int32_t* n_released, void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t st = check_serve(cfg, DSA_SERVE_WS_TABLES);
  if (st != DSA_OK) return st;
  if (!seq_lens || !keep_lens || !block_table || !new_lens || n_max < 0 ||
      (n_max > 0 && !pages) || !n_released)
    return DSA_ERR_INVALID_ARG;
  if ((st = check_serve_ws(cfg, DSA_SERVE_WS_TABLES, ws, ws_bytes)) != DSA_OK) return st;
  const void* ptrs[] = {seq_lens, keep_lens, block_table, new_lens, n_released};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DSA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(pages) & 3u) != 0) return DSA_ERR_MISALIGNED;
  const size_t B = (size_t)cfg->batch;
  const size_t list = n_max < (int64_t)1 << 40 ? n_max : (int64_t)1 << 40;
  const Span reads[] = {{seq_lens, B * 4},
                        {keep_lens, B * 4},
                        {block_table, B * (size_t)cfg->max_blocks * 4}};
  const Span writes[] = {{new_lens, B * 4}, {pages, list * 4}, {n_released, 4}, {ws, kHeader}};
  if (written_meets(writes, reads)) return DSA_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if ((st = make_ctx(ws, stream, &ctx)) != DSA_OK) return st;
  return cuda_status(launch_release_pages(ctx, serve_shape(cfg), seq_lens, keep_lens,
                                          block_table, new_lens, pages, n_max, n_released));
}

}  // extern "C"
