// C ABI entry points of the verification over a paged cache: host-side argument
// validation, then kernel launches (as in api.hip).
#include <math.h>

#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether n bytes at p and m bytes at q have one in common.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

// Whether one of the n rows of `row` bytes at p, p + p_step, ... has a byte in common with
// one of those at q, q + q_step, ...; at steps that differ, whether the ranges have.
bool rows_meet(const void* p, int64_t p_step, const void* q, int64_t q_step, int64_t n,
               int64_t row) {
  if (!overlap(p, (size_t)((n - 1) * p_step + row), q, (size_t)((n - 1) * q_step + row)))
    return false;
  if (n == 1 || p_step != q_step) return true;
  // row i of q begins m bytes behind the beginning of row i + k of p
  const int64_t by = (int64_t)(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p));
  const int64_t k = by / p_step - (by % p_step < 0 ? 1 : 0);
  const int64_t m = by - k * p_step;
  return (m < row && -n < k && k < n) || (m + row > p_step && -n < k + 1 && k + 1 < n);
}

bool head_dim_ok(int D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

dspark_status check_pages(const char* who, int page_size, int max_pages, int num_pages) {
  if (max_pages <= 0 || num_pages <= 0)
    return fail(DSPARK_EINVAL, "%s: max_pages and num_pages must be positive", who);
  if (page_shift(page_size) < 0)
    return fail(DSPARK_EINVAL, "%s: page_size must be a power of two in [16, 1024] (got %d)", who,
                page_size);
  return DSPARK_OK;
}

dspark_status check_cache_types(const char* who, int dtype, int cache_dtype, const float* k_scale,
                                const float* v_scale) {
  if (dtype != DSPARK_BF16 && dtype != DSPARK_FP16)
    return fail(DSPARK_EINVAL, "%s: dtype must be DSPARK_BF16 or DSPARK_FP16 (got %d)", who, dtype);
  if (cache_dtype != dtype && cache_dtype != DSPARK_E4M3)
    return fail(DSPARK_EINVAL, "%s: the cache must hold dtype or DSPARK_E4M3 (got %d)", who,
                cache_dtype);
  const bool f8 = cache_dtype == DSPARK_E4M3;
  if (f8 ? (!k_scale || !v_scale) : (k_scale || v_scale))
    return fail(DSPARK_EINVAL, "%s: scales go with a DSPARK_E4M3 cache, and with no other", who);
  return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using dspark::fail;

extern "C" {

dspark_status dspark_page_map(const int32_t* cur_len, const int32_t* cu_seqlens, int R,
                              int max_tokens, int page_size, int max_pages, int num_pages,
                              int32_t* block_table, const int32_t* ring,
                              const dspark_page_pool* pool, dspark_page_pool* pool_out,
                              int64_t* slots, int32_t* new_len, void* stream) {
  dspark::clear_error();
  if (!cur_len || !cu_seqlens || !block_table || !ring || !pool || !pool_out || !slots || !new_len)
    return fail(DSPARK_EINVAL, "page_map: NULL required pointer");
  if (R <= 0 || max_tokens <= 0) return fail(DSPARK_EINVAL, "page_map: sizes must be positive");
  const dspark_status st = dspark::check_pages("page_map", page_size, max_pages, num_pages);
  if (st != DSPARK_OK) return st;
  if (R > DSPARK_MAX_PAGE_REQUESTS)
    return fail(DSPARK_EUNSUPPORTED, "page_map: more than %d requests", DSPARK_MAX_PAGE_REQUESTS);
  const size_t lens = (size_t)R * sizeof(int32_t);
  if (dspark::overlap(pool, sizeof(*pool), pool_out, sizeof(*pool)) ||
      dspark::overlap(new_len, lens, cur_len, lens))
    return fail(DSPARK_EINVAL, "page_map: pool_out and new_len need memory of their own");
  return dspark::launch_page_map(cur_len, cu_seqlens, R, max_tokens, dspark::page_shift(page_size),
                                 max_pages, num_pages, block_table, ring, pool, pool_out, slots,
                                 new_len, reinterpret_cast<hipStream_t>(stream));
}

dspark_status dspark_page_trim(const int32_t* cur_len, const int32_t* keep_len, int R,
                               int page_size, int max_pages, int num_pages,
                               const int32_t* block_table, int32_t* ring,
                               const dspark_page_pool* pool, dspark_page_pool* pool_out,
                               void* stream) {
  dspark::clear_error();
  if (!cur_len || !keep_len || !block_table || !ring || !pool || !pool_out)
    return fail(DSPARK_EINVAL, "page_trim: NULL required pointer");
  if (R <= 0) return fail(DSPARK_EINVAL, "page_trim: R must be positive");
  const dspark_status st = dspark::check_pages("page_trim", page_size, max_pages, num_pages);
  if (st != DSPARK_OK) return st;
  if (dspark::overlap(pool, sizeof(*pool), pool_out, sizeof(*pool)))
    return fail(DSPARK_EINVAL, "page_trim: pool_out needs memory of its own");
  if (R > DSPARK_MAX_PAGE_REQUESTS)
    return fail(DSPARK_EUNSUPPORTED, "page_trim: more than %d requests", DSPARK_MAX_PAGE_REQUESTS);
  return dspark::launch_page_trim(cur_len, keep_len, R, dspark::page_shift(page_size), max_pages,
                                  num_pages, block_table, ring, pool, pool_out,
                                  reinterpret_cast<hipStream_t>(stream));
}

dspark_status dspark_kv_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                              int dtype, const int64_t* slots, const int32_t* count,
                              int max_tokens, int Hk, int D, int page_size, int num_pages,
                              int cache_dtype, const float* k_scale, const float* v_scale,
                              void* k_cache, void* v_cache, void* stream) {
  dspark::clear_error();
  if (!k || !v || !slots || !k_cache || !v_cache)
    return fail(DSPARK_EINVAL, "kv_store: NULL required pointer");
  if (max_tokens <= 0 || Hk <= 0 || D <= 0)
    return fail(DSPARK_EINVAL, "kv_store: sizes must be positive");
  dspark_status st = dspark::check_pages("kv_store", page_size, 1, num_pages);
  if (st != DSPARK_OK) return st;
  st = dspark::check_cache_types("kv_store", dtype, cache_dtype, k_scale, v_scale);
  if (st != DSPARK_OK) return st;
  if (!dspark::head_dim_ok(D) || Hk > 65535)
    return fail(DSPARK_EUNSUPPORTED, "kv_store: D must be 64, 96, 128, 192 or 256 and Hk <= 65535");
  if (k_stride % 8 || v_stride % 8 || k_stride < (int64_t)Hk * D || v_stride < (int64_t)Hk * D ||
      !dspark::aligned(k, 16) || !dspark::aligned(v, 16) || !dspark::aligned(k_cache, 16) ||
      !dspark::aligned(v_cache, 16))
    return fail(DSPARK_EINVAL, "kv_store: rows and caches must be 16-byte aligned, rows at least "
                               "Hk * D apart");
  return dspark::launch_kv_store(k, v, k_stride, v_stride, dtype, slots, count, max_tokens, Hk, D,
                                 dspark::page_shift(page_size), num_pages, cache_dtype, k_scale,
                                 v_scale, k_cache, v_cache, reinterpret_cast<hipStream_t>(stream));
}

dspark_status dspark_kv_commit(void* k_cache, void* v_cache, int64_t k_layer_stride,
                               int64_t v_layer_stride, int layers, int cache_dtype,
                               const int32_t* block_table, const int32_t* ctx_len,
                               const int32_t* path, const int32_t* accepted, int R, int max_nodes,
                               int Hk, int D, int page_size, int max_pages, int num_pages,
                               int32_t* new_len, void* stream) {
  return dspark_kv_commit_ex(k_cache, v_cache, k_layer_stride, v_layer_stride, layers, cache_dtype,
                             block_table, ctx_len, nullptr, path, accepted, R, max_nodes, Hk, D,
                             page_size, max_pages, num_pages, new_len, stream);
}

dspark_status dspark_kv_commit_ex(void* k_cache, void* v_cache, int64_t k_layer_stride,
                                  int64_t v_layer_stride, int layers, int cache_dtype,
                                  const int32_t* block_table, const int32_t* ctx_len,
                                  const int32_t* mapped_len, const int32_t* path,
                                  const int32_t* accepted, int R, int max_nodes, int Hk, int D,
                                  int page_size, int max_pages, int num_pages, int32_t* new_len,
                                  void* stream) {
  dspark::clear_error();
  if (!k_cache || !v_cache || !block_table || !ctx_len || !path || !accepted || !new_len)
    return fail(DSPARK_EINVAL, "kv_commit: NULL required pointer");
  if (R <= 0 || max_nodes <= 0 || Hk <= 0 || D <= 0 || layers <= 0)
    return fail(DSPARK_EINVAL, "kv_commit: sizes must be positive");
  const dspark_status st = dspark::check_pages("kv_commit", page_size, max_pages, num_pages);
  if (st != DSPARK_OK) return st;
  if (cache_dtype != DSPARK_BF16 && cache_dtype != DSPARK_FP16 && cache_dtype != DSPARK_E4M3)
    return fail(DSPARK_EINVAL, "kv_commit: unknown cache type %d", cache_dtype);
  if (!dspark::head_dim_ok(D) || layers > 65535 || R > 65535)
    return fail(DSPARK_EUNSUPPORTED, "kv_commit: D must be 64, 96, 128, 192 or 256, layers and R "
                                     "<= 65535");
  const int el = cache_dtype == DSPARK_E4M3 ? 1 : 2;
  if (!dspark::aligned(k_cache, 16) || !dspark::aligned(v_cache, 16) ||
      (k_layer_stride * el) % 16 || (v_layer_stride * el) % 16)
    return fail(DSPARK_EINVAL, "kv_commit: caches and layers must be 16-byte aligned");
  // a layer's workgroups wait for no other layer's
  const __int128 layer = (__int128)num_pages * page_size * Hk * D;
  const __int128 kl = k_layer_stride, vl = v_layer_stride;
  if (layers > 1 && ((kl < layer && -kl < layer) || (vl < layer && -vl < layer)))
    return fail(DSPARK_EINVAL, "kv_commit: the layers of a cache overlap");
  // every layer's workgroups read the lengths, one of them writes the new ones
  const size_t lens = (size_t)R * sizeof(int32_t);
  if (dspark::overlap(new_len, lens, ctx_len, lens) ||
      dspark::overlap(new_len, lens, accepted, lens) ||
      (mapped_len && dspark::overlap(new_len, lens, mapped_len, lens)))
    return fail(DSPARK_EINVAL, "kv_commit: new_len needs memory of its own");
  return dspark::launch_kv_commit(k_cache, v_cache, k_layer_stride, v_layer_stride, layers, el,
                                  block_table, ctx_len, mapped_len, path, accepted, R, max_nodes,
                                  Hk, D, dspark::page_shift(page_size), max_pages, num_pages,
                                  new_len, reinterpret_cast<hipStream_t>(stream));
}

size_t dspark_tree_attention_workspace(int R, int max_tokens, int Hq, int Hk, int D) {
  if (R <= 0 || max_tokens <= 0 || Hq <= 0 || Hk <= 0 || Hq % Hk || !dspark::head_dim_ok(D))
    return 0;
  if (R > (1 << 20) || (int64_t)max_tokens * Hq > 0x7fffffffLL) return 0;
  return dspark::tree_attention_workspace_bytes(R, max_tokens, Hq, Hk, D);
}

dspark_status dspark_tree_attention(const void* q, int64_t q_stride, int dtype,
                                    const void* k_cache, const void* v_cache, int cache_dtype,
                                    const float* k_scale, const float* v_scale,
                                    const int32_t* block_table, const int32_t* ctx_len,
                                    const int32_t* cu_seqlens, const uint32_t* tree_mask,
                                    int mask_words, int R, int max_tokens, int Hq, int Hk, int D,
                                    int page_size, int max_pages, int num_pages, float scale,
                                    void* out, int64_t out_stride, float* lse, void* workspace,
                                    size_t ws_bytes, void* stream) {
  return dspark_tree_attention_ex(q, q_stride, dtype, k_cache, v_cache, cache_dtype, k_scale,
                                  v_scale, block_table, ctx_len, nullptr, cu_seqlens, tree_mask,
                                  mask_words, R, max_tokens, Hq, Hk, D, page_size, max_pages,
                                  num_pages, scale, out, out_stride, lse, workspace, ws_bytes,
                                  stream);
}

dspark_status dspark_tree_attention_ex(const void* q, int64_t q_stride, int dtype,
                                       const void* k_cache, const void* v_cache, int cache_dtype,
                                       const float* k_scale, const float* v_scale,
                                       const int32_t* block_table, const int32_t* ctx_len,
                                       const int32_t* mapped_len, const int32_t* cu_seqlens,
                                       const uint32_t* tree_mask, int mask_words, int R,
                                       int max_tokens, int Hq, int Hk, int D, int page_size,
                                       int max_pages, int num_pages, float scale, void* out,
                                       int64_t out_stride, float* lse, void* workspace,
                                       size_t ws_bytes, void* stream) {
  dspark::clear_error();
  if (!q || !k_cache || !v_cache || !block_table || !ctx_len || !cu_seqlens || !out)
    return fail(DSPARK_EINVAL, "tree_attention: NULL required pointer");
  if (R <= 0 || max_tokens <= 0 || Hq <= 0 || Hk <= 0 || D <= 0)
    return fail(DSPARK_EINVAL, "tree_attention: sizes must be positive");
  if (Hq % Hk) return fail(DSPARK_EINVAL, "tree_attention: Hq must be a multiple of Hk");
  if (tree_mask ? mask_words <= 0 : mask_words != 0)
    return fail(DSPARK_EINVAL, "tree_attention: mask_words goes with tree_mask");
  const float scale2 = (float)((double)scale * 1.4426950408889634);   // scale log2(e)
  if (!isfinite(scale2)) return fail(DSPARK_EINVAL, "tree_attention: scale must be finite");
  dspark_status st = dspark::check_pages("tree_attention", page_size, max_pages, num_pages);
  if (st != DSPARK_OK) return st;
  st = dspark::check_cache_types("tree_attention", dtype, cache_dtype, k_scale, v_scale);
  if (st != DSPARK_OK) return st;
  const int64_t row = (int64_t)Hq * D;
  if (!dspark::aligned(q, 16) || !dspark::aligned(out, 16) || !dspark::aligned(k_cache, 16) ||
      !dspark::aligned(v_cache, 16) || q_stride % 8 || out_stride % 8 || q_stride < row ||
      out_stride < row)
    return fail(DSPARK_EINVAL, "tree_attention: rows and caches must be 16-byte aligned, rows at "
                               "least Hq * D apart");
  // a row may be written where it was read, but nowhere that another is
  if (!(out == q && (out_stride == q_stride || max_tokens == 1)) &&
      dspark::rows_meet(q, q_stride * 2, out, out_stride * 2, max_tokens, row * 2))
    return fail(DSPARK_EINVAL, "tree_attention: out may be q or apart from it, not a part of it");
  if (!dspark::head_dim_ok(D))
    return fail(DSPARK_EUNSUPPORTED, "tree_attention: D must be 64, 96, 128, 192 or 256 (got %d)", D);
  if (mask_words > DSPARK_MAX_MASK_WORDS)
    return fail(DSPARK_EUNSUPPORTED, "tree_attention: mask rows above %d words", DSPARK_MAX_MASK_WORDS);
  if (R > (1 << 20) || (int64_t)max_tokens * Hq > 0x7fffffffLL)
    return fail(DSPARK_EUNSUPPORTED, "tree_attention: R above 2^20 or max_tokens * Hq above 2^31 - 1");
  const size_t need = dspark::tree_attention_workspace_bytes(R, max_tokens, Hq, Hk, D);
  if (!workspace || ws_bytes < need)
    return fail(DSPARK_EWORKSPACE, "tree_attention: workspace needs %zu bytes (got %zu)", need,
                workspace ? ws_bytes : (size_t)0);
  if (!dspark::aligned(workspace, 256))
    return fail(DSPARK_EINVAL, "tree_attention: workspace must be 256-byte aligned");
  dspark::TreeAttnArgs a;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = block_table;
  a.ctx = ctx_len;
  a.mapped = mapped_len;
  a.cu = cu_seqlens;
  a.mask = tree_mask;
  a.out = out;
  a.lse = lse;
  a.ws = workspace;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.dtype = dtype;
  a.cache_dtype = cache_dtype;
  a.mask_words = mask_words;
  a.R = R;
  a.max_tokens = max_tokens;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = D;
  a.shift = dspark::page_shift(page_size);
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.scale2 = scale2;
  return dspark::launch_tree_attention(a, reinterpret_cast<hipStream_t>(stream));
}

dspark_status dspark_tree_pack(const int32_t* parents, const int32_t* cu_seqlens,
                               const int32_t* pos0, int R, int max_tokens, int mask_words,
                               uint32_t* mask, int32_t* flat_pos, int32_t* flat_req,
                               void* stream) {
  dspark::clear_error();
  if (!parents || !cu_seqlens || !mask)
    return fail(DSPARK_EINVAL, "tree_pack: NULL required pointer");
  if (R <= 0 || max_tokens <= 0 || mask_words <= 0)
    return fail(DSPARK_EINVAL, "tree_pack: sizes must be positive");
  if (mask_words > DSPARK_MAX_MASK_WORDS)
    return fail(DSPARK_EUNSUPPORTED, "tree_pack: mask rows above %d words", DSPARK_MAX_MASK_WORDS);
  return dspark::launch_tree_pack(parents, cu_seqlens, pos0, R, max_tokens, mask_words, mask,
                                  flat_pos, flat_req, reinterpret_cast<hipStream_t>(stream));
}

dspark_status dspark_verify_tree(const float* target_logits, const int32_t* cu_seqlens,
                                 const int32_t* tokens, const int32_t* parents, int R,
                                 int max_tokens, int max_nodes, int V, int32_t* target_argmax,
                                 int32_t* accepted, int32_t* path, int32_t* next_token,
                                 void* stream) {
  return dspark_verify_tree_ex(target_logits, cu_seqlens, tokens, parents, nullptr, nullptr, R,
                               max_tokens, max_nodes, V, target_argmax, accepted, path,
                               next_token, stream);
}

dspark_status dspark_verify_tree_ex(const float* target_logits, const int32_t* cu_seqlens,
                                    const int32_t* tokens, const int32_t* parents,
                                    const int32_t* ctx_len, const int32_t* mapped_len, int R,
                                    int max_tokens, int max_nodes, int V, int32_t* target_argmax,
                                    int32_t* accepted, int32_t* path, int32_t* next_token,
                                    void* stream) {
  dspark::clear_error();
  if (!target_logits || !cu_seqlens || !tokens || !parents || !target_argmax || !accepted ||
      !path || !next_token)
    return fail(DSPARK_EINVAL, "verify_tree: NULL required pointer");
  if (R <= 0 || max_tokens <= 0 || max_nodes <= 0 || V < 1)
    return fail(DSPARK_EINVAL, "verify_tree: sizes must be positive");
  if (!ctx_len != !mapped_len)
    return fail(DSPARK_EINVAL, "verify_tree: ctx_len and mapped_len go together");
  return dspark::launch_verify_tree(target_logits, cu_seqlens, tokens, parents, ctx_len,
                                    mapped_len, R, max_tokens, max_nodes, V, target_argmax,
                                    accepted, path, next_token,
                                    reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
