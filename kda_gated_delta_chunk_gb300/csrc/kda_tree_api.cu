// C entry points of the operators on drafted trees and on the cache's pages: argument checks and dispatch.  Declared in
// include/kda.h.
#include <cmath>

#include "kda_checks.cuh"
#include "kda_pages.cuh"
#include "kda_tree.cuh"

using namespace kda::checks;

namespace {

// What every call on trees is checked for.
int check_trees(const void* cu_seqlens, const void* parents, const void* workspace, int64_t total_tokens,
                int32_t num_seqs, int32_t max_q_len, size_t workspace_bytes) {
  if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0 || !cu_seqlens || !workspace)
    return KDA_ERR_INVALID_ARG;
  if (max_q_len < 0 || max_q_len > KDA_TREE_NODES) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!parents || max_q_len < 1)) return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(cu_seqlens, 4) || !aligned(parents, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

// What the recurrence and its commit have in common.  Nodes' tensors are checked where there are any.
int check_recur(const void* k, int64_t k_stride, const void* g, int64_t g_stride, const float* A_log,
                const float* dt_bias, float lower_bound, const void* initial_state, int state_dtype,
                const float* u, int64_t total_tokens, int32_t num_seqs, int32_t heads,
                kda::tree::RecurParams* p) {
  // (a row's stride times the nodes of a block has 32 bits)
  if (heads < 1 || heads > 1 << 20 || (int64_t)num_seqs * heads > INT32_MAX / 2 || !known_dtype(state_dtype) || !A_log || !dt_bias)
    return KDA_ERR_INVALID_ARG;
  if (!(lower_bound >= KDA_MIN_LOWER_BOUND && lower_bound <= 0.0f)) return KDA_ERR_UNSAFE_LOWER_BOUND;
  if (!aligned(A_log, 4) || !aligned(dt_bias, 16) || !aligned(initial_state, 16)) return KDA_ERR_MISALIGNED;
  if (total_tokens > 0) {
    int rc;
    if ((rc = check_rows(k, k_stride, heads)) != KDA_OK) return rc;
    if ((rc = check_rows(g, g_stride, heads)) != KDA_OK) return rc;
    if (!u) return KDA_ERR_INVALID_ARG;
    if (!aligned(u, 16)) return KDA_ERR_MISALIGNED;
  }
  p->k = static_cast<const __nv_bfloat16*>(k);
  p->g = static_cast<const __nv_bfloat16*>(g);
  p->s_k = k_stride;
  p->s_g = g_stride;
  p->A_log = A_log;
  p->dt_bias = dt_bias;
  p->lower_bound = lower_bound;
  p->initial_state = initial_state;
  p->state_bf16 = state_dtype == KDA_STATE_BF16;
  p->u = const_cast<float*>(u);
  p->total_tokens = total_tokens;
  p->num_seqs = num_seqs;
  p->heads = heads;
  return KDA_OK;
}

// The pool's own fields.
int check_pool(int32_t* refs, int32_t num_pages, int32_t* block_table, int64_t table_stride, int32_t num_rows,
               int32_t max_blocks, int32_t* kv_lens, int32_t page_size, void* workspace, size_t workspace_bytes,
               kda::pages::Pool* p) {
  if (!refs || !workspace || num_pages < 1 || num_rows < 0 || max_blocks < 0 || table_stride < max_blocks ||
      table_stride > ((int64_t)1 << 40) || page_size < 1 || (int64_t)max_blocks * page_size > INT32_MAX)
    return KDA_ERR_INVALID_ARG;
  if (num_rows > 0 && (!kv_lens || (!block_table && max_blocks > 0))) return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(refs, 16) || !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 16))
    return KDA_ERR_MISALIGNED;
  p->refs = refs;
  p->table = block_table;
  p->table_stride = table_stride;
  p->kv_lens = kv_lens;
  p->status = static_cast<int*>(workspace);
  p->num_pages = num_pages;
  p->page_size = page_size;
  p->num_rows = num_rows;
  p->max_blocks = max_blocks;
  return KDA_OK;
}
// Whether a list shares bytes with what a call on the pool changes.
bool over_pool(const int32_t* list, int64_t n, const kda::pages::Pool& p) {
  const int64_t table = p.num_rows > 0 ? (int64_t)((uint64_t)(p.num_rows - 1) * (uint64_t)p.table_stride) + p.max_blocks : 0;
  return overlap(list, n, p.refs, p.num_pages) || overlap(list, n, p.table, table) ||
         overlap(list, n, p.kv_lens, p.num_rows);
}

}  // namespace

extern "C" {

int kda_tree_plan(const int32_t* parents, const int32_t* cu_seqlens, const int32_t* kv_lens,
                  void* mask, int32_t* positions, void* workspace, kda_stream_t stream,
                  int64_t total_tokens, int32_t num_seqs, int32_t max_q_len, size_t workspace_bytes) {
  int rc = check_trees(cu_seqlens, parents, workspace, total_tokens, num_seqs, max_q_len, workspace_bytes);
  if (rc != KDA_OK) return rc;
  if (num_seqs > 0 && !kv_lens) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!mask || !positions)) return KDA_ERR_INVALID_ARG;
  if (!aligned(kv_lens, 4) || !aligned(mask, 8) || !aligned(positions, 4)) return KDA_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
  kda::tree::PlanParams p{};
  p.parents = parents;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = kv_lens;
  p.mask = static_cast<uint64_t*>(mask);
  p.positions = positions;
  p.status = static_cast<int*>(workspace);
  p.total_tokens = total_tokens;
  p.num_seqs = num_seqs;
  p.max_q_len = max_q_len;
  return launched(kda::tree::launch_plan(p, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_tree_recurrent_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const void* g, int64_t g_stride, const void* beta,
                           int64_t beta_stride, const float* A_log, const float* dt_bias, float lower_bound,
                           float scale, const void* initial_state, int state_dtype,
                           const int32_t* cu_seqlens, const int32_t* parents, void* out, float* u,
                           void* workspace, kda_stream_t stream, int64_t total_tokens, int32_t num_seqs,
                           int32_t heads, int32_t max_q_len, size_t workspace_bytes) {
  kda::tree::RecurParams p{};
  int rc = check_trees(cu_seqlens, parents, workspace, total_tokens, num_seqs, max_q_len, workspace_bytes);
  if (rc != KDA_OK) return rc;
  rc = check_recur(k, k_stride, g, g_stride, A_log, dt_bias, lower_bound, initial_state, state_dtype, u,
                   total_tokens, num_seqs, heads, &p);
  if (rc != KDA_OK) return rc;
  if (!std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    if ((rc = check_rows(q, q_stride, heads)) != KDA_OK) return rc;
    if ((rc = check_rows(v, v_stride, heads)) != KDA_OK) return rc;
    if (!beta || beta_stride < heads || beta_stride > ((int64_t)1 << 40) || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(beta, 2) || !aligned(out, 16)) return KDA_ERR_MISALIGNED;
  }
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.beta = static_cast<const __nv_bfloat16*>(beta);
  p.s_q = q_stride;
  p.s_v = v_stride;
  p.s_beta = beta_stride;
  p.scale = scale;
  p.cu_seqlens = cu_seqlens;
  p.parents = parents;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = static_cast<int*>(workspace);
  p.max_q_len = max_q_len;
  return launched(kda::tree::launch_recur(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_tree_commit(const void* k, int64_t k_stride, const void* g, int64_t g_stride, const float* A_log,
                    const float* dt_bias, float lower_bound, const void* initial_state, void* final_state,
                    int state_dtype, const int32_t* cu_seqlens, const int32_t* parents, const float* u,
                    const int32_t* accepted, void* workspace, kda_stream_t stream, int64_t total_tokens,
                    int32_t num_seqs, int32_t heads, int32_t max_q_len, size_t workspace_bytes) {
  kda::tree::RecurParams p{};
  int rc = check_trees(cu_seqlens, parents, workspace, total_tokens, num_seqs, max_q_len, workspace_bytes);
  if (rc != KDA_OK) return rc;
  rc = check_recur(k, k_stride, g, g_stride, A_log, dt_bias, lower_bound, initial_state, state_dtype, u,
                   total_tokens, num_seqs, heads, &p);
  if (rc != KDA_OK) return rc;
  if (num_seqs > 0 && (!accepted || !final_state)) return KDA_ERR_INVALID_ARG;
  if (!aligned(accepted, 4) || !aligned(final_state, 16)) return KDA_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0) return KDA_OK;
  p.final_state = final_state;
  p.cu_seqlens = cu_seqlens;
  p.parents = parents;
  p.accepted = accepted;
  p.status = static_cast<int*>(workspace);
  p.max_q_len = max_q_len;
  return launched(kda::tree::launch_commit(p, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_cache_accept(const kda_kv_cache* cache, const int32_t* cu_seqlens, const int32_t* parents,
                     const int32_t* accepted, int32_t* lens_out, void* workspace, kda_stream_t stream,
                     int64_t total_tokens, int32_t num_seqs, int32_t max_q_len, size_t workspace_bytes) {
  kda::tree::AcceptParams p{};
  int rc = check_trees(cu_seqlens, parents, workspace, total_tokens, num_seqs, max_q_len, workspace_bytes);
  if (rc != KDA_OK) return rc;
  if ((rc = check_cache(cache, num_seqs, &p.c)) != KDA_OK) return rc;
  if (num_seqs > 0 && (!accepted || !lens_out)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)num_seqs * cache->kv_heads * 2 > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (!aligned(accepted, 4) || !aligned(lens_out, 4)) return KDA_ERR_MISALIGNED;
  // (every head's CTAs, and other sequences', read what one of them would write)
  const int64_t table = num_seqs > 0 ? (int64_t)((uint64_t)(num_seqs - 1) * (uint64_t)cache->table_stride) + cache->max_blocks : 0;
  if (overlap(lens_out, num_seqs, cache->kv_lens, num_seqs) || overlap(lens_out, num_seqs, accepted, num_seqs) ||
      overlap(lens_out, num_seqs, cu_seqlens, (int64_t)num_seqs + 1) ||
      overlap(lens_out, num_seqs, parents, total_tokens) || overlap(lens_out, num_seqs, cache->block_table, table))
    return KDA_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0) return KDA_OK;
  p.cu_seqlens = cu_seqlens;
  p.parents = parents;
  p.accepted = accepted;
  p.lens_out = lens_out;
  p.status = static_cast<int*>(workspace);
  p.total_tokens = total_tokens;
  p.num_seqs = num_seqs;
  p.max_q_len = max_q_len;
  return launched(kda::tree::launch_accept(p, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_pages_free(int32_t* refs, int32_t num_pages, int32_t* block_table, int64_t table_stride,
                   int32_t num_rows, int32_t max_blocks, int32_t* kv_lens, int32_t page_size,
                   const int32_t* rows, int32_t num, void* workspace, size_t workspace_bytes,
                   kda_stream_t stream) {
  kda::pages::Pool p{};
  int rc = check_pool(refs, num_pages, block_table, table_stride, num_rows, max_blocks, kv_lens, page_size,
                      workspace, workspace_bytes, &p);
  if (rc != KDA_OK) return rc;
  if (num < 0) return KDA_ERR_INVALID_ARG;
  if (!aligned(rows, 4)) return KDA_ERR_MISALIGNED;
  if (rows && over_pool(rows, num, p)) return KDA_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_rows == 0 || (rows && num == 0)) return KDA_OK;
  return launched(kda::pages::launch_free(p, rows, num, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_pages_reserve(int32_t* refs, int32_t num_pages, int32_t* block_table, int64_t table_stride,
                      int32_t num_rows, int32_t max_blocks, int32_t* kv_lens, int32_t page_size,
                      const int32_t* new_tokens, void* workspace, size_t workspace_bytes,
                      kda_stream_t stream) {
  kda::pages::Pool p{};
  int rc = check_pool(refs, num_pages, block_table, table_stride, num_rows, max_blocks, kv_lens, page_size,
                      workspace, workspace_bytes, &p);
  if (rc != KDA_OK) return rc;
  // (the requests' sum has 32 bits)
  if (num_rows > kda::pages::kMaxRows || (int64_t)num_rows * max_blocks > INT32_MAX ||
      (num_rows > 0 && !new_tokens))
    return KDA_ERR_INVALID_ARG;
  if (!aligned(new_tokens, 4)) return KDA_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_rows == 0) return KDA_OK;
  return launched(kda::pages::launch_reserve(p, new_tokens, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_pages_fork(int32_t* refs, int32_t num_pages, int32_t* block_table, int64_t table_stride,
                   int32_t num_rows, int32_t max_blocks, int32_t* kv_lens, int32_t page_size,
                   const int32_t* src, const int32_t* dst, int32_t num, int32_t* from_pages,
                   int32_t* to_pages, void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  kda::pages::Pool p{};
  int rc = check_pool(refs, num_pages, block_table, table_stride, num_rows, max_blocks, kv_lens, page_size,
                      workspace, workspace_bytes, &p);
  if (rc != KDA_OK) return rc;
  if (num < 0 || num > kda::pages::kMaxRows || num_rows > kda::pages::kMaxRows) return KDA_ERR_INVALID_ARG;
  if (num > 0 && (!src || !dst || !from_pages || !to_pages)) return KDA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(from_pages, 4) || !aligned(to_pages, 4))
    return KDA_ERR_MISALIGNED;
  // (every pair's CTA reads all of src and dst)
  for (const int32_t* list : {src, dst, const_cast<const int32_t*>(from_pages), const_cast<const int32_t*>(to_pages)})
    if (over_pool(list, num, p)) return KDA_ERR_INVALID_ARG;
  for (const int32_t* out : {from_pages, to_pages})
    if (overlap(out, num, src, num) || overlap(out, num, dst, num)) return KDA_ERR_INVALID_ARG;
  if (overlap(from_pages, num, to_pages, num)) return KDA_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num == 0) return KDA_OK;
  return launched(kda::pages::launch_fork(p, src, dst, num, from_pages, to_pages,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int kda_pages_copy(const kda_kv_cache* cache, const int32_t* from_pages, const int32_t* to_pages, int64_t num,
                   void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  kda::attn::CacheView c{};
  int rc = check_cache(cache, 0, &c);
  if (rc != KDA_OK) return rc;
  if (!workspace || num < 0 || num > INT32_MAX || num * cache->kv_heads * 2 > INT32_MAX ||
      (num > 0 && (!from_pages || !to_pages)))
    return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(from_pages, 4) || !aligned(to_pages, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num == 0) return KDA_OK;
  return launched(kda::pages::launch_copy(c, from_pages, to_pages, num, static_cast<int*>(workspace),
                                          reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
