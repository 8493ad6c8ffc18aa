// C entry points of the full-attention layer's operators: argument checks and dispatch.
// Declared in include/kda.h.
#include <cmath>
#include <cstdint>

#include "kda_attn.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool known_dtype(int d) { return d == KDA_STATE_F32 || d == KDA_STATE_BF16; }

// KDA_OK on a supported current device; its multiprocessor count in *sms.
int current_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return KDA_ERR_CUDA;
  }
  const int rc = kda_device_check(dev);
  if (rc != KDA_OK) return rc;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KDA_ERR_CUDA;
  }
  return KDA_OK;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  cudaGetLastError();
  return KDA_ERR_LAUNCH_FAILED;
}

// The cache's own fields, and its view for the kernels.
int check_cache(const kda_kv_cache* c, int32_t num_seqs, kda::attn::CacheView* out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return KDA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!c->block_table || !c->kv_lens)) return KDA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return KDA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->max_blocks < 0 || c->table_stride < c->max_blocks ||
      c->scale_stride < c->kv_heads)
    return KDA_ERR_INVALID_ARG;
  if ((int64_t)c->max_blocks * c->page_size > INT32_MAX) return KDA_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 39;   // a TMA stride is below 2^40 bytes
  if (c->token_stride < KDA_HEAD_DIM || c->token_stride > most || c->head_stride < KDA_HEAD_DIM ||
      c->head_stride > most || c->page_stride < KDA_HEAD_DIM || c->page_stride > most)
    return KDA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4) || !aligned(c->kv_lens, 4) ||
      (c->token_stride | c->head_stride | c->page_stride) % 16 != 0)
    return KDA_ERR_MISALIGNED;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->page_stride = c->page_stride;
  out->head_stride = c->head_stride;
  out->token_stride = c->token_stride;
  out->scale_stride = c->scale_stride;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->kv_heads = c->kv_heads;
  out->block_table = c->block_table;
  out->table_stride = c->table_stride;
  out->max_blocks = c->max_blocks;
  out->kv_lens = c->kv_lens;
  return KDA_OK;
}

int check_batch(const int32_t* cu_seqlens, const void* workspace, int64_t total_tokens,
                int32_t num_seqs, int32_t heads, size_t workspace_bytes) {
  if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0 || heads < 1 || !cu_seqlens ||
      !workspace)
    return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(cu_seqlens, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

// A [T, heads, 128] bf16 tensor with dense heads and a token stride.
int check_rows(const void* p, int64_t stride, int32_t heads) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (stride < (int64_t)heads * KDA_HEAD_DIM || stride > ((int64_t)1 << 40)) return KDA_ERR_INVALID_ARG;
  if (!aligned(p, 16) || stride % 8 != 0) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                     int residual_dtype, const void* weight, int weight_dtype, float eps,
                     void* residual_out, int64_t lds, void* y, int64_t ldy, void* y8, int64_t ldy8,
                     float* y_scale, int32_t group, int64_t rows, int32_t cols,
                     kda_stream_t stream) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > 32768) return KDA_ERR_INVALID_ARG;
  if (group != 0 && group != 128) return KDA_ERR_INVALID_ARG;
  if (!known_dtype(weight_dtype) || (residual && !known_dtype(residual_dtype))) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.0f) return KDA_ERR_INVALID_ARG;
  if (rows > 0) {   // an empty tensor has no address
    if (!x || !weight || (!y && !y8) || (y8 == nullptr) != (y_scale == nullptr)) return KDA_ERR_INVALID_ARG;
    if (residual && !residual_out) return KDA_ERR_INVALID_ARG;
  }
  if (ldx < cols || (residual && (ldr < cols || lds < cols)) || (y && ldy < cols) || (y8 && ldy8 < cols))
    return KDA_ERR_INVALID_ARG;
  const bool rf = residual && residual_dtype == KDA_STATE_F32, wf = weight_dtype == KDA_STATE_F32;
  if (!aligned(x, 2) || !aligned(residual, rf ? 4 : 2) || !aligned(residual_out, rf ? 4 : 2) ||
      !aligned(weight, wf ? 4 : 2) || !aligned(y, 2) || !aligned(y_scale, 4))
    return KDA_ERR_MISALIGNED;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (rows == 0) return KDA_OK;
  const int re = rf ? 4 : 8;   // residual elements in 16 bytes
  const bool wide = cols % 8 == 0 && aligned(x, 16) && ldx % 8 == 0 && aligned(weight, 16) &&
                    (!residual || (aligned(residual, 16) && aligned(residual_out, 16) &&
                                   ldr % re == 0 && lds % re == 0)) &&
                    (!y || (aligned(y, 16) && ldy % 8 == 0)) &&
                    (!y8 || (aligned(y8, 8) && ldy8 % 8 == 0));
  kda::attn::NormParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = residual;
  p.weight = weight;
  p.residual_out = residual_out;
  p.y = static_cast<__nv_bfloat16*>(y);
  p.y8 = static_cast<uint8_t*>(y8);
  p.y_scale = y_scale;
  p.ldx = ldx;
  p.ldr = ldr;
  p.lds = lds;
  p.ldy = ldy;
  p.ldy8 = ldy8;
  p.rows = rows;
  p.cols = cols;
  p.group = group;
  p.residual_f32 = rf;
  p.weight_f32 = wf;
  p.eps = eps;
  return launched(kda::attn::launch_norm(p, wide, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const void* v, int64_t v_stride, const float* rope, int64_t rope_rows,
                    int32_t rot_dim, int32_t interleaved, const int32_t* positions, void* q_out,
                    int64_t q_out_stride, const kda_kv_cache* cache, const int32_t* cu_seqlens,
                    void* workspace, kda_stream_t stream, int64_t total_tokens, int32_t num_seqs,
                    int32_t heads, size_t workspace_bytes) {
  kda::attn::AppendParams p{};
  int rc = check_batch(cu_seqlens, workspace, total_tokens, num_seqs, heads, workspace_bytes);
  if (rc != KDA_OK) return rc;
  rc = check_cache(cache, num_seqs, &p.c);
  if (rc != KDA_OK) return rc;
  if (rot_dim < 0 || rot_dim > KDA_HEAD_DIM || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1))
    return KDA_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!rope || rope_rows < 1)) return KDA_ERR_INVALID_ARG;
  if (rot_dim > 0 && !aligned(rope, 16)) return KDA_ERR_MISALIGNED;
  if (!aligned(positions, 4)) return KDA_ERR_MISALIGNED;
  if (total_tokens > 0) {
    if ((rc = check_rows(k, k_stride, cache->kv_heads)) != KDA_OK) return rc;
    if ((rc = check_rows(v, v_stride, cache->kv_heads)) != KDA_OK) return rc;
    if (q && ((rc = check_rows(q, q_stride, heads)) != KDA_OK ||
              (rc = check_rows(q_out, q_out_stride, heads)) != KDA_OK))
      return rc;
  }
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.qo_stride = q_out_stride;
  p.rope = rope;
  p.rope_rows = rope_rows;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved;
  p.positions = positions;
  p.cu_seqlens = cu_seqlens;
  p.total_tokens = total_tokens;
  p.num_seqs = num_seqs;
  p.heads = heads;
  p.status = static_cast<int*>(workspace);
  return launched(kda::attn::launch_append(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_attention_workspace_size(int32_t num_seqs, int32_t heads, int32_t kv_heads,
                                    int32_t max_q_len) {
  if (num_seqs < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 ||
      heads / kv_heads > 256 || max_q_len < 0)
    return 0;
  return (kda::attn::attn_workspace_bytes(heads, max_q_len) + 15) & ~(size_t)15;
}

int kda_cached_attention(const void* q, int64_t q_stride, const kda_kv_cache* cache,
                         const int32_t* cu_seqlens, float scale, float softcap, int32_t window,
                         void* out, int64_t out_stride, float* lse, void* workspace,
                         kda_stream_t stream, int64_t total_tokens, int32_t num_seqs, int32_t heads,
                         int32_t max_q_len, size_t workspace_bytes) {
  kda::attn::AttnParams p{};
  int rc = check_batch(cu_seqlens, workspace, total_tokens, num_seqs, heads, workspace_bytes);
  if (rc != KDA_OK) return rc;
  rc = check_cache(cache, num_seqs, &p.c);
  if (rc != KDA_OK) return rc;
  if (heads % cache->kv_heads != 0 || heads / cache->kv_heads > 256 || max_q_len < 0 || window < 0)
    return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.0f) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    if ((rc = check_rows(q, q_stride, heads)) != KDA_OK) return rc;
    if ((rc = check_rows(out, out_stride, heads)) != KDA_OK) return rc;
    if (max_q_len < 1) return KDA_ERR_INVALID_ARG;
  }
  if (!aligned(lse, 4)) return KDA_ERR_MISALIGNED;
  if (workspace_bytes < kda::attn::attn_call_bytes(heads, cache->kv_heads, max_q_len))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.cu_seqlens = cu_seqlens;
  p.scale = scale;
  // (a cap below 2^-100 differs from that by less than a score's precision; its reciprocal would overflow)
  p.softcap = softcap > 0.0f ? fmaxf(softcap, 0x1p-100f) : 0.0f;
  // (a window as long as the longest sequence that the table holds hides nothing)
  p.window = window < (int64_t)cache->max_blocks * cache->page_size ? window : 0;
  p.total_tokens = total_tokens;
  p.num_seqs = num_seqs;
  p.heads = heads;
  p.max_q_len = max_q_len;
  p.status = static_cast<int*>(workspace);
  return launched(kda::attn::launch_attn(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
