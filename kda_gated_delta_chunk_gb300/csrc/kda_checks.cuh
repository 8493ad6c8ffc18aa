// Argument checks shared by the C entry points of the layer operators.
#pragma once

#include <cstdint>

#include "kda_attn.cuh"

namespace kda {
namespace checks {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether two arrays of na and nb int32 have bytes in common.
inline bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + 4 * (uintptr_t)nb && y < x + 4 * (uintptr_t)na;
}

inline bool known_dtype(int d) { return d == KDA_STATE_F32 || d == KDA_STATE_BF16; }

// KDA_OK on a supported current device; its multiprocessor count in *sms.
inline int current_device(int* sms) {
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

inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  cudaGetLastError();
  return KDA_ERR_LAUNCH_FAILED;
}

// The cache's own fields, and its view for the kernels.
inline int check_cache(const kda_kv_cache* c, int32_t num_seqs, kda::attn::CacheView* out) {
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

inline int check_batch(const int32_t* cu_seqlens, const void* workspace, int64_t total_tokens,
                int32_t num_seqs, int32_t heads, size_t workspace_bytes) {
  if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0 || heads < 1 || !cu_seqlens ||
      !workspace)
    return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(cu_seqlens, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

// A [T, heads, 128] bf16 tensor with dense heads and a token stride.
inline int check_rows(const void* p, int64_t stride, int32_t heads) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (stride < (int64_t)heads * KDA_HEAD_DIM || stride > ((int64_t)1 << 40)) return KDA_ERR_INVALID_ARG;
  if (!aligned(p, 16) || stride % 8 != 0) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

}  // namespace checks
}  // namespace kda
