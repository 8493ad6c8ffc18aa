// Shared by the full-attention layer's operators: the residual norm, the rotary append to a
// paged 8-bit cache, and the attention over that cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace attn {

constexpr float kE4M3Max = 448.0f;

// ------------------------------------------------------------ launches
// A launch, on request as the programmatic dependent of the one before it on the stream (it may
// then start before that one has ended, and waits in the kernel if it must).
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, bool dependent,
                   cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------ e4m3
// Two floats -> two e4m3 bytes (round to nearest even, finite overflow and infinities to
// +-448, NaN to NaN); `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two e4m3 bytes (the low half of `v`) -> two floats, exactly (every e4m3 value is an f16).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------ eight bf16 / fp32 values
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------ norm
struct NormParams {
  const __nv_bfloat16* x;
  const void* residual;      // bf16 or fp32, or null
  const void* weight;        // bf16 or fp32
  void* residual_out;        // the residual's type, or null
  __nv_bfloat16* y;          // or null
  uint8_t* y8;               // or null
  float* y_scale;            // [rows, groups]
  int64_t ldx, ldr, lds, ldy, ldy8;   // row strides (elements); lds of residual_out
  int64_t rows;
  int32_t cols, group;       // group: 0 (one scale per row) or 128
  int32_t residual_f32, weight_f32;
  float eps;
};
cudaError_t launch_norm(const NormParams& p, bool aligned, cudaStream_t stream);

// ------------------------------------------------------------ paged cache
// Mirrors kda_kv_cache of kda.h.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, head_stride, token_stride, scale_stride;
  int32_t num_pages, page_size, kv_heads;
  const int32_t* block_table;
  int64_t table_stride;
  int32_t max_blocks;
  const int32_t* kv_lens;
};

struct AppendParams {
  const __nv_bfloat16* q;    // or null
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  int64_t q_stride, k_stride, v_stride, qo_stride;
  const float* rope;         // [rope_rows, rot_dim]: cosines, then sines; null when rot_dim = 0
  int64_t rope_rows;
  int32_t rot_dim, interleaved;
  const int32_t* positions;  // [total_tokens] or null (the cache positions)
  const int32_t* cu_seqlens;
  CacheView c;
  int64_t total_tokens;
  int32_t num_seqs, heads;
  int* status;
};
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream);

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;                // [total_tokens, heads] or null
  int64_t q_stride, out_stride;
  const int32_t* cu_seqlens;
  CacheView c;
  float scale, softcap;      // softcap 0: none
  int32_t window;            // 0: none
  const uint64_t* tree;      // [total_tokens] masks of a tree's nodes, or null (causal)
  int64_t total_tokens;
  int32_t num_seqs, heads, max_q_len;
  int* status;               // workspace: 256 bytes of status words, then the partial results
};
// What serves any call with at most these sizes, and what one of exactly these uses.
size_t attn_workspace_bytes(int32_t heads, int32_t max_q_len);
size_t attn_call_bytes(int32_t heads, int32_t kv_heads, int32_t max_q_len);
cudaError_t launch_attn(const AttnParams& p, int sms, cudaStream_t stream);

// The sequence that token t belongs to: the last n with cu[n] <= t (cu non-decreasing,
// cu[0] <= t < cu[N]).
__device__ __forceinline__ int seq_of(const int32_t* cu, int num_seqs, int64_t t) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace attn
}  // namespace kda
