// Attention over the paged e4m3 cache, first form: one warp per (token, query head).
//   s_j = scale * k_scale(page) * (q . k8_j), optionally cap * tanh(s_j / cap)
//   out = sum_j softmax(s)_j * v_scale(page) * v8_j over max(0, p - window + 1) <= j <= p
// with a running maximum and sum, all in fp32.  Four channels a lane.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

__global__ void __launch_bounds__(128) kda_attn_kernel(const __grid_constant__ AttnParams p, int min_rows) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int32_t* cu = p.cu_seqlens;
  const int N = p.num_seqs;
  if (cu[0] != 0 || (int64_t)cu[N] > p.total_tokens) {
    if (threadIdx.x == 0) record_error(p.status, KDA_ERR_BAD_CU_SEQLENS, 300);
    return;
  }
  const int64_t t = w / p.heads;
  if (t >= (int64_t)cu[N]) return;
  const int h = (int)(w % p.heads), hk = h / (p.heads / p.c.kv_heads);
  const int n = seq_of(cu, N, t);
  const int len = p.c.kv_lens[n];
  if (cu[n + 1] - cu[n] > p.max_q_len) {
    if (lane == 0) record_error(p.status, KDA_ERR_INVALID_ARG, 303);
    return;
  }
  if ((cu[n + 1] - cu[n]) * (p.heads / p.c.kv_heads) < min_rows) return;
  const int pos = len - (int)(cu[n + 1] - t);
  const int P = p.c.page_size;
  if (len < 0 || (int64_t)len > (int64_t)p.c.max_blocks * P) {
    if (lane == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 301);
    return;
  }
  const uint2 qu = *reinterpret_cast<const uint2*>(p.q + t * p.q_stride + h * kHeadDim + 4 * lane);
  const float q0 = __uint_as_float(qu.x << 16), q1 = __uint_as_float(qu.x & 0xffff0000u);
  const float q2 = __uint_as_float(qu.y << 16), q3 = __uint_as_float(qu.y & 0xffff0000u);
  float m = -INFINITY, l = 0.0f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  for (int j = lo; j <= pos; ++j) {
    const int page = p.c.block_table[n * p.c.table_stride + j / P];
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 302);
      return;
    }
    const int64_t at = page * p.c.page_stride + hk * p.c.head_stride + (j % P) * p.c.token_stride + 4 * lane;
    const uint32_t ku = *reinterpret_cast<const uint32_t*>(p.c.k + at);
    const float2 ka = from_e4m3x2(ku & 0xffff), kb = from_e4m3x2(ku >> 16);
    float s = q0 * ka.x + q1 * ka.y + q2 * kb.x + q3 * kb.y;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale * p.c.k_scale[page * p.c.scale_stride + hk];
    if (p.softcap > 0.0f) s = p.softcap * tanhf(s / p.softcap);
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), e = expf(s - mn);
    m = mn;
    l = l * f + e;
    const uint32_t vu = *reinterpret_cast<const uint32_t*>(p.c.v + at);
    const float2 va = from_e4m3x2(vu & 0xffff), vb = from_e4m3x2(vu >> 16);
    const float ev = e * p.c.v_scale[page * p.c.scale_stride + hk];
    o[0] = o[0] * f + ev * va.x;
    o[1] = o[1] * f + ev * va.y;
    o[2] = o[2] * f + ev * vb.x;
    o[3] = o[3] * f + ev * vb.y;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // no key seen: a row of zeros
  __nv_bfloat16* out = p.out + t * p.out_stride + h * kHeadDim + 4 * lane;
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
  *reinterpret_cast<__nv_bfloat162*>(out + 2) = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  if (p.lse && lane == 0) p.lse[t * p.heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_workspace_bytes(int32_t, int32_t, int32_t, int32_t) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    sms = kDefaultSmCount;
  }
  return (size_t)kWorkspaceBytes + decode_workspace_bytes(sms);
}

cudaError_t launch_attn(const AttnParams& p, int sms, cudaStream_t stream) {
  const int group = p.heads / p.c.kv_heads;
  const int64_t rows = (int64_t)p.max_q_len * group;
  const int decode_rows = group <= 32 ? (int)(rows < 32 ? rows : 32) : 0;
  if (decode_rows > 0) {
    cudaError_t e = launch_attn_decode(p, 1, decode_rows, reinterpret_cast<char*>(p.status) + kWorkspaceBytes,
                                       sms, stream);
    if (e != cudaSuccess) return e;
  }
  if (rows > decode_rows) {
    const int64_t grid = (p.total_tokens * p.heads + 3) / 4;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    kda_attn_kernel<<<(unsigned)grid, 128, 0, stream>>>(p, decode_rows + 1);
  }
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
