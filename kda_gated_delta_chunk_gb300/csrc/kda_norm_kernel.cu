// Root-mean-square norm of a sum, with bf16 and / or 8-bit outputs:
//   s = x + r        y = s * (mean_c(s^2) + eps)^(-1/2) * w
// r (bf16 or fp32; absent: s = x) is the residual stream, and s is written back in its type.
// y leaves as bf16 and / or as e4m3 with fp32 scales, one per 128 columns or one per row:
//   scale = max(max|y| / 448, 2^-40)      y8 = e4m3(y / scale)
// The sum, its squares, the norm and the scales are fp32; s enters the norm as the fp32 sum,
// not as it is rounded for the residual stream, so that y is rounded once.  max|y| / 448 puts
// the largest value of a group on the largest e4m3 value; the floor keeps 1 / scale finite
// for a group of zeros.
//
// Bound by memory: one read of x and r, one write of s and y, no reuse.  A row stays in the
// registers of one CTA (kV chunks of 8 columns a thread, 16-byte accesses) between the sum of
// squares and the outputs, so nothing is read twice; rows of at most 256 columns take one warp
// each.  16384 x 7168 in bf16: 150.4 us, 6.25 TB/s; 4096 x 7168 to 8 bits with an fp32 residual:
// 52.0 us, 6.23 TB/s; 14 x 7168 2.4 us.  Groups of 128 columns are 16 adjacent lanes: their maximum is four shuffles.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16, true>(const __nv_bfloat16* p, int, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
template <>
__device__ __forceinline__ void load8<float, true>(const float* p, int, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16, false>(const __nv_bfloat16* p, int n, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
}
template <>
__device__ __forceinline__ void load8<float, false>(const float* p, int n, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
}
template <bool kVec>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, const float (&v)[8]) {
  if (kVec) {
    *reinterpret_cast<uint4*>(p) = pack8(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}
template <bool kVec>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (kVec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <bool kVec>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int n, const float (&v)[8]) {
  const uint32_t a = e4m3x4(v[0], v[1], v[2], v[3]), b = e4m3x4(v[4], v[5], v[6], v[7]);
  if (kVec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? a >> (8 * i) : b >> (8 * (i - 4))) & 0xff);
  }
}

template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? max_nan(a, b) : a + b;
}
// Reduction over the threads of a row: a warp (kWarpRow) or the CTA; every thread gets it.
template <bool kMax, bool kWarpRow>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (kWarpRow) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.0f;   // 0 is neutral: sums of squares and magnitudes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kV: chunks of 8 columns per thread.  kVec: every row starts on 16 bytes (y8: 8) and cols is
// a multiple of 8; else element by element.  kWarpRow: one warp per row, else one CTA per row.
template <typename R, typename Wt, int kV, bool kVec, bool kWarpRow>
__global__ void __launch_bounds__(1024) kda_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2][32];
  sm100::pdl_wait();   // (launched as a programmatic dependent of the work before it)
  sm100::pdl_launch_dependents();
  const int tr = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;   // thread within the row
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int64_t row = kWarpRow ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                               : (int64_t)blockIdx.x;
  if (kWarpRow && row >= p.rows) return;   // whole warps, and no CTA barrier below
  const int C = p.cols;
  const __nv_bfloat16* x = p.x + row * p.ldx;
  const R* r = p.residual ? static_cast<const R*>(p.residual) + row * p.ldr : nullptr;
  float s[kV][8];
  float ss = 0.0f;
  const float inv_c = 1.0f / (float)C;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = 8 * (tr + i * nt);
    if (c < C) {
      load8<__nv_bfloat16, kVec>(x + c, C - c, s[i]);
      if (r) {
        float t[8];
        load8<R, kVec>(r + c, C - c, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[i][e] += t[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += s[i][e] * (s[i][e] * inv_c);   // the mean itself: C squares
                                                                    // need not fit fp32's range
  }
  if (r) {
    R* so = static_cast<R*>(p.residual_out) + row * p.lds;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = 8 * (tr + i * nt);
      if (c < C) store8<kVec>(so + c, C - c, s[i]);
    }
  }
  ss = row_reduce<false, kWarpRow>(ss, red[0]);
  const float rho = 1.0f / sqrtf(ss + p.eps);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = 8 * (tr + i * nt);
    if (c < C) {
      float w[8];
      load8<Wt, kVec>(static_cast<const Wt*>(p.weight) + c, C - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] = s[i][e] * rho * w[e];
      if (p.y) store8<kVec>(p.y + row * p.ldy + c, C - c, s[i]);
    }
    if (p.y8 && p.group) {   // 16 adjacent lanes hold a group
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(s[i][e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (c < C) {
        const float scale = max_nan(m / kE4M3Max, 0x1p-40f), inv = 1.0f / scale;
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = s[i][e] * inv;
        store8_e4m3<kVec>(p.y8 + row * p.ldy8 + c, C - c, q);
        if ((threadIdx.x & 15) == 0) p.y_scale[row * ((C + 127) / 128) + c / 128] = scale;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(s[i][e]));
    }
  }
  if (p.y8 && !p.group) {
    top = row_reduce<true, kWarpRow>(top, red[1]);
    const float scale = max_nan(top / kE4M3Max, 0x1p-40f), inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = 8 * (tr + i * nt);
      if (c < C) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = s[i][e] * inv;
        store8_e4m3<kVec>(p.y8 + row * p.ldy8 + c, C - c, q);
      }
    }
    if (tr == 0) p.y_scale[row] = scale;
  }
}

template <typename R, typename Wt, int kV, bool kVec>
cudaError_t launch_v(const NormParams& p, cudaStream_t stream) {
  const int chunks = (p.cols + 7) / 8;
  if constexpr (kV == 1) {
    if (chunks <= 32) {   // a warp per row, eight rows a CTA
      const unsigned grid = (unsigned)((p.rows + 7) / 8);
      return launch(kda_norm_kernel<R, Wt, kV, kVec, true>, dim3(grid), dim3(256), 0, true, stream, p);
    }
  }
  const int threads = ((chunks + kV - 1) / kV + 31) / 32 * 32;
  return launch(kda_norm_kernel<R, Wt, kV, kVec, false>, dim3((unsigned)p.rows), dim3(threads), 0, true,
                stream, p);
}

template <typename R, typename Wt, bool kVec>
cudaError_t launch_rw(const NormParams& p, cudaStream_t stream) {
  // One chunk a thread as long as a CTA has the threads for a row (cols <= 8192): 32 registers, two
  // full CTAs an SM.  Against four chunks a thread on a GB300, bf16 in and out: 131072 x 256
  // 42.6 / 65.3 us, 16384 x 4096 82.3 / 89.7, 16384 x 7168 152.3 / 164.0 (93% / 86% of the copy
  // rate), and the shortest chain of loads for a few rows.  Wider rows take four (12288 columns:
  // two chunks 178.0 us, four 154.3).
  return p.cols <= 8 * 1024 ? launch_v<R, Wt, 1, kVec>(p, stream) : launch_v<R, Wt, 4, kVec>(p, stream);
}

template <typename R, typename Wt>
cudaError_t launch_r(const NormParams& p, bool aligned, cudaStream_t stream) {
  return aligned ? launch_rw<R, Wt, true>(p, stream) : launch_rw<R, Wt, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool aligned, cudaStream_t stream) {
  if (p.residual_f32)
    return p.weight_f32 ? launch_r<float, float>(p, aligned, stream)
                        : launch_r<float, __nv_bfloat16>(p, aligned, stream);
  return p.weight_f32 ? launch_r<__nv_bfloat16, float>(p, aligned, stream)
                      : launch_r<__nv_bfloat16, __nv_bfloat16>(p, aligned, stream);
}

}  // namespace attn
}  // namespace kda
