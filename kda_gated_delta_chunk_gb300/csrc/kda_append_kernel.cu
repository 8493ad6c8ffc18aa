// Rotary positions on new queries and keys, and the append of new keys and values to a paged
// cache held in e4m3 with one scale per (page, kv head).
//
// Token i of a sequence with t new tokens and a cache length of L (new tokens included) sits
// at position p = L - t + i.  Over the first rot_dim channels the pair (a, b) -- channels
// (2j, 2j + 1), or (j, j + rot_dim / 2) -- becomes (a cos - b sin, b cos + a sin), with the
// cosine and sine of row p of the caller's table.
//
// A page's scale is a power of two, the least 2^e (e >= -64) with max|x| <= 448 * 2^e over the
// tokens written.  When the page held tokens of the sequence already, the larger of that and
// the page's old scale holds, and if it grew the old entries are brought to it: a power of two
// only shifts an e4m3 value's exponent, so that is exact except where a value falls below the
// smallest normal, and the cache does not depend on how the tokens were split over calls.
// e4m3 is a floating format, so a power of two loses nothing of its precision against
// max|x| / 448.  Non-finite entries do not enter the maximum; infinities are stored as
// +-448 * scale, NaN as NaN.  The rotation's products and sums are fp32, each rounded on its
// own; keys are quantised from the fp32 values.
//
// One launch, two kinds of CTA.  The first ones each take one page slot and kv head: half of
// the threads the keys, half the values, 16 lanes a token row with its values in registers
// between the maximum and the store.  Sequence n's pages are given the slots from
// floor(cu[n] / P) + 2 n on, which leaves room for the partial pages at both ends without a
// prefix sum; unused slots exit.  The rest rotate the queries, 16 lanes a (token, 4 heads).
// Bound by memory in a prefill, by the chain of dependent loads in a decode step.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kHeadsPerUnit = 4;

// cos / sin of the 8 channels of `lane` (16 lanes a row) at table row `cs`.
struct Turn {
  float c[8], s[8];   // half layout: [e] per channel; interleaved: [0..3] per pair
};
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
template <bool kInter>
__device__ __forceinline__ void load_turn(const float* cs, int rot, int lane, Turn& t) {
  const int half = rot >> 1;
  if (8 * lane >= rot) return;
  if (kInter) {
    load4(cs + 4 * lane, t.c);
    load4(cs + half + 4 * lane, t.s);
  } else {
    const int j = 8 * lane < half ? 8 * lane : 8 * lane - half;
    load4(cs + j, t.c);
    load4(cs + j + 4, t.c + 4);
    load4(cs + half + j, t.s);
    load4(cs + half + j + 4, t.s + 4);
  }
}
// Products and sums rounded one by one (no contraction): the value does not depend on which
// of the two products a fused multiply-add would keep unrounded.
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
// Rotate the 8 channels of this lane (all 16 lanes of the row take part; `mask` names the
// lanes of the warp that are here).
template <bool kInter>
__device__ __forceinline__ void rotate8(float (&v)[8], int rot, int lane, const Turn& t,
                                        uint32_t mask) {
  if (kInter) {
    if (8 * lane < rot) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j], b = v[2 * j + 1];
        v[2 * j] = turn_a(a, b, t.c[j], t.s[j]);
        v[2 * j + 1] = turn_b(a, b, t.c[j], t.s[j]);
      }
    }
  } else {
    const int hl = rot >> 4;   // lanes per half (rot is a multiple of 16)
    const bool first = lane < hl, in = lane < 2 * hl;
    const int src = (threadIdx.x & 16) + (in ? (first ? lane + hl : lane - hl) : lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_sync(mask, v[e], src);
      if (in) v[e] = first ? turn_a(v[e], o, t.c[e], t.s[e]) : turn_b(o, v[e], t.c[e], t.s[e]);
    }
  }
}

// The least 2^e >= 2^-64 with top <= 448 * 2^e (top finite, not negative).
__device__ __forceinline__ float pow2_scale(float top) {
  if (!(top > 448.0f * 0x1p-64f)) return 0x1p-64f;
  const uint32_t u = __float_as_uint(top);
  // top = m * 2^x with m in [1, 2); 448 = 1.75 * 2^8
  const int x = (int)(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// kRows: token rows a 16-lane group takes of a page (page size = kRows * groups per half).
template <int kRows, bool kInter>
__global__ void __launch_bounds__(512) kda_append_kernel(const __grid_constant__ AppendParams p, int64_t page_ctas) {
  __shared__ float top_s[2][16];
  const int tid = threadIdx.x, lane = tid & 15;
  const int32_t* cu = p.cu_seqlens;
  const int N = p.num_seqs;
  if (cu[0] != 0 || (int64_t)cu[N] > p.total_tokens) {
    if (tid == 0) record_error(p.status, KDA_ERR_BAD_CU_SEQLENS, 200);
    return;
  }
  if ((int64_t)blockIdx.x < page_ctas) {
    // ---- keys and values of one (page slot, kv head)
    const int hk = (int)(blockIdx.x % p.c.kv_heads);
    const int64_t slot = blockIdx.x / p.c.kv_heads;
    const int P = p.c.page_size;
    int lo = 0, hi = N - 1;   // the last n with floor(cu[n] / P) + 2 n <= slot
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)(cu[mid] / P) + 2 * (int64_t)mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    const int n = lo;
    const int t0 = cu[n], t1 = cu[n + 1];
    if (t0 < 0 || t1 < t0 || (int64_t)t1 > p.total_tokens) {
      if (tid == 0) record_error(p.status, KDA_ERR_BAD_CU_SEQLENS, 201);
      return;
    }
    const int len = p.c.kv_lens[n];
    const int start = len - (t1 - t0);
    if (t1 == t0) return;
    if (start < 0 || (int64_t)len > (int64_t)p.c.max_blocks * P) {
      if (tid == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 202);
      return;
    }
    const int64_t b = start / P + (slot - (t0 / P + 2 * (int64_t)n));
    if (b > (len - 1) / P) return;   // a slot this sequence does not use
    const int s0 = b * P < start ? start - (int)b * P : 0;              // new rows of the page:
    const int s1 = min(P, len - (int)b * P);                            // [s0, s1)
    const int page = p.c.block_table[n * p.c.table_stride + b];
    if (page < 0 || page >= p.c.num_pages) {
      if (tid == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 203);
      return;
    }
    const int hthreads = blockDim.x >> 1, groups = hthreads >> 4;
    const bool is_v = tid >= hthreads;
    const int ht = is_v ? tid - hthreads : tid, grp = ht >> 4;
    const __nv_bfloat16* src = is_v ? p.v : p.k;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    uint8_t* dst = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + hk * p.c.head_stride;
    float* scale_p = (is_v ? p.c.v_scale : p.c.k_scale) + page * p.c.scale_stride + hk;
    const float old = s0 > 0 ? *scale_p : 0.0f;
    float x[kRows][8];
    float top = 0.0f;
    const uint32_t gmask = 0xffffu << (tid & 16);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = grp + i * groups;
      if (row >= s0 && row < s1) {
        const int64_t t = t0 + (b * P + row - start);
        unpack8(*reinterpret_cast<const uint4*>(src + t * stride + hk * kHeadDim + 8 * lane), x[i]);
        if (!is_v && p.rot_dim) {
          const int64_t pos = p.positions ? (int64_t)p.positions[t] : b * P + row;
          if (pos < 0 || pos >= p.rope_rows) {   // the row is stored unrotated
            if (lane == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 204);
          } else {
            Turn tn;
            load_turn<kInter>(p.rope + pos * p.rot_dim, p.rot_dim, lane, tn);
            rotate8<kInter>(x[i], p.rot_dim, lane, tn, gmask);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = fabsf(x[i][e]);
          if (a <= 3.402823466e38f) top = fmaxf(top, a);   // finite ones
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) top_s[is_v][ht >> 5] = top;
    __syncthreads();
    for (int w = 0; w < hthreads / 32; ++w) top = fmaxf(top, top_s[is_v][w]);
    float scale = pow2_scale(top);
    if (s0 > 0) scale = fmaxf(scale, old);
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = grp + i * groups;
      if (row >= s0 && row < s1) {
        uint2 o;
        o.x = e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
        o.y = e4m3x4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
        *reinterpret_cast<uint2*>(dst + row * p.c.token_stride + 8 * lane) = o;
      }
    }
    if (s0 > 0 && scale > old) {   // the page's older rows, brought to the new scale
      const float ratio = old * inv;
      for (int row = grp; row < s0; row += groups) {
        uint2* w = reinterpret_cast<uint2*>(dst + row * p.c.token_stride + 8 * lane);
        const uint2 u = *w;
        const float2 a = from_e4m3x2(u.x & 0xffff), b2 = from_e4m3x2(u.x >> 16);
        const float2 c = from_e4m3x2(u.y & 0xffff), d = from_e4m3x2(u.y >> 16);
        *w = make_uint2(e4m3x4(a.x * ratio, a.y * ratio, b2.x * ratio, b2.y * ratio),
                        e4m3x4(c.x * ratio, c.y * ratio, d.x * ratio, d.y * ratio));
      }
    }
    if (ht == 0 && !(s0 > 0 && scale == old)) *scale_p = scale;
    return;
  }
  // ---- queries: 16 lanes a (token, kHeadsPerUnit heads)
  const int units = (p.heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
  const int64_t u = ((int64_t)blockIdx.x - page_ctas) * (blockDim.x >> 4) + (tid >> 4);
  const int64_t t = u / units;
  if (t >= (int64_t)cu[N]) return;
  const int h0 = (int)(u % units) * kHeadsPerUnit;
  const uint32_t gmask = 0xffffu << (tid & 16);
  float x[kHeadsPerUnit][8];
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i)
    if (h0 + i < p.heads)
      unpack8(*reinterpret_cast<const uint4*>(p.q + t * p.q_stride + (h0 + i) * kHeadDim + 8 * lane), x[i]);
  if (p.rot_dim) {
    int64_t pos;
    if (p.positions) {
      pos = p.positions[t];
    } else {
      const int n = seq_of(cu, N, t);
      pos = (int64_t)p.c.kv_lens[n] - ((int64_t)cu[n + 1] - t);
    }
    if (pos < 0 || pos >= p.rope_rows) {
      if (lane == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 205);
    } else {
      Turn tn;
      load_turn<kInter>(p.rope + pos * p.rot_dim, p.rot_dim, lane, tn);
#pragma unroll
      for (int i = 0; i < kHeadsPerUnit; ++i)
        if (h0 + i < p.heads) rotate8<kInter>(x[i], p.rot_dim, lane, tn, gmask);
    }
  }
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i)
    if (h0 + i < p.heads)
      *reinterpret_cast<uint4*>(p.q_out + t * p.qo_stride + (h0 + i) * kHeadDim + 8 * lane) = pack8(x[i]);
}

template <int kRows>
cudaError_t launch_rows(const AppendParams& p, int threads, cudaStream_t stream) {
  const int64_t slots = p.total_tokens / p.c.page_size + 2 * (int64_t)p.num_seqs;
  const int64_t page_ctas = slots * p.c.kv_heads;
  const int64_t units = p.q ? p.total_tokens * ((p.heads + kHeadsPerUnit - 1) / kHeadsPerUnit) : 0;
  const int64_t grid = page_ctas + (units + threads / 16 - 1) / (threads / 16);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (p.interleaved)
    kda_append_kernel<kRows, true><<<(unsigned)grid, threads, 0, stream>>>(p, page_ctas);
  else
    kda_append_kernel<kRows, false><<<(unsigned)grid, threads, 0, stream>>>(p, page_ctas);
  return cudaGetLastError();
}

}  // namespace

// Page sizes 16 to 128: 16 lanes a row and half of the threads for the keys, so that a group
// takes 2, 4 or 8 rows, and 8 rows of 8 fp32 values stay in its registers.
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  switch (p.c.page_size) {
    case 16: return launch_rows<2>(p, 256, stream);
    case 32: return launch_rows<4>(p, 256, stream);
    case 64: return launch_rows<8>(p, 256, stream);
    default: return launch_rows<8>(p, 512, stream);   // 128
  }
}

}  // namespace attn
}  // namespace kda
