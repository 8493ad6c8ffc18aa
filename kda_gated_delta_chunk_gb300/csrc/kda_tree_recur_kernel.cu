// The KDA recurrence along the branches of drafted trees, without a state per node.  Per (sequence, head), with
// S0 the state before the tree, a_i the decays of node i and c_i their product from the cached text to i:
//   K_ij = kh_i . (a_i ... a_{after j} kh_j),  Q_ij = qh_i . (the same)     j an ancestor of i (Q: or i)
//   u_i = b_i (v_i - S0^T (c_i kh_i) - sum_j K_ij u_j)
//   o_i =            S0^T (c_i qh_i) + sum_j Q_ij u_j
// which is the gated delta rule with every node's state written out from S0.  So the state is read once and
// none is written (a state a node would be 64 KB each); kda_tree_commit makes the accepted one of the u.
//
// S0^T times the 2 n vectors is one tcgen05 product: M = 128 value channels (S0 as it lies in memory is the
// MN-major operand), N = 2 n, K = 128 key channels, f16 with fp32 sums.  fp32 values enter as two f16
// terms, hi hi + hi lo + lo hi: 22 bits.  f16's range is met by powers of two: one a key channel, which
// goes from S0's row to the vectors, one a vector, taken out of its sums.  (A state in bf16 is exact in one term.)
// The rest is fp32: a node's walk up its branch carries kh and qh times the decays met, 8 lanes a node
// and 16 channels a lane, one pair of products an ancestor, and ends as c_i kh_i and c_i qh_i; then a thread a
// value channel takes the nodes in order, its own u in shared memory (no barriers).
#include <cuda_fp16.h>

#include "kda_tree.cuh"
#include "kda_tc_common.cuh"

namespace kda {
namespace tree {
namespace {

using namespace sm100;

constexpr int kThreads = 256;

// Instruction descriptor of kind::f16 with f16 operands, fp32 sums.
constexpr uint32_t idesc_half(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

template <int NT>      // nodes at most
struct Cfg {
  static constexpr int kRows = 2 * NT;
  static constexpr int kA = 32768, kB = kRows * 256;              // one term
  static constexpr int kOffB = 2 * kA;
  static constexpr int kOffDecay = kOffB + 2 * kB;                // float [NT][128], see decay_at
  static constexpr int kOffK = kOffDecay + NT * 512;              // bf16 [NT][128]
  static constexpr int kOffV = kOffK + NT * 256;                  // bf16 [NT][128]
  static constexpr int kPairs = NT * (NT + 1) / 2;
  static constexpr int kOffKQ = kOffV + NT * 256;                 // float2 [kPairs]: node i's ancestors, itself first
  static constexpr int kOffAnc = kOffKQ + kPairs * 8;             // uint8 [kPairs]
  static constexpr int kOffEk = (kOffAnc + kPairs + 15) / 16 * 16;   // float [128]
  static constexpr int kOffMul = kOffEk + 512;                    // float [kRows]
  static constexpr int kOffIk = kOffMul + kRows * 4;              // float [NT]
  static constexpr int kOffBeta = kOffIk + NT * 4;                // float [NT]
  static constexpr int kOffLink = kOffBeta + NT * 4;              // int [NT]
  static constexpr int kOffDepth = kOffLink + NT * 4;             // int [NT]: ancestors, itself included
  static constexpr int kOffBar = kOffDepth + NT * 4;
  static constexpr int kBytes = kOffBar + 16 + 1024;
  static constexpr uint32_t kTmem = kRows <= 32 ? 32 : kRows;
  static_assert(NT * 512 <= 2 * kA, "u over the state's terms");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void mma_half(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Exponent that brings a row with this largest magnitude (its bits) to [2^13, 2^14)
__device__ __forceinline__ int to_half_range(uint32_t bits) { return min(max((int)(bits >> 23) - 127 - 13, -100), 100); }
// |x|'s bits, 0 for what is not finite
__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// Two f16 terms of a pair of floats
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 b = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - b.x, y - b.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Place of channel ch in a row of decays: a lane's eight channels are two runs of four, so that the 8 lanes of a
// node read whole lines.
__device__ __forceinline__ int decay_at(int ch) {
  return (ch & 64) + ((ch & 4) << 3) + ((ch & 63) >> 3) * 4 + (ch & 3);
}

template <int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads, NT <= 16 ? 2 : 1)
    kda_tree_recur_kernel(const __grid_constant__ RecurParams p) {
  using C = Cfg<NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.heads, seq = blockIdx.x / p.heads;
  pdl_wait();
  pdl_launch_dependents();
  Nodes s;
  int err;
  if (!nodes_of(p.cu_seqlens, seq, p.total_tokens, p.max_q_len, &s, &err) || s.n == 0) {
    if (err != KDA_OK && h == 0 && tid == 0) record_error(p.status, err, 440);
    return;
  }
  const int64_t hoff = (int64_t)h * kHeadDim;

  // ---- the state's rows on their way: 16 a warp, 4 channels a lane
  float4 st[16];
  {
    const int64_t at = ((int64_t)seq * p.heads + h) * (kHeadDim * kHeadDim) + 16 * warp * kHeadDim + 4 * lane;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      st[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!p.initial_state) continue;
      if (kBf16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.initial_state) + at +
                                                        r * kHeadDim);
        const float2 a = tcc::unpack_bf16x2(w.x), b = tcc::unpack_bf16x2(w.y);
        st[r] = make_float4(a.x, a.y, b.x, b.y);
      } else {
        st[r] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.initial_state) + at + r * kHeadDim);
      }
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_s), C::kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(sb + C::kOffBar, 1);
    mbar_fence_init();
  }
  float* decay = reinterpret_cast<float*>(sm + C::kOffDecay);
  float* ek = reinterpret_cast<float*>(sm + C::kOffEk);
  float* mul = reinterpret_cast<float*>(sm + C::kOffMul);
  float* ik = reinterpret_cast<float*>(sm + C::kOffIk);
  float* beta = reinterpret_cast<float*>(sm + C::kOffBeta);
  int* link = reinterpret_cast<int*>(sm + C::kOffLink);
  int* depth = reinterpret_cast<int*>(sm + C::kOffDepth);
  float2* kq = reinterpret_cast<float2*>(sm + C::kOffKQ);
  uint8_t* anc = sm + C::kOffAnc;
  const float gsc = expf(p.A_log[h]);

  // ---- the nodes' keys, values, decays: a warp a node, 4 channels a lane
  {
    const float4 dt = *reinterpret_cast<const float4*>(p.dt_bias + hoff + 4 * lane);
    for (int i = warp; i < s.n; i += kThreads / 32) {
      const int64_t t = s.tok0 + i;
      const uint2 kw = *reinterpret_cast<const uint2*>(p.k + t * p.s_k + hoff + 4 * lane);
      const uint2 vw = *reinterpret_cast<const uint2*>(p.v + t * p.s_v + hoff + 4 * lane);
      const uint2 gw = *reinterpret_cast<const uint2*>(p.g + t * p.s_g + hoff + 4 * lane);
      const float2 k0 = tcc::unpack_bf16x2(kw.x), k1 = tcc::unpack_bf16x2(kw.y);
      const float2 g0 = tcc::unpack_bf16x2(gw.x), g1 = tcc::unpack_bf16x2(gw.y);
      float sum = k0.x * k0.x + k0.y * k0.y + k1.x * k1.x + k1.y * k1.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      *reinterpret_cast<uint2*>(sm + C::kOffK + i * 256 + 8 * lane) = kw;
      *reinterpret_cast<uint2*>(sm + C::kOffV + i * 256 + 8 * lane) = vw;
      *reinterpret_cast<float4*>(decay + i * 128 + decay_at(4 * lane)) =
          make_float4(decay_of(g0.x, dt.x, gsc, p.lower_bound), decay_of(g0.y, dt.y, gsc, p.lower_bound),
                      decay_of(g1.x, dt.z, gsc, p.lower_bound), decay_of(g1.y, dt.w, gsc, p.lower_bound));
      if (lane == 0) {
        ik[i] = rsqrtf(sum + kL2Eps);
        beta[i] = 1.0f / (1.0f + expf(-__bfloat162float(p.beta[t * p.s_beta + h])));
        link[i] = parent_of(p.parents, s, i, p.status, h == 0);
      }
    }
  }
  // ---- the state as two f16 terms, a power of two a row
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int k = 16 * warp + r;
    const float4 x = st[r];
    const uint32_t top = __reduce_max_sync(
        0xffffffffu, max(max(magnitude(x.x), magnitude(x.y)), max(magnitude(x.z), magnitude(x.w))));
    const int e = to_half_range(top);
    const float f = pow2(-e);
    uint2 hi, lo;
    split(x.x * f, x.y * f, hi.x, lo.x);
    split(x.z * f, x.w * f, hi.y, lo.y);
    const uint32_t off = mnmajor_off(4 * lane, k, 16384);
    *reinterpret_cast<uint2*>(sm + off) = hi;
    if (!kBf16) *reinterpret_cast<uint2*>(sm + C::kA + off) = lo;
    if (lane == 0) ek[k] = pow2(e);
  }
  __syncthreads();
  const uint32_t tmem = tmem_s;

  // ---- walks: 8 lanes a node, channels 8 s .. 8 s + 7 and 64 + 8 s .. a lane
  {
    const int sub = lane & 7;
    auto load_decay = [&](int j, float (&a)[16]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(decay + j * 128 + (c >> 1) * 64 + (c & 1) * 32 + 4 * sub);
        a[4 * c] = x.x;
        a[4 * c + 1] = x.y;
        a[4 * c + 2] = x.z;
        a[4 * c + 3] = x.w;
      }
    };
    auto load_k = [&](int j, float (&x)[16]) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float y[8];
        attn::unpack8(*reinterpret_cast<const uint4*>(sm + C::kOffK + j * 256 + c * 128 + 16 * sub), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * c + e] = y[e];
      }
    };
    for (int i0 = 4 * warp; i0 < NT; i0 += kThreads / 8) {
      const int i = i0 + (lane >> 3);
      const bool live = i < s.n;
      if (!__any_sync(0xffffffffu, live)) break;
      float wk[16], wq[16], x[16];
      {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (live)
            w = *reinterpret_cast<const uint4*>(p.q + (int64_t)(s.tok0 + i) * p.s_q + hoff + 64 * c + 8 * sub);
          float y[8];
          attn::unpack8(w, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            wq[8 * c + e] = y[e];
            sum += y[e] * y[e];
          }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float iq = p.scale * rsqrtf(sum + kL2Eps);
        const float ki = live ? ik[i] : 0.0f;
        load_k(live ? i : 0, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          wq[e] *= iq;
          wk[e] = x[e] * ki;
        }
      }
      int j = live ? i : -1, d = 0;
      const int base = i * (i + 1) / 2;
      while (__any_sync(0xffffffffu, j >= 0)) {
        const int jj = max(j, 0);
        load_k(jj, x);
        float a[16];
        load_decay(jj, a);
        float dk = 0.0f, dq = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          dk = fmaf(wk[e], x[e], dk);
          dq = fmaf(wq[e], x[e], dq);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          dk += __shfl_xor_sync(0xffffffffu, dk, o);
          dq += __shfl_xor_sync(0xffffffffu, dq, o);
        }
        if (j >= 0) {
          if (sub == 0) {
            kq[base + d] = make_float2(dk * ik[j], dq * ik[j]);
            anc[base + d] = (uint8_t)j;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            wk[e] *= a[e];
            wq[e] *= a[e];
          }
          j = link[j];
          ++d;
        }
      }
      if (live && sub == 0) depth[i] = d;
      // c_i kh_i and c_i qh_i as rows of the operand, a power of two each
      uint32_t tk = 0, tq = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = ek[64 * c + 8 * sub + e];
          wk[8 * c + e] *= f;
          wq[8 * c + e] *= f;
          tk = max(tk, magnitude(wk[8 * c + e]));
          tq = max(tq, magnitude(wq[8 * c + e]));
        }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        tk = max(tk, __shfl_xor_sync(0xffffffffu, tk, o));
        tq = max(tq, __shfl_xor_sync(0xffffffffu, tq, o));
      }
      const int fk = to_half_range(tk), fq = to_half_range(tq);
      const int rk = 16 * (i >> 3) + (i & 7), rq = rk + 8;
      if (i < NT) {
        const float mk = pow2(-fk), mq = pow2(-fq);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split(wk[8 * c + 2 * e] * mk, wk[8 * c + 2 * e + 1] * mk, hi[e], lo[e]);
          uint32_t off = C::kOffB + kmajor_off(rk, 64 * c + 8 * sub, C::kRows);
          *reinterpret_cast<uint4*>(sm + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sm + off + C::kB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) split(wq[8 * c + 2 * e] * mq, wq[8 * c + 2 * e + 1] * mq, hi[e], lo[e]);
          off = C::kOffB + kmajor_off(rq, 64 * c + 8 * sub, C::kRows);
          *reinterpret_cast<uint4*>(sm + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sm + off + C::kB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (sub == 0) {
          mul[rk] = pow2(fk);
          mul[rq] = pow2(fq);
        }
      }
    }
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // ---- S0^T [c kh; c qh]^T: 128 value channels by 2 NT vectors (rows past the nodes are not read back)
  if (tid == 0) {
    constexpr uint32_t id = idesc_half(128, C::kRows, 1, 0);
#pragma unroll
    for (int term = 0; term < (kBf16 ? 2 : 3); ++term) {
      const uint32_t a = sb + (term == 2 ? C::kA : 0), b = sb + C::kOffB + (term == 1 ? C::kB : 0);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_half(tmem, tcc::mndesc(a, 16384, ks), tcc::kdesc(b, C::kRows, ks), id, term > 0 || ks > 0);
    }
    mma_commit(sb + C::kOffBar);
  }
  bool ok = mbar_wait(sb + C::kOffBar, 0);
  ok = __syncthreads_and(ok);
  tc_fence_after();

  // ---- the nodes in order, a thread a value channel (u over the state's terms: the product is done)
  if (!ok) {
    if (tid == 0) record_error(p.status, KDA_ERR_DEVICE_TIMEOUT, 441);
  } else if (warp < 4) {
    float* us = reinterpret_cast<float*>(sm) + tid;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const __nv_bfloat16* vs = reinterpret_cast<const __nv_bfloat16*>(sm + C::kOffV) + tid;
    const int64_t row = ((int64_t)s.tok0 * p.heads + h) * kHeadDim + tid;
    for (int i0 = 0; i0 < s.n; i0 += 8) {
      uint32_t x[16];
      tmem_ld16(tmem + lanes + 2 * i0, x);
      tmem_wait_ld();
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int i = i0 + r;
        if (i < s.n) {
          const int base = i * (i + 1) / 2;
          float stk = __uint_as_float(x[r]) * mul[2 * i0 + r], o = __uint_as_float(x[8 + r]) * mul[2 * i0 + 8 + r];
          const int d = depth[i];
#pragma unroll 4
          for (int e = 1; e < d; ++e) {
            const float2 w = kq[base + e];
            const float uj = us[anc[base + e] * 128];
            stk = fmaf(w.x, uj, stk);
            o = fmaf(w.y, uj, o);
          }
          const float u = beta[i] * (__bfloat162float(vs[i * 128]) - stk);
          us[i * 128] = u;
          o = fmaf(kq[base].y, u, o);
          const int64_t at = row + (int64_t)i * p.heads * kHeadDim;
          p.u[at] = u;
          p.out[at] = __float2bfloat16_rn(o);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// The state after the accepted branch: S' = diag(c) S0 + sum_e (decays after e . kh_e) u_e^T over the branch's nodes e.
// A CTA takes a (sequence, head): the state's rows in registers, 16 a warp and 4 value channels a lane, on
// their way while the branch is found and its keys are scaled.  Bound by the state's read and write.
__host__ __device__ constexpr int commit_bytes(int nodes) { return nodes * 1024; }   // keys and u, fp32

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 2) kda_tree_commit_kernel(const __grid_constant__ RecurParams p) {
  extern __shared__ __align__(16) float dyn[];
  __shared__ int links[kNodes], node_s[kNodes];
  __shared__ float c_s[kHeadDim];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.heads, seq = blockIdx.x / p.heads;
  pdl_wait();
  pdl_launch_dependents();
  Nodes s;
  int err;
  bool ok = nodes_of(p.cu_seqlens, seq, p.total_tokens, p.max_q_len, &s, &err);
  const int node = p.accepted[seq];
  if (ok && s.n > 0 && (node < -1 || node >= s.n)) {
    err = KDA_ERR_BAD_TREE;
    ok = false;
  }
  const int64_t hoff = (int64_t)h * kHeadDim;
  const int64_t at = ((int64_t)seq * p.heads + h) * (kHeadDim * kHeadDim) + 16 * warp * kHeadDim + 4 * lane;
  float4 st[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    st[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!p.initial_state) continue;
    if (kBf16) {
      const uint2 w =
          *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.initial_state) + at + r * kHeadDim);
      const float2 a = tcc::unpack_bf16x2(w.x), b = tcc::unpack_bf16x2(w.y);
      st[r] = make_float4(a.x, a.y, b.x, b.y);
    } else {
      st[r] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.initial_state) + at + r * kHeadDim);
    }
  }
  int L = 0;
  float* keys = dyn;                                   // [L][128]
  float* us = dyn + p.max_q_len * kHeadDim;            // [L][128]
  if (!ok) {      // (the state stays)
    if (h == 0 && tid == 0) record_error(p.status, err, 442);
  } else if (s.n > 0 && node >= 0) {
    const uint64_t on = branch_of(p.parents, s, node, links, p.status, h == 0);
    L = __popcll(on);
    if (tid < s.n && ((on >> tid) & 1)) node_s[__popcll(on & ((1ull << tid) - 1))] = tid;
    __syncthreads();
    // keys of the branch, their decays beside them in the place of u
    const float gsc = expf(p.A_log[h]);
    const float4 dt = *reinterpret_cast<const float4*>(p.dt_bias + hoff + 4 * lane);
    for (int e = warp; e < L; e += kThreads / 32) {
      const int64_t t = s.tok0 + node_s[e];
      const uint2 kw = *reinterpret_cast<const uint2*>(p.k + t * p.s_k + hoff + 4 * lane);
      const uint2 gw = *reinterpret_cast<const uint2*>(p.g + t * p.s_g + hoff + 4 * lane);
      const float2 k0 = tcc::unpack_bf16x2(kw.x), k1 = tcc::unpack_bf16x2(kw.y);
      const float2 g0 = tcc::unpack_bf16x2(gw.x), g1 = tcc::unpack_bf16x2(gw.y);
      float sum = k0.x * k0.x + k0.y * k0.y + k1.x * k1.x + k1.y * k1.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float ik = rsqrtf(sum + kL2Eps);
      *reinterpret_cast<float4*>(keys + e * kHeadDim + 4 * lane) =
          make_float4(k0.x * ik, k0.y * ik, k1.x * ik, k1.y * ik);
      *reinterpret_cast<float4*>(us + e * kHeadDim + 4 * lane) =
          make_float4(decay_of(g0.x, dt.x, gsc, p.lower_bound), decay_of(g0.y, dt.y, gsc, p.lower_bound),
                      decay_of(g1.x, dt.z, gsc, p.lower_bound), decay_of(g1.y, dt.w, gsc, p.lower_bound));
    }
    __syncthreads();
    if (tid < kHeadDim) {
      float c = 1.0f;
      for (int e = L - 1; e >= 0; --e) {
        keys[e * kHeadDim + tid] *= c;
        c *= us[e * kHeadDim + tid];
      }
      c_s[tid] = c;
    }
    __syncthreads();
    for (int e = warp; e < L; e += kThreads / 32)
      *reinterpret_cast<float4*>(us + e * kHeadDim + 4 * lane) = *reinterpret_cast<const float4*>(
          p.u + ((int64_t)(s.tok0 + node_s[e]) * p.heads + h) * kHeadDim + 4 * lane);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float c = c_s[16 * warp + r];
      st[r] = make_float4(st[r].x * c, st[r].y * c, st[r].z * c, st[r].w * c);
    }
    for (int e = 0; e < L; ++e) {
      const float4 u = *reinterpret_cast<const float4*>(us + e * kHeadDim + 4 * lane);
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(keys + e * kHeadDim + 16 * warp + r);
        const float k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          st[r + x].x = fmaf(k[x], u.x, st[r + x].x);
          st[r + x].y = fmaf(k[x], u.y, st[r + x].y);
          st[r + x].z = fmaf(k[x], u.z, st[r + x].z);
          st[r + x].w = fmaf(k[x], u.w, st[r + x].w);
        }
      }
    }
  }
  if (L == 0 && p.final_state == p.initial_state) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (kBf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.final_state) + at + r * kHeadDim) =
          make_uint2(pack_bf16x2(st[r].x, st[r].y), pack_bf16x2(st[r].z, st[r].w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.final_state) + at + r * kHeadDim) = st[r];
  }
}

template <int NT, bool kBf16>
cudaError_t launch_nodes(const RecurParams& p, cudaStream_t stream) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&]() -> cudaError_t {
    return cudaFuncSetAttribute(kda_tree_recur_kernel<NT, kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<NT>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return attn::launch(kda_tree_recur_kernel<NT, kBf16>, dim3((unsigned)(p.num_seqs * p.heads)), dim3(kThreads),
                      Cfg<NT>::kBytes, true, stream, p);
}
template <bool kBf16>
cudaError_t launch_dtype(const RecurParams& p, cudaStream_t stream) {
  return p.max_q_len <= 8    ? launch_nodes<8, kBf16>(p, stream)
         : p.max_q_len <= 16 ? launch_nodes<16, kBf16>(p, stream)
         : p.max_q_len <= 32 ? launch_nodes<32, kBf16>(p, stream)
                             : launch_nodes<64, kBf16>(p, stream);
}
template <bool kBf16>
cudaError_t launch_commit_dtype(const RecurParams& p, cudaStream_t stream) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&]() -> cudaError_t {
    return cudaFuncSetAttribute(kda_tree_commit_kernel<kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                commit_bytes(kNodes));
  });
  if (e != cudaSuccess) return e;
  return attn::launch(kda_tree_commit_kernel<kBf16>, dim3((unsigned)(p.num_seqs * p.heads)), dim3(kThreads),
                      (size_t)commit_bytes(p.max_q_len), true, stream, p);
}

}  // namespace

cudaError_t launch_recur(const RecurParams& p, cudaStream_t stream) {
  return p.state_bf16 ? launch_dtype<true>(p, stream) : launch_dtype<false>(p, stream);
}
cudaError_t launch_commit(const RecurParams& p, cudaStream_t stream) {
  return p.state_bf16 ? launch_commit_dtype<true>(p, stream) : launch_commit_dtype<false>(p, stream);
}

}  // namespace tree
}  // namespace kda
