// The KDA recurrence along the branches of drafted trees, without a state per node.  Per (sequence, head), with
// S0 the state before the tree, a_i the decays of node i and c_i their product from the cached text to i:
//   K_ij = kh_i . (a_i ... a_{after j} kh_j),  Q_ij = qh_i . (the same)     j an ancestor of i (Q: or i)
//   u_i = b_i (v_i - S0^T (c_i kh_i) - sum_j K_ij u_j)
//   o_i =            S0^T (c_i qh_i) + sum_j Q_ij u_j
// which is the gated delta rule with every node's state written out from S0.  So the state is read once and
// none is written (a state a node would be 64 KB each); kda_tree_commit makes the accepted one of the u.
//
// S0^T times the 2 n vectors is one tcgen05 product: M = 128 value channels, N = 2 n, K = 128 key channels, f16
// with fp32 sums.  fp32 values enter as two f16 terms, hi hi + hi lo + lo hi.  f16's range is met by powers of two,
// one a value channel of S0 and one a vector, which bring the largest to 2^13 or more and are taken out of the sums
// again: a factor is exact to 2^-22 of itself, and to f16's half step of 2^-25, 2^-38 of the largest (so one of 2^-24
// of it keeps 14 bits).  The low terms' own product, 2^-22 again, is left out.  (A state in bf16 is exact in one
// term down to 2^-30 of its column's largest.)  S0 goes from registers to tensor memory, a thread half a column of it: that
// operand needs no shared memory and no transposition.  The rest is fp32:
//  - a node's walk up its branch carries kh and qh times the decays met, 8 lanes a node and 16 channels a
//    lane, one pair of products an ancestor, and ends as c_i kh_i and c_i qh_i;
//  - then the nodes in blocks of 8, a thread a value channel: four warps make u, the other four follow a block
//    behind with o.  Sums over earlier blocks have no chain but their own length, and blocks without a pair
//    of node and ancestor are left out.
// 64 sequences of 32 nodes, 32 heads, fp32 states, inputs cold: 78 us with random parents, 82.6 where every second
// node follows the one before it (252 MB of inputs and outputs, 134 of them states: 3.1 TB/s), 115 for chains; with
// bf16 states (185 MB) 75 and 79.5; 64 nodes 193 and 206 (fp32), 183 and 197 (bf16), two CTAs an SM; one tree of 8 nodes,
// 16 heads 5.5.  Not bound by memory: a (sequence, head) takes 30,000 cycles of three on an SM (the nodes' loads
// 3,000, gates and norms 2,400, walks and vectors 10,000, the state 3,500 and its terms 1,400, the products 2,300,
// the nodes in order 7,000), and half the state's bytes save 3 us.  Measured and not
// kept: 512 threads a CTA (99 us, two CTAs of 256 95), the state towards L2 ahead (no gain), the next ancestor's
// rows loaded ahead, half the shuffles of a walk, keys in bf16 there (none), the inverse of 1 + b K solved for
// beside the product and a second product with it (101).
#include <cuda_fp16.h>

#include "kda_attn_tc.cuh"
#include "kda_tc_common.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

using namespace sm100;
using attn::kLog2e;
using tcc::unpack_bf16x2;

constexpr int kThreads = 256;
constexpr int kBlock = 8;          // nodes of a block

template <int NT, bool kBf16, bool kMany>      // nodes at most; the state's type; more CTAs than run at once
struct Cfg {
  // Three CTAs an SM have 80 registers a thread and 128 columns of tensor memory each.  So the state comes late, when
  // the walks are done (its first rows a little earlier), and its two terms take the same columns one after the
  // other.  Alone on an SM that costs time, beside two others it hides: 64 sequences of 8, 16, 32 nodes with random
  // parents, 32 heads, fp32 44, 53, 78 us (all of the state late 45, 54, 80), two CTAs with the state on its way from
  // the start 52, 62, 91; 10 sequences of 32 nodes 20 : 23.
  static constexpr int kCtas = kMany && NT <= 32 ? 3 : 2;         // an SM
  static constexpr bool kLate = kCtas == 3;
  static constexpr int kEarly = 24;                               // (of 64)
  static constexpr int kRows = 2 * NT;
  static constexpr int kB = kRows * 256;                          // one term of the vectors
  static constexpr int kBlocks = NT / kBlock, kPairs = kBlocks * (kBlocks + 1) / 2;
  // keys [NT][128] and decays [NT][128] (fp32), then over them the vectors' two terms, then u [NT][128]
  static constexpr int kOffDecay = NT * 512;
  static constexpr int kOffV = NT * 1024;                         // bf16 [NT][128]
  static constexpr int kOffKK = kOffV + NT * 256;                 // K: blocks (b, pb <= b) of [8 j][8 i]
  static constexpr int kOffQQ = kOffKK + kPairs * 256;
  static constexpr int kOffMax = kOffQQ + kPairs * 256;           // float [2][128]; then uint8 [kBlocks][128]
  static constexpr int kOffMul = kOffMax + 1024;                  // float [kRows]
  static constexpr int kOffBeta = kOffMul + kRows * 4;            // float [NT]
  static constexpr int kOffLink = kOffBeta + NT * 4;              // int [NT]
  static constexpr int kOffFlag = kOffLink + NT * 4;              // int [kPairs]: the block has a pair
  static constexpr int kOffAnc = (kOffFlag + kPairs * 4 + 15) / 16 * 16;   // uint64 [NT]: a node's branch
  static constexpr int kOffBar = kOffAnc + NT * 8;
  static constexpr int kBytes = kOffBar + 16 + 1024;
  static constexpr uint32_t kTD = kBf16 || kLate ? 64 : 128;      // the state's terms, then the sums
  static constexpr uint32_t kTmem = kTD + kRows <= 128 ? 128 : 256;
  static_assert(2 * kB == NT * 1024, "the vectors over keys and decays");
  static_assert(kBlocks * 128 <= 1024, "the blocks' marks over the maxima");
  static_assert(kCtas * kBytes <= 226 * 1024 && kCtas * kTmem <= 512, "CTAs an SM");
};
__device__ __forceinline__ int pair_block(int b, int pb) { return b * (b + 1) / 2 + pb; }

// D[tmem] (+)= A[tmem] B[smem]^T with f16 operands.
__device__ __forceinline__ void mma_half_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Instruction descriptor of kind::f16 with f16 operands, both K-major, fp32 sums.
constexpr uint32_t idesc_half(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// 1 / (1 + e^-x), and a channel's decay exp(lower sigmoid(exp(A_log) x)), x = g + dt_bias, with gate =
// -exp(A_log) log2(e) and lower = lower_bound log2(e).  The special functions are within 2^-22 of their
// results and lower within 7.3, so a decay is within 2^-20 of itself.
__device__ __forceinline__ float sigmoid_of(float x) { return attn::rcp(1.0f + attn::ex2(-kLog2e * x)); }
__device__ __forceinline__ float decay_of(float x, float gate, float lower) {
  return attn::ex2(lower * attn::rcp(1.0f + attn::ex2(gate * x)));
}

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Exponent that brings a row with this largest magnitude (its bits) to [2^13, 2^14)
__device__ __forceinline__ int to_half_range(uint32_t bits) { return min(max((int)(bits >> 23) - 127 - 13, -100), 114); }
// |x|'s bits, 0 for what is not finite
__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// Two f16 terms of a pair of floats
__device__ __forceinline__ void split(float2 x, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 b = __half22float2(h);
  const __half2 l = __floats2half2_rn(x.x - b.x, x.y - b.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Place of channel ch in a row of keys or decays: a lane's eight channels are two runs of four, so that the
// 8 lanes of a node read whole lines.
__device__ __forceinline__ int place(int ch) {
  return (ch & 64) + ((ch & 4) << 3) + ((ch & 63) >> 3) * 4 + (ch & 3);
}

template <int NT, bool kBf16, bool kMany>
__global__ void __launch_bounds__(kThreads, Cfg<NT, kBf16, kMany>::kCtas)
    kda_tree_recur_kernel(const __grid_constant__ RecurParams p) {
  using C = Cfg<NT, kBf16, kMany>;
  using attn::fma2;
  using attn::mul2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.heads, seq = blockIdx.x / p.heads;
  pdl_wait();
  Nodes s;
  int err;
  if (!nodes_of(p.cu_seqlens, seq, p.total_tokens, p.max_q_len, &s, &err) || s.n == 0) {
    if (err != KDA_OK && h == 0 && tid == 0) record_error(p.status, err, 440);
    return;
  }
  const int64_t hoff = (int64_t)h * kHeadDim;

  // ---- loads on their way: the nodes' (a warp a node, 4 channels a lane; kAhead nodes a warp at a time),
  // then the state (or later), a thread half a column of it (64 of its 128 key channels)
  constexpr int kPer = NT / 8, kAhead = kPer < 4 ? kPer : 4;
  uint2 kw[kAhead], vw[kAhead], gw[kAhead];
  auto load_nodes = [&](int m0) {
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int i = warp + 8 * (m0 + m);
      kw[m] = vw[m] = gw[m] = make_uint2(0, 0);
      if (i < s.n) {
        const int64_t t = s.tok0 + i, at = hoff + 4 * lane;
        kw[m] = *reinterpret_cast<const uint2*>(p.k + t * p.s_k + at);
        gw[m] = *reinterpret_cast<const uint2*>(p.g + t * p.s_g + at);
        vw[m] = *reinterpret_cast<const uint2*>(p.v + t * p.s_v + at);
      }
    }
  };
  load_nodes(0);
  float beta_in = 0.0f;
  int link_in = -1;
  if (tid < s.n) {
    beta_in = __bfloat162float(p.beta[(s.tok0 + tid) * p.s_beta + h]);
    link_in = parent_of(p.parents, s, tid, p.status, h == 0);
  }
  const float4 dt = *reinterpret_cast<const float4*>(p.dt_bias + hoff + 4 * lane);
  const float gate = -kLog2e * expf(p.A_log[h]), lower = p.lower_bound * kLog2e;
  const int col = tid & 127, part = tid >> 7;
  float st[64];
  auto load_state = [&](int r0, int r1) {       // rows [r0, r1) of the 64
    const int64_t at = ((int64_t)seq * p.heads + h) * (kHeadDim * kHeadDim) + part * (64 * kHeadDim) + col;
    if (!p.initial_state) {
#pragma unroll
      for (int r = r0; r < r1; ++r) st[r] = 0.0f;
    } else if (kBf16) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.initial_state) + at;
#pragma unroll
      for (int r = r0; r < r1; ++r) st[r] = __bfloat162float(src[r * kHeadDim]);
    } else {
      const float* src = static_cast<const float*>(p.initial_state) + at;
#pragma unroll
      for (int r = r0; r < r1; ++r) st[r] = src[r * kHeadDim];
    }
  };
  if (!C::kLate) load_state(0, 64);
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_s), C::kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(sb + C::kOffBar, 1);
    mbar_fence_init();
  }
  float* keys = reinterpret_cast<float*>(sm);
  float* decay = reinterpret_cast<float*>(sm + C::kOffDecay);
  float* kk = reinterpret_cast<float*>(sm + C::kOffKK);
  float* qq = reinterpret_cast<float*>(sm + C::kOffQQ);
  float* maxs = reinterpret_cast<float*>(sm + C::kOffMax);
  float* mul = reinterpret_cast<float*>(sm + C::kOffMul);
  float* beta = reinterpret_cast<float*>(sm + C::kOffBeta);
  int* link = reinterpret_cast<int*>(sm + C::kOffLink);
  int* flag = reinterpret_cast<int*>(sm + C::kOffFlag);
  uint64_t* anc = reinterpret_cast<uint64_t*>(sm + C::kOffAnc);
  uint8_t* bad_s = sm + C::kOffMax;      // (over the maxima; a block its own: u's warps run ahead of o's)

  if (tid < NT) {      // (past the nodes: zeros)
    beta[tid] = tid < s.n ? sigmoid_of(beta_in) : 0.0f;
    link[tid] = link_in;
    anc[tid] = 0;
  }
  for (int i = tid; i < C::kPairs * 32; i += kThreads)      // (K and Q, 512 bytes a block)
    reinterpret_cast<float4*>(kk)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid < C::kPairs) flag[tid] = 0;
  // ---- the nodes' keys, values, decays
#pragma unroll
  for (int m0 = 0; m0 < kPer; m0 += kAhead) {
    if (m0 > 0) load_nodes(m0);
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int i = warp + 8 * (m0 + m);
      const float2 k0 = unpack_bf16x2(kw[m].x), k1 = unpack_bf16x2(kw[m].y);
      const float2 g0 = unpack_bf16x2(gw[m].x), g1 = unpack_bf16x2(gw[m].y);
      float sum = fmaf(k0.x, k0.x, k0.y * k0.y) + fmaf(k1.x, k1.x, k1.y * k1.y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float ik = rsqrtf(sum + kL2Eps);
      *reinterpret_cast<float4*>(keys + i * 128 + place(4 * lane)) =
          make_float4(k0.x * ik, k0.y * ik, k1.x * ik, k1.y * ik);
      *reinterpret_cast<float4*>(decay + i * 128 + place(4 * lane)) =
          make_float4(decay_of(g0.x + dt.x, gate, lower), decay_of(g0.y + dt.y, gate, lower),
                      decay_of(g1.x + dt.z, gate, lower), decay_of(g1.y + dt.w, gate, lower));
      *reinterpret_cast<uint2*>(sm + C::kOffV + i * 256 + 8 * lane) = vw[m];
    }
  }
  // the queries of this lane's nodes in the walks: 8 lanes a node, channels 8 sub .. and 64 + 8 sub ..
  constexpr int kPasses = (NT + kThreads / 8 - 1) / (kThreads / 8);
  const int sub = lane & 7, node0 = 4 * warp + (lane >> 3);
  uint4 qw[kPasses][2];
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      qw[pass][c] = make_uint4(0, 0, 0, 0);
      if (32 * pass + node0 < s.n)
        qw[pass][c] = *reinterpret_cast<const uint4*>(p.q + (int64_t)(s.tok0 + 32 * pass + node0) * p.s_q + hoff +
                                                      64 * c + 8 * sub);
    }
  auto column_max = [&] {
    float top = 0.0f;
#pragma unroll
    for (int r = 0; r < 64; r += 2) top = attn::max3_abs(top, st[r], st[r + 1]);
    if (top > 3.402823466e38f) {     // (infinities: the largest of the others)
      top = 0.0f;
#pragma unroll
      for (int r = 0; r < 64; ++r) top = fmaxf(top, __uint_as_float(magnitude(st[r])));
    }
    maxs[tid] = top;
  };
  if (!C::kLate) column_max();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (not before this CTA has its tensor memory: a dependent might take it, and wait for this grid's end)
  pdl_launch_dependents();
  const uint32_t tmem = tmem_s;
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;

  // ---- the state as f16 terms, a power of two a column: channels 2 c, 2 c + 1 in column c
  float unscale = 1.0f;
  uint32_t hi[32];       // (late: the low terms go first, and these take their place)
  auto put_state = [&] {
    const int fe = to_half_range(__float_as_uint(fmaxf(maxs[col], maxs[128 + col])));
    unscale = pow2(fe);
    const float f = pow2(-fe);
#pragma unroll
    for (int c0 = 0; c0 < 32; c0 += 16) {
      uint32_t lo[16];
#pragma unroll
      for (int c = 0; c < 16; ++c)
        split(mul2(make_float2(st[2 * (c0 + c)], st[2 * (c0 + c) + 1]), make_float2(f, f)), hi[c0 + c], lo[c]);
      if (!kBf16) tmem_st16(tmem + lanes + (C::kLate ? 0 : 64) + 32 * part + c0, lo);
    }
    if (kBf16 || !C::kLate) tmem_st32(tmem + lanes + 32 * part, hi);
  };
  if (!C::kLate) put_state();

  // ---- walks
  float2 wk[kPasses][8], wq[kPasses][8];
  auto load_row = [&](const float* row, float2 (&x)[8]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 y = *reinterpret_cast<const float4*>(row + (c >> 1) * 64 + (c & 1) * 32 + 4 * sub);
      x[2 * c] = make_float2(y.x, y.y);
      x[2 * c + 1] = make_float2(y.z, y.w);
    }
  };
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int i = 32 * pass + node0;
    const bool live = i < s.n;
    if (!__any_sync(0xffffffffu, live)) break;
    {
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t x[4] = {qw[pass][c].x, qw[pass][c].y, qw[pass][c].z, qw[pass][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          wq[pass][4 * c + e] = unpack_bf16x2(x[e]);
          sum = fma2(wq[pass][4 * c + e], wq[pass][4 * c + e], sum);
        }
      }
      float all = sum.x + sum.y;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      const float iq = p.scale * rsqrtf(all + kL2Eps);
      load_row(keys + (live ? i : 0) * 128, wk[pass]);
#pragma unroll
      for (int e = 0; e < 8; ++e) wq[pass][e] = mul2(wq[pass][e], make_float2(iq, iq));
    }
    int j = live ? i : -1;
    uint64_t branch = 0;
    const int row0 = (i / kBlock) * (i / kBlock + 1) / 2, in_block = i % kBlock;
    while (__any_sync(0xffffffffu, j >= 0)) {
      const int jj = max(j, 0);
      float2 x[8], a[8];
      load_row(keys + jj * 128, x);
      load_row(decay + jj * 128, a);
      const int up = link[jj];
      float2 dk = make_float2(0.f, 0.f), dq = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dk = fma2(wk[pass][e], x[e], dk);
        dq = fma2(wq[pass][e], x[e], dq);
      }
      float rk = dk.x + dk.y, rq = dq.x + dq.y;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        rk += __shfl_xor_sync(0xffffffffu, rk, o);
        rq += __shfl_xor_sync(0xffffffffu, rq, o);
      }
      if (j >= 0) {
        branch |= 1ull << j;
        if (sub == 0) {
          const int blk = row0 + j / kBlock, at = blk * 64 + (j % kBlock) * 8 + in_block;
          kk[at] = rk;          // (a node's with itself is not used)
          qq[at] = rq;
          flag[blk] = 1;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wk[pass][e] = mul2(wk[pass][e], a[e]);
          wq[pass][e] = mul2(wq[pass][e], a[e]);
        }
        j = up;
      }
    }
    if (live && sub == 0) anc[i] = branch;
  }
  if (C::kLate) load_state(0, C::kEarly);
  else tmem_wait_st();
  __syncthreads();            // keys and decays have been read: the vectors go over them
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int i = 32 * pass + node0;
    if (i >= NT) break;
    auto put = [&](float2 (&w)[8], int row, bool live) {
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!live) w[e] = make_float2(0.f, 0.f);
        top = attn::max3_abs(top, w[e].x, w[e].y);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int f = to_half_range(__float_as_uint(top));     // (infinite: the vector's sums are no numbers)
      const float m = pow2(-f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(mul2(w[4 * c + e], make_float2(m, m)), hi[e], lo[e]);
        const uint32_t off = kmajor_off(row, 64 * c + 8 * sub, C::kRows);
        *reinterpret_cast<uint4*>(sm + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sm + C::kB + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (sub == 0) mul[row] = pow2(f);
    };
    const int row = 2 * kBlock * (i / kBlock) + i % kBlock;       // a block's vectors of k, then of q
    put(wk[pass], row, i < s.n);
    put(wq[pass], row + kBlock, i < s.n);
  }
  if (C::kLate) {
    load_state(C::kEarly, 64);
    column_max();
    __syncthreads();
    put_state();
    tmem_wait_st();
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // ---- S0^T [c kh; c qh]^T
  constexpr uint32_t id = idesc_half(128, C::kRows);
  auto product = [&](uint32_t a, uint32_t b, bool more) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      mma_half_ts(tmem + C::kTD, a + 8 * ks, tcc::kdesc(b, C::kRows, ks), id, more || ks > 0);
  };
  constexpr bool kTwice = C::kLate && !kBf16;
  if (tid == 0) {           // (the state's low terms first, whichever way: a sequence's sums are the same in every batch)
    if (!kBf16) product(tmem + (kTwice ? 0 : 64), sb, false);
    if (!kTwice) {
      product(tmem, sb, !kBf16);
      product(tmem, sb + C::kB, true);
    }
    mma_commit(sb + C::kOffBar);
  }
  bool ok = mbar_wait(sb + C::kOffBar, 0);
  if (kTwice) {
    tc_fence_after();
    tmem_st32(tmem + lanes + 32 * part, hi);
    tmem_wait_st();
    tc_fence_before();
    ok = __syncthreads_and(ok);
    tc_fence_after();
    if (ok && tid == 0) {
      product(tmem, sb, true);
      product(tmem, sb + C::kB, true);
      mma_commit(sb + C::kOffBar);
    }
    if (ok) ok = mbar_wait(sb + C::kOffBar, 1);
  }
  ok = __syncthreads_and(ok);
  tc_fence_after();

  // ---- the nodes in order (u over the vectors: the product is done)
  if (!ok) {
    if (tid == 0) record_error(p.status, KDA_ERR_DEVICE_TIMEOUT, 441);
  } else {
    float* us = reinterpret_cast<float*>(sm) + col;
    const __nv_bfloat16* vs = reinterpret_cast<const __nv_bfloat16*>(sm + C::kOffV) + col;
    const int64_t row = ((int64_t)s.tok0 * p.heads + h) * kHeadDim + col;
    const int step = p.heads * kHeadDim;
    const float* pairs = part == 0 ? kk : qq;
    float* u_out = p.u + row;
    __nv_bfloat16* o_out = p.out + row;
    bool bad = false;       // some node so far has no number in this channel
    for (int b = 0; b * kBlock < s.n; ++b) {
      const int left = s.n - b * kBlock;
      const float* diag = pairs + pair_block(b, b) * 64;
      uint32_t x[16];
      tmem_ld16(tmem + lanes + C::kTD + 2 * kBlock * b, x);
      tmem_wait_ld();
      float first[8];       // (a vector's power first, 2^-13 at most for keys: a column's may take the sum past fp32's end)
#pragma unroll
      for (int r = 0; r < 8; r += 4) {
        const float4 m = *reinterpret_cast<const float4*>(mul + 2 * kBlock * b + kBlock * part + r);
        const float ms[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) first[r + e] = __uint_as_float(part == 0 ? x[r + e] : x[8 + r + e]) * ms[e] * unscale;
      }
      float2 acc[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = make_float2(first[2 * r], first[2 * r + 1]);
      // block (b, pb)'s part of the eight sums
      auto add = [&](int pb) {
        const float* w = pairs + pair_block(b, pb) * 64;
        const float* uj = us + pb * (kBlock * 128);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = uj[j * 128];
          const float4 w0 = *reinterpret_cast<const float4*>(w + 8 * j), w1 = *reinterpret_cast<const float4*>(w + 8 * j + 4);
          const float2 uu = make_float2(u, u);
          acc[0] = fma2(make_float2(w0.x, w0.y), uu, acc[0]);
          acc[1] = fma2(make_float2(w0.z, w0.w), uu, acc[1]);
          acc[2] = fma2(make_float2(w1.x, w1.y), uu, acc[2]);
          acc[3] = fma2(make_float2(w1.z, w1.w), uu, acc[3]);
        }
      };
      // The same sum for node r of the block by its own branch: a node without a number must not meet the
      // zeros of those that do not descend from it.
      auto sum_of = [&](int r, uint64_t on) -> float {
        float sum = first[r];
        while (on) {
          const int j = __ffsll((long long)on) - 1;
          on &= on - 1;
          sum = fmaf(pairs[pair_block(b, j / kBlock) * 64 + (j % kBlock) * 8 + r], us[j * 128], sum);
        }
        return sum;
      };
      for (int pb = 0; pb < b; ++pb)
        if (flag[pair_block(b, pb)]) add(pb);
      if (part == 0) {
        float v[8], u[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = __bfloat162float(vs[(kBlock * b + r) * 128]);
        const float4 b0 = *reinterpret_cast<const float4*>(beta + kBlock * b);
        const float4 b1 = *reinterpret_cast<const float4*>(beta + kBlock * b + 4);
        const float bs[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        float sums[8], most = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) sums[r] = r & 1 ? acc[r >> 1].y : acc[r >> 1].x;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          u[r] = bs[r] * (v[r] - sums[r]);
          most = attn::max_nan(most, fabsf(u[r]));
          float w[8];
          *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(diag + 8 * r);
          *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(diag + 8 * r + 4);
#pragma unroll
          for (int y = r + 1; y < 8; ++y) sums[y] = fmaf(w[y], u[r], sums[y]);
        }
        if (bad || !(most <= 3.402823466e38f)) {
          bad = true;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int i = kBlock * b + r;
            u[r] = i < s.n ? bs[r] * (v[r] - sum_of(r, anc[i] & ~(1ull << i))) : 0.0f;
            us[i * 128] = u[r];
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          us[(kBlock * b + r) * 128] = u[r];
          if (r < left) u_out[r * step] = u[r];
        }
        u_out += (int64_t)kBlock * step;
        bad_s[128 * b + col] = bad;
        bar_arrive(1 + b, kThreads);
      } else {
        named_barrier_sync(1 + b, kThreads);
        bad = bad_s[128 * b + col] != 0;
        add(b);
        if (bad) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float o = sum_of(r, anc[kBlock * b + r]);
            if (r & 1) acc[r >> 1].y = o;
            else acc[r >> 1].x = o;
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < left) o_out[r * step] = __float2bfloat16_rn(r & 1 ? acc[r >> 1].y : acc[r >> 1].x);
        o_out += (int64_t)kBlock * step;
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
// A CTA takes half of a (sequence, head)'s key channels: the state's rows in registers, kRows a warp and 4 value
// channels a lane, on their way while the branch is found and its keys are scaled.  Bound by the state's
// read and write: 64 sequences of 32 nodes, 32 heads, fp32 (268 MB) 50.2 us, 5.4 TB/s; a whole (sequence, head) a CTA
// and two CTAs an SM 54.4.  bf16 (134 MB) takes 40, and 34 with 8 nodes: what a CTA does
// before its sums (the branch, its keys, decays and u) does not shrink with the state.
constexpr int kCommitRows = 8, kHalves = kHeadDim / (kCommitRows * kThreads / 32);
__host__ __device__ constexpr int commit_bytes(int nodes) { return nodes * 1024; }   // keys and u, fp32

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) kda_tree_commit_kernel(const __grid_constant__ RecurParams p) {
  extern __shared__ __align__(16) float dyn[];
  __shared__ int links[kNodes], node_s[kNodes];
  __shared__ float c_s[kHeadDim];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ch0 = (int)(blockIdx.x % kHalves) * (kHeadDim / kHalves), item = blockIdx.x / kHalves;
  const int h = item % p.heads, seq = item / p.heads;
  const bool lead = h == 0 && ch0 == 0;      // reports
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
  const int64_t at = ((int64_t)seq * p.heads + h) * (kHeadDim * kHeadDim) +
                     (ch0 + kCommitRows * warp) * kHeadDim + 4 * lane;
  float4 st[kCommitRows];
#pragma unroll
  for (int r = 0; r < kCommitRows; ++r) {
    st[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!p.initial_state) continue;
    if (kBf16) {
      const uint2 w =
          *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.initial_state) + at + r * kHeadDim);
      const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y);
      st[r] = make_float4(a.x, a.y, b.x, b.y);
    } else {
      st[r] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.initial_state) + at + r * kHeadDim);
    }
  }
  int L = 0;
  float* keys = dyn;                                   // [L][128]
  float* us = dyn + p.max_q_len * kHeadDim;            // [L][128]
  if (!ok) {      // (the state stays)
    if (lead && tid == 0) record_error(p.status, err, 442);
  } else if (s.n > 0 && node >= 0) {
    const uint64_t on = branch_of(p.parents, s, node, links, p.status, lead);
    L = __popcll(on);
    if (tid < s.n && ((on >> tid) & 1)) node_s[__popcll(on & ((1ull << tid) - 1))] = tid;
    __syncthreads();
    // keys of the branch, their decays beside them in the place of u
    const float gate = -kLog2e * expf(p.A_log[h]), lower = p.lower_bound * kLog2e;
    const float4 dt = *reinterpret_cast<const float4*>(p.dt_bias + hoff + 4 * lane);
    for (int e = warp; e < L; e += kThreads / 32) {
      const int64_t t = s.tok0 + node_s[e];
      const uint2 kw = *reinterpret_cast<const uint2*>(p.k + t * p.s_k + hoff + 4 * lane);
      const uint2 gw = *reinterpret_cast<const uint2*>(p.g + t * p.s_g + hoff + 4 * lane);
      const float2 k0 = unpack_bf16x2(kw.x), k1 = unpack_bf16x2(kw.y);
      const float2 g0 = unpack_bf16x2(gw.x), g1 = unpack_bf16x2(gw.y);
      float sum = k0.x * k0.x + k0.y * k0.y + k1.x * k1.x + k1.y * k1.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float ik = rsqrtf(sum + kL2Eps);
      *reinterpret_cast<float4*>(keys + e * kHeadDim + 4 * lane) =
          make_float4(k0.x * ik, k0.y * ik, k1.x * ik, k1.y * ik);
      *reinterpret_cast<float4*>(us + e * kHeadDim + 4 * lane) =
          make_float4(decay_of(g0.x + dt.x, gate, lower), decay_of(g0.y + dt.y, gate, lower),
                      decay_of(g1.x + dt.z, gate, lower), decay_of(g1.y + dt.w, gate, lower));
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
    for (int r = 0; r < kCommitRows; ++r) {
      const float c = c_s[ch0 + kCommitRows * warp + r];
      st[r] = make_float4(st[r].x * c, st[r].y * c, st[r].z * c, st[r].w * c);
    }
    for (int e = 0; e < L; ++e) {
      const float4 u = *reinterpret_cast<const float4*>(us + e * kHeadDim + 4 * lane);
#pragma unroll
      for (int r = 0; r < kCommitRows; r += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(keys + e * kHeadDim + ch0 + kCommitRows * warp + r);
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
  for (int r = 0; r < kCommitRows; ++r) {
    if (kBf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.final_state) + at + r * kHeadDim) =
          make_uint2(pack_bf16x2(st[r].x, st[r].y), pack_bf16x2(st[r].z, st[r].w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.final_state) + at + r * kHeadDim) = st[r];
  }
}

template <int NT, bool kBf16, bool kMany>
cudaError_t launch_nodes(const RecurParams& p, cudaStream_t stream) {
  using C = Cfg<NT, kBf16, kMany>;
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&]() -> cudaError_t {
    return cudaFuncSetAttribute(kda_tree_recur_kernel<NT, kBf16, kMany>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kBytes);
  });
  if (e != cudaSuccess) return e;
  return attn::launch(kda_tree_recur_kernel<NT, kBf16, kMany>, dim3((unsigned)(p.num_seqs * p.heads)), dim3(kThreads),
                      C::kBytes, true, stream, p);
}
template <bool kBf16, bool kMany>
cudaError_t launch_dtype(const RecurParams& p, cudaStream_t stream) {
  return p.max_q_len <= 8    ? launch_nodes<8, kBf16, kMany>(p, stream)
         : p.max_q_len <= 16 ? launch_nodes<16, kBf16, kMany>(p, stream)
         : p.max_q_len <= 32 ? launch_nodes<32, kBf16, kMany>(p, stream)
                             : launch_nodes<64, kBf16, false>(p, stream);
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
  return attn::launch(kda_tree_commit_kernel<kBf16>, dim3((unsigned)(p.num_seqs * p.heads * kHalves)), dim3(kThreads),
                      (size_t)commit_bytes(p.max_q_len), true, stream, p);
}

}  // namespace

cudaError_t launch_recur(const RecurParams& p, int sms, cudaStream_t stream) {
  const bool many = p.num_seqs * p.heads > 2 * sms;
  if (many) return p.state_bf16 ? launch_dtype<true, true>(p, stream) : launch_dtype<false, true>(p, stream);
  return p.state_bf16 ? launch_dtype<true, false>(p, stream) : launch_dtype<false, false>(p, stream);
}
cudaError_t launch_commit(const RecurParams& p, cudaStream_t stream) {
  return p.state_bf16 ? launch_commit_dtype<true>(p, stream) : launch_commit_dtype<false>(p, stream);
}

}  // namespace tree
}  // namespace kda
