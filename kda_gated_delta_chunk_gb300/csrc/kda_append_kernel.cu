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
// One launch, two kinds of CTA.  The first ones share out the (page, kv head, keys or values) units
// of the step: every CTA adds up the pages of all sequences (a load and a scan), takes an equal,
// contiguous range of units and holds a unit's rows in registers, 16 lanes a row, between the
// maximum and the store.  The others rotate the queries, 16 lanes a (token, group of heads) with
// the token's table row in registers.  A lane holds both channels of its pairs -- four and four
// half the rotated part apart, or eight in a row -- so that the rotation needs no exchange.
// Bound by memory in a prefill, by the chain of dependent loads in a decode step: 8 x 2048 tokens of
// 16 heads over 4 in 36.5 us (5.3 TB/s), 16 ragged sequences of up to 1000 in pages of 16 in 19.4 us
// (4.1 TB/s), 64 x 1 token of 32 heads over 8 in 5.8 us.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kSearchRounds = 4;   // sequences per thread that a CTA looks through for its tokens
constexpr int kRegs = 64;   // of a thread: with 1024 threads an SM, 64 KB of loads in flight

// The channels of lane `lane` of 16: two runs of four, [c0, c0 + 4) and [c1, c1 + 4), and the
// column of its first cosine (negative: these channels are not rotated).
struct Lane {
  int c0, c1, col;
};
template <bool kInter>
__device__ __forceinline__ Lane lane_of(int lane, int rot) {
  Lane l;
  if (kInter || 8 * lane >= rot) {       // eight in a row: four interleaved pairs, or the rest
    l.c0 = 8 * lane;
    l.c1 = 8 * lane + 4;
  } else {
    l.c0 = 4 * lane;
    l.c1 = (rot >> 1) + 4 * lane;
  }
  l.col = 8 * lane < rot ? 4 * lane : -1;
  return l;
}
struct Row8 {     // eight bf16 channels as loaded
  uint2 a, b;
};
__device__ __forceinline__ Row8 load_row(const __nv_bfloat16* p, const Lane& l) {
  return {*reinterpret_cast<const uint2*>(p + l.c0), *reinterpret_cast<const uint2*>(p + l.c1)};
}
__device__ __forceinline__ void unpack_row(const Row8& r, float (&v)[8]) {
  unpack8(make_uint4(r.a.x, r.a.y, r.b.x, r.b.y), v);
}
struct Turn {
  float4 c, s;
};
__device__ __forceinline__ Turn load_turn(const float* row, int rot, const Lane& l) {
  if (l.col < 0) return {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  return {*reinterpret_cast<const float4*>(row + l.col),
          *reinterpret_cast<const float4*>(row + (rot >> 1) + l.col)};
}
// Products and sums rounded one by one (no contraction): the value does not depend on which
// of the two products a fused multiply-add would keep unrounded.
__device__ __forceinline__ void turn1(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}
template <bool kInter>
__device__ __forceinline__ void rotate8(float (&v)[8], const Lane& l, const Turn& t) {
  if (l.col < 0) return;
  const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) turn1(v[kInter ? 2 * j : j], v[kInter ? 2 * j + 1 : 4 + j], c[j], s[j]);
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

// Pages that sequence n's new tokens touch; 0 for a malformed one, whose error `report` records.
struct SeqPages {
  int t0, t1, len, start, pages;
};
__device__ __forceinline__ SeqPages seq_pages(const AppendParams& p, int n, bool report) {
  SeqPages q = {p.cu_seqlens[n], p.cu_seqlens[n + 1], p.c.kv_lens[n], 0, 0};
  const int P = p.c.page_size;
  if (q.t0 < 0 || q.t1 < q.t0 || (int64_t)q.t1 > p.total_tokens) {
    if (report) record_error(p.status, KDA_ERR_BAD_CU_SEQLENS, 201);
    return q;
  }
  if (q.t1 == q.t0) return q;
  q.start = q.len - (q.t1 - q.t0);
  if (q.start < 0 || (int64_t)q.len > (int64_t)p.c.max_blocks * P) {
    if (report) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 202);
    return q;
  }
  q.pages = (q.len - 1) / P - q.start / P + 1;
  return q;
}

// kRows: token rows a 16-lane group takes of a page at a time (page size = kRows * groups * kPasses).
// kHeads: query heads a 16-lane group takes of a token.
template <int kRows, int kHeads, int kThreads, int kPasses, bool kInter>
__global__ void __launch_bounds__(kThreads, 65536 / kRegs / kThreads)
    kda_append_kernel(const __grid_constant__ AppendParams p, int page_ctas) {
  __shared__ float top_s[2][kThreads / 32];
  __shared__ long long sum_s[kThreads / 32], first_s;
  __shared__ int n_s;
  __shared__ int64_t pos_s[kThreads / 16];
  const int tid = threadIdx.x, lane16 = tid & 15, grp = tid >> 4;
  constexpr int groups = kThreads / 16, warps = kThreads / 32, kStep = kRows * groups;
  const int warp = tid >> 5;
  const Lane ln = lane_of<kInter>(lane16, p.rot_dim);
  const int32_t* cu = p.cu_seqlens;
  const int N = p.num_seqs;
  sm100::pdl_wait();   // (launched as a programmatic dependent of the work before it)
  sm100::pdl_launch_dependents();
  if ((int)blockIdx.x < page_ctas) {
    // ---- this CTA's range of units, and the sequence that it begins in
    const int hk = p.c.kv_heads, P = p.c.page_size;
    if (blockIdx.x == 0 && tid == 0 && (cu[0] != 0 || (int64_t)cu[N] > p.total_tokens))
      record_error(p.status, KDA_ERR_BAD_CU_SEQLENS, 200);
    long long mine = 0, first = 0;
    for (int n0 = 0; n0 < N; n0 += blockDim.x) {
      const int pages = n0 + tid < N ? seq_pages(p, n0 + tid, blockIdx.x == 0).pages : 0;
      if (n0 == 0) first = pages;
      mine += pages;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((tid & 31) == 0) sum_s[warp] = mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < warps; ++w) total += sum_s[w];
    total *= 2 * hk;
    __syncthreads();
    // (64-bit divisions only where they are needed: they would be half of a decode step's instructions)
    const bool small = total <= (long long)(0xffffffffu / (unsigned)page_ctas);
    auto share = [&](unsigned i) -> long long {
      return small ? (long long)(i * (unsigned)total / (unsigned)page_ctas) : (long long)i * total / page_ctas;
    };
    long long u = share(blockIdx.x);
    const long long u_end = share(blockIdx.x + 1);
    if (u >= u_end) return;
    const long long page0 = small ? (unsigned)u / (unsigned)(2 * hk) : u / (2 * hk);
    long long before = 0;
    for (int n0 = 0; n0 < N && before <= page0; n0 += blockDim.x) {
      const long long w = n0 == 0 ? first : (n0 + tid < N ? seq_pages(p, n0 + tid, false).pages : 0);
      long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if ((tid & 31) >= o) inc += x;
      }
      if ((tid & 31) == 31) sum_s[warp] = inc;
      __syncthreads();
      long long off = before;
      for (int x = 0; x < warp; ++x) off += sum_s[x];
      if (w > 0 && page0 >= off + inc - w && page0 < off + inc) {
        n_s = n0 + tid;
        first_s = off + inc - w;
      }
      for (int x = 0; x < warps; ++x) before += sum_s[x];
      __syncthreads();
    }
    int n = n_s;
    SeqPages q = seq_pages(p, n, false);
    int blk = (int)(page0 - first_s), unit = (int)(u - page0 * (2 * hk));   // page of the sequence, unit of the page
    // ---- the units: keys or values of one (page, kv head)
    uint32_t par = 0;      // buffer of the warps' maxima: the other one at each unit that reaches the barrier
    for (; u < u_end; ++u) {
      while (blk >= q.pages) {
        if (++n >= N) return;   // (lengths that changed under the kernel)
        q = seq_pages(p, n, false);
        blk = 0;
      }
      const bool is_v = unit >= hk;
      const int h = is_v ? unit - hk : unit;
      const int b = q.start / P + blk;
      const int s0 = b * P < q.start ? q.start - b * P : 0, s1 = min(P, q.len - b * P);   // new rows
      const int t_row0 = q.t0 + b * P - q.start;            // token of the page's row 0
      if (++unit == 2 * hk) {
        unit = 0;
        ++blk;
      }
      const int page = p.c.block_table[n * p.c.table_stride + b];
      const __nv_bfloat16* src = (is_v ? p.v : p.k) + h * kHeadDim;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      // rows are taken kStep at a time, from the first pass that holds a new one to the last
      const int pass0 = kPasses > 1 ? s0 / kStep : 0, pass1 = kPasses > 1 ? (s1 - 1) / kStep : 0;
      Row8 raw[kRows];
      auto fetch = [&](int pass) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = pass * kStep + grp + i * groups;
          raw[i] = {make_uint2(0, 0), make_uint2(0, 0)};
          if (row >= s0 && row < s1) raw[i] = load_row(src + (int64_t)(t_row0 + row) * stride, ln);
        }
      };
      fetch(pass0);
      if (page < 0 || page >= p.c.num_pages) {
        if (tid == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 203);
        continue;
      }
      uint8_t* dst = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + h * p.c.head_stride;
      float* scale_p = (is_v ? p.c.v_scale : p.c.k_scale) + page * p.c.scale_stride + h;
      const float old = s0 > 0 ? *scale_p : 0.0f;
      float x[kRows][8];
      float top = 0.0f;
      bool some = kHeads > 2;       // of this warp's rows are new (few tokens: mostly none)
      auto turn = [&](int pass) -> float {   // the rows fetched, rotated; their largest finite entry
        if (kHeads <= 2) {
          some = false;
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int row = pass * kStep + grp + i * groups;
            some = some || (row >= s0 && row < s1);
          }
          some = __any_sync(0xffffffffu, some);
        }
        float most = 0.0f;
        if (!some) return most;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = pass * kStep + grp + i * groups;
          unpack_row(raw[i], x[i]);
          if (!is_v && p.rot_dim && row >= s0 && row < s1) {
            const int64_t pos = p.positions ? (int64_t)p.positions[t_row0 + row] : (int64_t)b * P + row;
            if (pos >= 0 && pos < p.rope_rows)
              rotate8<kInter>(x[i], ln, load_turn(p.rope + pos * p.rot_dim, p.rot_dim, ln));
            else if (lane16 == 0)   // the row is stored unrotated
              record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 204);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[i][e]));
        }
        if (most > 3.402823466e38f) {   // an infinity: the maximum of the finite ones
          most = 0.0f;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (fabsf(x[i][e]) <= 3.402823466e38f) most = fmaxf(most, fabsf(x[i][e]));
        }
        return most;
      };
      top = turn(pass0);
      for (int pass = pass0 + 1; kPasses > 1 && pass <= pass1; ++pass) {
        fetch(pass);
        top = fmaxf(top, turn(pass));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if ((tid & 31) == 0) top_s[par][warp] = top;
      __syncthreads();              // (the other parity's readers are past the barrier before this)
      for (int w = 0; w < warps; ++w) top = fmaxf(top, top_s[par][w]);
      par ^= 1;
      float scale = pow2_scale(top);
      if (s0 > 0) scale = fmaxf(scale, old);
      const float inv = 1.0f / scale;
      for (int pass = pass0; pass <= pass1; ++pass) {
        if (pass1 > pass0) {        // (more than one: the registers hold the last)
          fetch(pass);
          turn(pass);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = pass * kStep + grp + i * groups;
          if (some && row >= s0 && row < s1) {
            uint8_t* w = dst + row * p.c.token_stride;
            *reinterpret_cast<uint32_t*>(w + ln.c0) = e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
            *reinterpret_cast<uint32_t*>(w + ln.c1) = e4m3x4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
          }
        }
      }
      if (s0 > 0 && scale > old) {   // the page's older rows, brought to the new scale
        const float ratio = old * inv;
        for (int first = 0; first < (kPasses > 1 ? s0 : 1); first += kStep) {
          uint2 kept[kRows];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int row = first + grp + i * groups;
            if (row < s0) kept[i] = *reinterpret_cast<const uint2*>(dst + row * p.c.token_stride + 8 * lane16);
          }
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int row = first + grp + i * groups;
            if (row >= s0) continue;
            const float2 a = from_e4m3x2(kept[i].x & 0xffff), b2 = from_e4m3x2(kept[i].x >> 16);
            const float2 c = from_e4m3x2(kept[i].y & 0xffff), d = from_e4m3x2(kept[i].y >> 16);
            *reinterpret_cast<uint2*>(dst + row * p.c.token_stride + 8 * lane16) =
                make_uint2(e4m3x4(a.x * ratio, a.y * ratio, b2.x * ratio, b2.y * ratio),
                           e4m3x4(c.x * ratio, c.y * ratio, d.x * ratio, d.y * ratio));
          }
        }
      }
      if (tid == 0 && (s0 == 0 || scale > old)) *scale_p = scale;
    }
    return;
  }
  // ---- queries: 16 lanes a (token, kHeads heads)
  const int units = (p.heads + kHeads - 1) / kHeads;
  const int64_t u0 = ((int64_t)blockIdx.x - page_ctas) * groups, u = u0 + grp;
  const int64_t t = u / units, tok0 = u0 / units;
  const int64_t tokens = min((int64_t)cu[N], p.total_tokens);
  const int h0 = (int)(u % units) * kHeads;
  Row8 raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (t < tokens && h0 + i < p.heads) raw[i] = load_row(p.q + t * p.q_stride + (h0 + i) * kHeadDim, ln);
  int64_t pos = 0;
  if (p.rot_dim && !p.positions) {
    // cache positions of this CTA's tokens (at most one per group), found as the slots are
    const int64_t tok1 = min(tokens, (u0 + groups - 1) / units + 1);
    if (N <= kSearchRounds * (int)blockDim.x) {
      for (int n = tid; n < N; n += blockDim.x) {
        const int64_t a = cu[n], b = cu[n + 1], len = p.c.kv_lens[n];
        for (int64_t x = max(a, tok0); x < min(b, tok1); ++x) pos_s[x - tok0] = len - (b - x);
      }
    } else if (tid < tok1 - tok0) {
      const int n = seq_of(cu, N, tok0 + tid);
      pos_s[tid] = (int64_t)p.c.kv_lens[n] - ((int64_t)cu[n + 1] - (tok0 + tid));
    }
    __syncthreads();
    if (t < tokens) pos = pos_s[t - tok0];
  } else if (p.rot_dim && t < tokens) {
    pos = p.positions[t];
  }
  if (t >= tokens) return;
  const bool turns = p.rot_dim && pos >= 0 && pos < p.rope_rows;
  Turn tn;
  if (turns) tn = load_turn(p.rope + pos * p.rot_dim, p.rot_dim, ln);
  else if (p.rot_dim && lane16 == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 205);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (h0 + i >= p.heads) break;
    float x[8];
    unpack_row(raw[i], x);
    if (turns) rotate8<kInter>(x, ln, tn);
    const uint4 o = pack8(x);
    __nv_bfloat16* dst = p.q_out + t * p.qo_stride + (h0 + i) * kHeadDim;
    *reinterpret_cast<uint2*>(dst + ln.c0) = make_uint2(o.x, o.y);
    *reinterpret_cast<uint2*>(dst + ln.c1) = make_uint2(o.z, o.w);
  }
}

template <int kRows, int kHeads, int kThreads, int kPasses>
cudaError_t launch_heads(const AppendParams& p, int sms, cudaStream_t stream) {
  const int64_t resident = (int64_t)sms * (65536 / kRegs / kThreads);
  // at most so many units: every sequence has a partial page at both ends
  const int64_t most = 2 * (p.total_tokens / p.c.page_size + 2 * (int64_t)p.num_seqs) * p.c.kv_heads;
  const int page_ctas = (int)(most < resident ? most : resident);
  const int64_t units = p.q ? p.total_tokens * ((p.heads + kHeads - 1) / kHeads) : 0;
  const int64_t grid = page_ctas + (units + kThreads / 16 - 1) / (kThreads / 16);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 g((unsigned)grid), t(kThreads);
  return p.interleaved ? launch(kda_append_kernel<kRows, kHeads, kThreads, kPasses, true>, g, t, 0, true, stream, p, page_ctas)
                       : launch(kda_append_kernel<kRows, kHeads, kThreads, kPasses, false>, g, t, 0, true, stream, p, page_ctas);
}

// Query heads of a token that share one read of its table row: 4 where there are tokens enough
// to fill the GPU all the same, else 2 for the shorter chain.
template <int kRows, int kThreads, int kPasses = 1>
cudaError_t launch_rows(const AppendParams& p, int sms, cudaStream_t stream) {
  return p.total_tokens >= 1024 ? launch_heads<kRows, 4, kThreads, kPasses>(p, sms, stream)
                                : launch_heads<kRows, 2, kThreads, kPasses>(p, sms, stream);
}

}  // namespace

// Page sizes 16 to 128: a group of 16 lanes takes four rows, whose fp32 values and table entries
// are kept to 64 registers.  Against two rows a group (and twice the threads) on a GB300, as first
// measured: 8 x 2048 tokens in pages of 64 36.9 / 40.8 us, 64 single tokens 8.2 / 10.5; pages of
// 16, ragged, the same.
// In pages of 64 and 128 with few new tokens a sequence (P / 16 on average) a CTA of 64 threads takes
// a page 16 rows at a time, and the new rows twice where they are in more than one such part: most
// warps of a CTA that covers the page would have no new row.  Against that, 64 sequences in pages
// of 64: one token each 5.8 / 7.4 us, 8 9.2 / 9.2, 1 to 40 14.6 / 10.1; in pages of 128: one 6.0 / 11.4,
// 1 to 10 8.4 / 11.6, 1 to 40 15.3 / 14.4.  In pages of 32 one token each 5.9 / 5.7.
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream) {
  if (p.total_tokens <= p.c.page_size / 16 * (int64_t)p.num_seqs) {
    if (p.c.page_size == 64) return launch_rows<4, 64, 4>(p, sms, stream);
    if (p.c.page_size == 128) return launch_rows<4, 64, 8>(p, sms, stream);
  }
  switch (p.c.page_size) {
    case 16: return launch_rows<4, 64>(p, sms, stream);
    case 32: return launch_rows<4, 128>(p, sms, stream);
    case 64: return launch_rows<4, 256>(p, sms, stream);
    default: return launch_rows<4, 512>(p, sms, stream);   // 128
  }
}

}  // namespace attn
}  // namespace kda
