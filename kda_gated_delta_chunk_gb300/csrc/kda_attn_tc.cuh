// Shared by the tcgen05 attention kernels: e4m3 matrix instructions, the paged cache's tensor
// maps, and the split of a batch's key tiles over the CTAs.
#pragma once

#include <cuda.h>

#include "kda_attn.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace attn {

using namespace sm100;

constexpr int kTile = 128;              // keys of a tile
constexpr int kMaxLen = 0x7fffffff - (kTile - 1);   // cached tokens of a sequence: whole tiles end below 2^31
constexpr int kOver = 3;                // units (tiles' worth of time) an item takes besides its tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 operations in one instruction (each rounded as its scalar form).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r, x, y, z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
// Maximum over the warp (NaN lanes do not count).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}

// ------------------------------------------------------------ capped scores
// cap tanh(s / cap) log2(e) + a from t = s log2(e), with y = s / cap:
//   caps of at most 64: tanh y = 1 - 2 / (1 + e^(2 y)) for every y: two special functions, and an error
//     of 2^-22 of the cap, 2^-16 of a score at most, which the sum of its products leaves as well
//   larger caps, whose own precision would be an error of the score (2e-3 at 10^4): to fp32's relative
//     precision of the capped score whatever the cap,
//       |y| < 0.6:  tanh y = y + y^3 g(y^2), g of degree 3 with the least largest relative error of
//                   tanh there (6.6e-8; with the roundings of fp32 1.6e-7), found by linear programming
//       else:       the form above, which cancels no more than half of itself
//     The first takes no special function, and most scores are that small beside such a cap: a
//     group of them is looked at before, and the second left out where none is larger.
// Prefill, 4096 tokens at 16384: caps of at most 64 597 us; larger ones 585, and 759 where every group has
// scores past 0.6 of the cap, which is why the smaller caps, that meet such scores, do without.
enum { kNoCap = 0, kCapPlain = 1, kCapExact = 2 };
inline int cap_kind(float softcap) { return softcap <= 0.0f ? kNoCap : softcap <= 64.0f ? kCapPlain : kCapExact; }
constexpr float kCapSmall = 0.6f;
struct Cap {
  float inv, cap;     // 1 / (cap log2(e)), cap log2(e)
};
__device__ __forceinline__ Cap cap_of(float softcap) { return {1.0f / (softcap * kLog2e), softcap * kLog2e}; }
// For caps of at most 64: x times `mul` is t; to_e = 2 log2(e) inv mul.
__device__ __forceinline__ float cap_plain(float x, float to_e, const Cap& c, float a) {
  return fmaf(-2.0f * c.cap, rcp(1.0f + ex2(x * to_e)), c.cap + a);
}
// For larger ones, where |y| < 0.6.
__device__ __forceinline__ float2 cap_small(float2 t, const Cap& c, float2 a) {
  const float2 y = mul2(t, make_float2(c.inv, c.inv)), u = mul2(y, y);
  float2 g = fma2(u, make_float2(0.0154861547f, 0.0154861547f), make_float2(-0.0521145090f, -0.0521145090f));
  g = fma2(g, u, make_float2(0.133107468f, 0.133107468f));
  g = fma2(g, u, make_float2(-0.333324194f, -0.333324194f));
  return fma2(mul2(t, u), g, add2(t, a));
}
// For larger ones, either form by the size of each.
__device__ __forceinline__ float2 cap_any(float2 t, const Cap& c, float2 a) {
  auto large = [&](float x, float b) {
    return fmaf(fmaf(-2.0f, rcp(1.0f + ex2(x * c.inv * (2.0f * kLog2e))), 1.0f), c.cap, b);
  };
  const float2 s = cap_small(t, c, a), l = make_float2(large(t.x, a.x), large(t.y, a.y));
  return make_float2(fabsf(t.x * c.inv) < kCapSmall ? s.x : l.x, fabsf(t.y * c.inv) < kCapSmall ? s.y : l.y);
}
// max(a, |b|, |c|), a not negative
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float y;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f8f6f4 with e4m3 operands, fp32 accumulate; K = 32.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator, A and B e4m3 (format 0).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// ... of kind::f16 with f16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return idesc_e4m3(M, N, a_mn, b_mn);   // format 0 of both is f16 there
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  return h;
}
// Two e4m3 terms of a pair of values that f16 holds exactly (bf16 values scaled to at most 448):
// x = first + second but for what lies below 2^-10.  Low halves of the results.
__device__ __forceinline__ void split_e4m3x2(float x0, float x1, uint32_t& first, uint32_t& second) {
  const uint32_t h = f16x2_of(x0, x1);
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h));
  const uint32_t back = f16x2_of_e4m3x2(a);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(r));
  first = a;
  second = b;
}
// r / g for 0 <= r < 256 and 1 <= g <= 256, with magic = 65535 / g + 1.
__device__ __forceinline__ int div_small(int r, uint32_t magic) { return (int)(((uint32_t)r * magic) >> 16); }
// 8-bit tiles with the 128-byte swizzle: a row of 128 bytes per token (key, query row), rows in
// groups of 8; the 16-byte chunk index is XORed with row % 8.  As a K-major operand (channels
// along K) a K step of 32 is 32 bytes on; as an MN-major one (tokens along K) 32 rows.
__device__ __forceinline__ uint32_t tile_off(int row, int byte) {
  return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
}
__device__ __forceinline__ uint64_t kmajor8(uint32_t tile, int ks) {
  return sdesc_sw128(tile + 32 * ks, 16, 1024);
}
__device__ __forceinline__ uint64_t mnmajor8(uint32_t tile, int ks) {
  return sdesc_sw128(tile + 4096 * ks, 16, 1024);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// The same, for a warp that stays together: issued by the lane(s) whose `on` is set, so that the
// operands can live in uniform registers.
__device__ __forceinline__ void mma_e4m3_on(uint32_t on, uint32_t d_tmem, uint64_t adesc,
                                            uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts_on(uint32_t on, uint32_t d_tmem, uint32_t a_tmem,
                                               uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// Waits for the loads from tensor memory.  Naming their registers keeps the compiler from moving
// what reads them to before the wait, when a load and its wait stand apart.
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void mma_commit_on(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Keys and values as [page][head][slot][128 bytes]; a box is one page of one head.
struct CacheMaps {
  CUtensorMap k, v;
};
bool make_cache_maps(const CacheView& c, CacheMaps* m);

// ------------------------------------------------------------ the kernels of a call
// With both kernels in a call the decode kernel runs beside the prefill kernel, whose programmatic
// dependent it is: were it to wait for that grid, as a dependent does for what it reads, nothing
// would overlap.  It reads nothing of the prefill kernel's, only what the work before the call
// wrote, and gets that through a word of the workspace: a thread of the prefill kernel, having
// waited for that work, stores the call's number there (release) before it lets dependents start, and
// the decode kernel's CTAs load it (acquire).  A CTA that does not find the number waits for the
// whole prefill grid instead.  The last kernel of the call sets the word back to 0.
constexpr int kGateWord = 16;      // int index in the workspace's 256 bytes of status words
// Sequences with at most max_rows (at most 32) rows: new tokens x heads per kv head, unless they
// add up to fewer than `least` units.  `gate`: the call's number when the prefill kernel is launched
// before it, else 0.
size_t decode_workspace_bytes(int sms);
cudaError_t launch_attn_decode(const AttnParams& p, const CacheMaps& maps, int max_rows, int64_t least,
                               int gate, void* work, int sms, cudaStream_t stream);
// Sequences with more than `few` rows, and the others when those add up to fewer than `least`
// units (heads per kv head at most 256).
size_t prefill_workspace_bytes(int sms);
cudaError_t launch_attn_prefill(const AttnParams& p, const CacheMaps& maps, int few, int64_t least,
                                int gate, void* work, int sms, cudaStream_t stream);
// The parts of items that the cut divided, merged: as the programmatic dependent of the kernel
// before, which they wait for.
cudaError_t launch_attn_decode_merge(const AttnParams& p, int max_rows, void* work, int sms,
                                     cudaStream_t stream);
cudaError_t launch_attn_prefill_merge(const AttnParams& p, int gate, void* work, int sms,
                                      cudaStream_t stream);

// ------------------------------------------------------------ one sequence of a batch
struct SeqInfo {
  int tok0, q_len, len;   // first new token, new tokens, cached tokens (new ones included)
  int tile0, tiles;       // key tiles any of its queries sees; at least one (whose keys may all
                          // be masked), so that every query row is written; 0: not in this launch
};
// The first position that a query at `pos` or a later one sees.  (A position before 0 sees nothing;
// taken as 0, it leaves the difference in range whatever the window.)
__device__ __forceinline__ int first_seen(int pos, int window) {
  return window > 0 ? max(0, max(pos, 0) - window + 1) : 0;
}
// Sequences with min_rows <= q_len * group <= max_rows are this launch's.  `err`: the code to
// record for a malformed sequence (which is left out), or KDA_OK.
__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int n, int min_rows, int max_rows,
                                            int* err) {
  SeqInfo s;
  const int t0 = p.cu_seqlens[n], t1 = p.cu_seqlens[n + 1];
  s.tok0 = t0;
  s.q_len = t1 - t0;
  s.len = p.c.kv_lens[n];
  s.tile0 = s.tiles = 0;
  *err = KDA_OK;
  if (t0 < 0 || t1 < t0 || (int64_t)t1 > p.total_tokens) {
    *err = KDA_ERR_BAD_CU_SEQLENS;
    return s;
  }
  if (s.len < 0 || s.len > kMaxLen || (int64_t)s.len > (int64_t)p.c.max_blocks * p.c.page_size) {
    *err = KDA_ERR_BAD_CACHE_INDEX;
    return s;
  }
  if (s.q_len > p.max_q_len) {
    *err = KDA_ERR_INVALID_ARG;
    return s;
  }
  const int64_t rows = (int64_t)s.q_len * (p.heads / p.c.kv_heads);
  if (s.q_len == 0 || rows < min_rows || rows > max_rows) return s;
  s.tile0 = first_seen(s.len - s.q_len, p.window) / kTile;
  s.tiles = max(1, (s.len + kTile - 1) / kTile - s.tile0);
  return s;
}

}  // namespace attn
}  // namespace kda
