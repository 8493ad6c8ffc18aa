// Attention over the paged e4m3 cache for few query rows (decode, speculative verify): up to 32
// rows -- new tokens x query heads of one kv head -- share a pass over the keys.  For a tile of
// 128 keys, on tcgen05 with the e4m3 cache as it lies in memory as the A operand of both
// products (nothing of the cache is converted):
//   S^T  = K8 [q1; q2]^T     M = 128 keys, N = 2 x rows: q = q1 + q2, two e4m3 terms
//   P^T  = softmax numerators, thread = key, written as two e4m3 terms
//   O^T  = V8^T [P1; P2]^T   M = 128 channels (V read MN-major), N = 2 x rows
// Two e4m3 terms hold the 8 significant bits of a bf16 query exactly (relative to the row's
// largest entry: to 2^-18), and a numerator to 2^-8 of itself or 2^-18 of the tile's largest: a
// tile's P is scaled by its own maximum, and O^T is added to fp32 registers (thread = channel)
// with the factor to the running maximum, so no tile loses range to an earlier one.  The value
// scale of a key's page enters the exponent, max and all (P = 2^(s + log2 v_scale - max)), and
// leaves again in the sum of the denominators, which takes the unrounded fp32 numerators.
//
// Bound by the cache's bytes (2 x 128 per key and kv head; the products take a few percent of the
// tensor cores).  So that every SM streams the same amount whatever the lengths, the tiles
// of all (sequence, kv head) items are laid end to end and cut into one equal range per CTA, two
// CTAs per SM, each with three 32 KB stages in flight; an item counts kOver tiles more than it
// has, for the time that its queries and its end take.  A CTA's range covers the end of one
// item, whole items and the beginning of another; the (at most two) partial results go to the
// workspace and a second kernel, launched as the first's programmatic dependent, merges them.
// With the merge: 64 ragged sequences of up to 16384 tokens, 32 heads over 8, 67.4 us (5.4 TB/s);
// 4 of 65536, 32 heads over 4, 50.0 us (5.4 TB/s), 16 of them 97% of the rate of a copy; 512 tokens
// 8.8 us.  At 16 rows with capped scores the softmax of a tile takes as long as its copy (16 x 4
// tokens over up to 16384: 52.9 us, 4.3 TB/s), at 32 rows longer (8 tokens each: 86 us, 2.7 TB/s).
//
// Warps: 0-3 softmax and accumulation, 4 the TMA producer, 5 the MMA issuer.  Every wait is
// bounded; one that gives up records KDA_ERR_DEVICE_TIMEOUT and the CTA leaves.
//
// Masked entries: pages before every window are not read; scores by selection; a V row that no query
// sees (past the length, before every window) is zeroed in shared memory before the product, since
// 0 x NaN is NaN; a NaN in a row that only some of the queries see is zeroed too and put into those
// queries' sums by hand.
#include "kda_attn_tc.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kThreads = 192;
constexpr int kStageBytes = 2 * kTile * kHeadDim;   // K and V
constexpr int kCached = 32;                          // sequences whose lengths a CTA keeps in shared memory
constexpr float kPScale = 256.0f;                    // largest numerator, in the e4m3 operand

template <int NR>
struct Cfg {
  static constexpr int kN = 2 * NR;                  // MMA N: both terms
  static constexpr int kStages = NR <= 16 ? 3 : 2;   // what leaves room for two CTAs an SM
  static constexpr uint32_t kTmemCols = kN * 3 <= 64 ? 64 : (kN * 3 <= 128 ? 128 : 256);
  static constexpr uint32_t kTO = 2 * kN;            // S in columns [0, 2 kN), O after it
  // shared memory, from a 1024-byte aligned base
  static constexpr int kOffQ = kStages * kStageBytes;
  static constexpr int kOffP = kOffQ + kN * 128;
  static constexpr int kOffFac = kOffP + kN * 128;              // float4 [2][4 warps][NR]
  static constexpr int kOffMax = kOffFac + 2 * 4 * NR * 16;     // float [2][NR][4]
  static constexpr int kOffSum = kOffMax + 2 * NR * 16;         // float [NR][4]
  static constexpr int kOffPoison = kOffSum + NR * 16;          // uint4 [2][128]
  static constexpr int kOffQmul = kOffPoison + 2 * 128 * 16;    // float [NR]
  static constexpr int kOffScale = kOffQmul + NR * 4;           // float [stages][2][8]
  static constexpr int kOffBar = kOffScale + kStages * 64;      // full, empty, s[2], o, p, q, end
  static constexpr int kOffMisc = kOffBar + 8 * (2 * kStages + 6);
  static constexpr int kOffSeq = kOffMisc + 128;                // SeqInfo [kCached]
  static constexpr int kBytes = kOffSeq + kCached * 20 + 1024;
};

// Workspace after the status words: desc [ctas], then per CTA two slots of [NR][128] sums,
// [NR] maxima and [NR] denominators.
struct PartDesc {
  int parts;          // CTAs whose parts make up the item that this CTA begins; 0: none is cut
  int tok0, rows;     // its first token's row of q and out, its query rows
  int head0;          // its first query head
};
template <int NR>
constexpr int kSlotFloats = NR * 130;

struct DecodeParams {
  AttnParams a;
  CacheMaps maps;
  int group;                 // query heads of a kv head
  uint32_t group_magic;      // 65535 / group + 1 (div_small)
  int gate;                  // the call's number, when this kernel runs beside the prefill kernel; else 0
  int64_t least;             // units below which the prefill kernel takes these sequences too
  int min_rows, max_rows;
  PartDesc* desc;
  float* slots;
};

// The walk over a CTA's range, segment by segment (every role runs its own).  The range is in
// units: an item has kOver of them, then one per tile.
template <bool kTree>
struct Walk {
  int64_t pos, end, base;   // global unit; base: of sequence n's first
  int n, n0;                // sequence; the first of the cached ones
  const SeqInfo* cache;
  SeqInfo s;
  int h, a, b;              // segment: kv head, tiles [a, b) of the item (relative to tile0)
  __device__ __forceinline__ bool next(const DecodeParams& p) {
    while (pos < end) {
      while (true) {
        const int64_t size = s.tiles ? (int64_t)(s.tiles + kOver) * p.a.c.kv_heads : 0;
        if (pos < base + size) break;
        base += size;
        if (++n >= p.a.num_seqs) return false;   // (lengths that changed under the kernel)
        if (n - n0 < kCached) {
          s = cache[n - n0];
        } else {
          int err;
          s = seq_info<kTree>(p.a, n, p.min_rows, p.max_rows, &err);
        }
      }
      const int size = s.tiles + kOver;
      const int64_t x = pos - base;
      h = (int)(x / size);
      const int o = (int)(x % size), o1 = (int)min((int64_t)size, o + (end - pos));
      pos += o1 - o;
      a = max(0, o - kOver);
      b = o1 - kOver;
      if (b > a) return true;       // (else the range ends before the item's first tile)
    }
    return false;
  }
  // unit of the segment's item that its tile t takes
  __device__ __forceinline__ int64_t unit_of(int t) const {
    return base + (int64_t)h * (s.tiles + kOver) + kOver + t;
  }
};

template <int NR, int kCap, bool kTree>
__global__ void __launch_bounds__(kThreads, 2)
    kda_attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<NR>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar_full = sb + C::kOffBar, bar_empty = bar_full + 8 * kStages;
  const uint32_t bar_s = bar_empty + 8 * kStages, bar_o = bar_s + 16, bar_p = bar_o + 8, bar_q = bar_p + 8,
                 bar_end = bar_q + 8;
  struct Misc {
    long long part[8];
    long long total, start_base;
    int start_n;
    uint32_t tmem;
  };
  Misc* misc = reinterpret_cast<Misc*>(sm + C::kOffMisc);
  static_assert(sizeof(Misc) <= 128, "misc");
  const int hk = p.a.c.kv_heads, N = p.a.num_seqs, P = p.a.c.page_size;
  const int G = p.group;
  const uint32_t gm = p.group_magic;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_s + 8, 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_p, 128);
    mbar_init(bar_q, 128);
    mbar_init(bar_end, 1);
    mbar_fence_init();
    tma_prefetch_desc(&p.maps.k);
    tma_prefetch_desc(&p.maps.v);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&misc->tmem), C::kTmemCols);
    tmem_relinquish();
  }
  // (launched as a programmatic dependent: of the work before this call, or of the prefill kernel,
  // which has waited for that and says so)
  if (p.gate == 0) {
    pdl_wait();
  } else {
    if (tid == 0 && ld_acquire_gpu(p.a.status + kGateWord) != p.gate) pdl_wait();
    __syncthreads();
    fence_proxy_async_global();
  }
  pdl_launch_dependents();

  // ---- this CTA's range: total tiles, then the sequence its first tile lies in
  if (tid == 0 && blockIdx.x == 0 && p.a.cu_seqlens[0] != 0) record_error(p.a.status, KDA_ERR_BAD_CU_SEQLENS, 310);
  auto cost = [&](int n, bool report) -> long long {
    if (n >= N) return 0;
    int err;
    const SeqInfo s = seq_info<kTree>(p.a, n, p.min_rows, p.max_rows, &err);
    if (err != KDA_OK && report && blockIdx.x == 0) record_error(p.a.status, err, 311);
    return s.tiles ? (long long)(s.tiles + kOver) * hk : 0;
  };
  long long mine = 0, first = 0;
  for (int n0 = 0; n0 < N; n0 += kThreads) {
    const long long w = cost(n0 + tid, true);
    if (n0 == 0) first = w;
    mine += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) misc->part[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += misc->part[w];
  __syncthreads();
  if (total < p.least) total = 0;
  Walk<kTree> walk;
  // (no more ranges than tiles: between two CTAs of an item there is none without a part)
  const int ranges = (int)min((long long)gridDim.x, total);
  walk.pos = walk.end = 0;
  if ((int)blockIdx.x < ranges) {
    walk.pos = (int64_t)blockIdx.x * total / ranges;
    walk.end = (int64_t)(blockIdx.x + 1) * total / ranges;
  }
  if (walk.pos < walk.end) {
    long long before = 0;
    for (int n0 = 0; n0 < N; n0 += kThreads) {
      const long long w = n0 == 0 ? first : cost(n0 + tid, false);
      long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 31) misc->part[warp] = inc;
      __syncthreads();
      long long off = before;
      for (int x = 0; x < warp; ++x) off += misc->part[x];
      if (w > 0 && walk.pos >= off + inc - w && walk.pos < off + inc) {
        misc->start_n = n0 + tid;
        misc->start_base = off + inc - w;
      }
      for (int x = 0; x < kThreads / 32; ++x) before += misc->part[x];
      __syncthreads();
      if (before > walk.pos) break;
    }
    walk.n = misc->start_n;
    walk.base = misc->start_base;
    walk.n0 = walk.n;
    walk.cache = reinterpret_cast<const SeqInfo*>(sm + C::kOffSeq);
    if (tid < kCached && walk.n + tid < N) {
      int err;
      reinterpret_cast<SeqInfo*>(sm + C::kOffSeq)[tid] =
          seq_info<kTree>(p.a, walk.n + tid, p.min_rows, p.max_rows, &err);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  if (walk.pos < walk.end) walk.s = walk.cache[0];

  if (warp == 4) {
    // ================= producer: pages of each tile, K and V of one head
    // A tile's pages are looked up two tiles ahead and its scales one, over the segments' ends.
    uint32_t it = 0;
    bool ok = true;
    const int boxes = kTile / P;                         // pages of a tile
    struct Ahead {
      int h, pg;
      bool more, load;   // more: there is such a tile; load: this lane fetches page pg of it
    };
    int t = 0;
    bool in_seg = false;
    auto look = [&]() -> Ahead {
      if (!in_seg || t >= walk.b) {
        in_seg = walk.next(p);
        if (!in_seg) return {0, 0, false, false};
        t = walk.a;
      }
      const int b = (walk.s.tile0 + t++) * boxes + lane;
      // (a page wholly before every query's window is not looked up: its entry may be stale)
      if (lane >= boxes || b >= (walk.s.len + P - 1) / P ||
          (b + 1) * P <= first_seen(low_pos<kTree>(walk.s.len - walk.s.q_len), p.a.window))
        return {walk.h, 0, true, false};
      return {walk.h, p.a.c.block_table[walk.n * p.a.c.table_stride + b], true, true};
    };
    float ks = 1.0f, vs = 1.0f;
    auto scales = [&](Ahead& x) {
      ks = vs = 1.0f;
      if (!x.load) return;
      if (x.pg < 0 || x.pg >= p.a.c.num_pages) {
        record_error(p.a.status, KDA_ERR_BAD_CACHE_INDEX, 312);
        x.pg = p.a.c.num_pages;                          // outside the map: the load gives zeros
        return;
      }
      ks = p.a.c.k_scale[(int64_t)x.pg * p.a.c.scale_stride + x.h];
      vs = p.a.c.v_scale[(int64_t)x.pg * p.a.c.scale_stride + x.h];
    };
    Ahead cur = look(), nxt = {0, 0, false, false};
    if (cur.more) {
      scales(cur);
      nxt = look();
    }
    for (; cur.more; ++it) {
      const uint32_t st = it % kStages;
      const float ks_now = ks, vs_now = vs;
      Ahead after = {0, 0, false, false};
      if (nxt.more) {
        scales(nxt);
        after = look();
      }
      if (it >= kStages) ok = mbar_wait_sleep(bar_empty + 8 * st, (it / kStages - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 313);
        break;
      }
      const uint32_t dst = sb + st * kStageBytes;
      if (lane < boxes) {
        float* sc = reinterpret_cast<float*>(sm + C::kOffScale + st * 64);
        sc[lane] = ks_now;
        sc[8 + lane] = vs_now > 0.0f ? vs_now : NAN;
      }
      const uint32_t loads = __popc(__ballot_sync(0xffffffffu, cur.load));
      __syncwarp();
      if (lane == 0) mbar_expect_tx(bar_full + 8 * st, loads * 2 * P * kHeadDim);
      __syncwarp();
      if (cur.load) {
        tma_load_4d(dst + lane * P * 128, &p.maps.k, 0, 0, cur.h, cur.pg, bar_full + 8 * st);
        tma_load_4d(dst + kTile * 128 + lane * P * 128, &p.maps.v, 0, 0, cur.h, cur.pg, bar_full + 8 * st);
      }
      cur = nxt;
      nxt = after;
    }
    // the copies in flight end before the CTA does
    for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
      mbar_wait_sleep(bar_full + 8 * (i % kStages), (i / kStages) & 1);
  } else if (warp == 5) {
    // ================= MMA issuer
    if (elect_one()) {
      constexpr uint32_t id_s = idesc_e4m3(128, C::kN, 0, 0), id_o = idesc_e4m3(128, C::kN, 1, 0);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      auto pv = [&](uint32_t i) {       // O^T of tile i, once its P is written
        ok = mbar_wait_sleep(bar_p, i & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t v = sb + (i % kStages) * kStageBytes + kTile * 128;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_e4m3(tmem + C::kTO, mnmajor8(v, ks), kmajor8(sb + C::kOffP, ks), id_o, ks > 0);
        mma_commit(bar_o);
        mma_commit(bar_empty + 8 * (i % kStages));
      };
      while (ok && walk.next(p)) {
        ok = mbar_wait_sleep(bar_q, seg & 1);
        ++seg;
        for (int t = walk.a; t < walk.b && ok; ++t, ++it) {
          ok = mbar_wait_sleep(bar_full + 8 * (it % kStages), (it / kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k = sb + (it % kStages) * kStageBytes;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_e4m3(tmem + (it & 1) * C::kN, kmajor8(k, ks), kmajor8(sb + C::kOffQ, ks), id_s, ks > 0);
          mma_commit(bar_s + 8 * (it & 1));
          if (t > walk.a) pv(it - 1);
        }
        if (ok) pv(it - 1);
      }
      if (!ok) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 314);
      // what was issued ends, its arrivals included, before shared and tensor memory go
      mma_commit(bar_end);
      mbar_wait_sleep(bar_end, 0);
      for (uint32_t i = it > kStages ? it - kStages : 0; ok && i < it; ++i)
        mbar_wait_sleep(bar_empty + 8 * (i % kStages), (i / kStages) & 1);
    }
    __syncwarp();
  } else {
    // ================= softmax and accumulation: thread = key of S^T, channel of O^T
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    float4* fac = reinterpret_cast<float4*>(sm + C::kOffFac);     // [2][4][NR]: max, f1, f2
    float* wmax = reinterpret_cast<float*>(sm + C::kOffMax);      // [2][NR][4]
    float* sums = reinterpret_cast<float*>(sm + C::kOffSum);
    uint4* poison = reinterpret_cast<uint4*>(sm + C::kOffPoison);
    float* qmul = reinterpret_cast<float*>(sm + C::kOffQmul);
    const Cap cap = kCap ? cap_of(p.a.softcap) : Cap{0.0f, 0.0f};
    const float to_e = 2.0f * kLog2e * cap.inv;
    PartDesc part = {0, 0, 0, 0};
    uint32_t it = 0;
    // A wait that gives up clears its thread's `ok`; the thread leaves with the others, at a barrier
    // that has told them.
    bool ok = true;
    uint4 qraw[NR / 8];     // this thread's part of the next segment's queries, 16 lanes a row
    auto load_q = [&](const Walk<kTree>& w) {
#pragma unroll
      for (int i = 0; i < NR / 8; ++i) {
        const int r = 8 * i + (tid >> 4);
        qraw[i] = make_uint4(0, 0, 0, 0);
        const int t = div_small(r, gm);
        if (r < w.s.q_len * G)
          qraw[i] = *reinterpret_cast<const uint4*>(p.a.q + (int64_t)(w.s.tok0 + t) * p.a.q_stride +
                                                    (w.h * G + r - t * G) * kHeadDim + 8 * (tid & 15));
      }
    };
    bool more = walk.next(p);
    if (more) load_q(walk);
    while (more) {
      const int rows = walk.s.q_len * G;
      const int first_pos = walk.s.len - walk.s.q_len;   // position of query 0
      // ---- queries: two e4m3 terms each, 16 lanes a row
#pragma unroll
      for (int r0 = 0; r0 < NR; r0 += 8) {
        const int r = r0 + (tid >> 4), c = tid & 15;
        float x[8];
        float top = 0.0f;
        unpack8(qraw[r0 / 8], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        // a power of two that brings the row's largest entry into (224, 448]
        const int e2 = (int)((__float_as_uint(top) >> 23) & 255) - 127 - 8 +
                       ((__float_as_uint(top) & 0x7fffffu) > 0x600000u ? 1 : 0);
        const int e2c = max(e2, -100);
        const float inv = __uint_as_float((uint32_t)(127 - e2c) << 23);
        uint32_t t1[4], t2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_e4m3x2(x[2 * e] * inv, x[2 * e + 1] * inv, t1[e], t2[e]);
        const uint32_t w1[2] = {t1[0] | (t1[1] << 16), t1[2] | (t1[3] << 16)};
        const uint32_t w2[2] = {t2[0] | (t2[1] << 16), t2[2] | (t2[3] << 16)};
        *reinterpret_cast<uint2*>(sm + C::kOffQ + tile_off(r, 8 * c)) = make_uint2(w1[0], w1[1]);
        *reinterpret_cast<uint2*>(sm + C::kOffQ + tile_off(NR + r, 8 * c)) = make_uint2(w2[0], w2[1]);
        if (c == 0) {   // a non-finite query makes its row NaN
          const float sq = top <= 3.402823466e38f ? __uint_as_float((uint32_t)(127 + e2c) << 23) : NAN;
          qmul[r] = sq * p.a.scale * kLog2e;
        }
      }
      fence_proxy_async();
      mbar_arrive(bar_q);
      if (bar_any(1, 128, !ok)) { ok = false; break; }   // qmul is written (and nobody gave up)
      // a tree's masks: lane i that of node i (there are at most 32)
      const uint32_t nodes =
          kTree && lane < walk.s.q_len
              ? (uint32_t)(p.a.tree[walk.s.tok0 + lane] & node_bits(walk.s.q_len)) : 0;
      Walk<kTree> ahead = walk;
      more = ahead.next(p);
      if (more) load_q(ahead);

      float acc[NR], l[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[r] = l[r] = 0.0f;
      float run = -INFINITY;         // lane r: running maximum of row r
      bool poisoned = false;         // the tile before has NaN entries that some rows do not see
      bool left = false;             // somebody's wait gave up: all 128 threads leave
      // O^T of tile i added to the sums (its factors and poison words: parity i & 1)
      auto add_o = [&](uint32_t i, int t) {
        ok = mbar_wait_sleep(bar_o, i & 1) && ok;
        __syncwarp();
        tc_fence_after();
        const float4* f = fac + ((i & 1) * 4 + warp) * NR;
        if (NR <= 16) {
          uint32_t o[C::kN <= 16 ? 16 : 32];
          if constexpr (C::kN <= 16) tmem_ld16(tmem + lane_base + C::kTO, o);
          else tmem_ld32(tmem + lane_base + C::kTO, o);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float4 c = f[r];
            acc[r] = acc[r] * c.y + (__uint_as_float(o[r]) + __uint_as_float(o[NR + r])) * c.z;
          }
        } else {
#pragma unroll
          for (int q = 0; q < NR; q += 16) {
            uint32_t o1[16], o2[16];
            tmem_ld16(tmem + lane_base + C::kTO + q, o1);
            tmem_ld16(tmem + lane_base + C::kTO + NR + q, o2);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const float4 c = f[q + r];
              acc[q + r] = acc[q + r] * c.y + (__uint_as_float(o1[r]) + __uint_as_float(o2[r])) * c.z;
            }
          }
        }
        if (poisoned) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(poison + (i & 1) * 128);
          for (int x = 0; x < kTile; ++x) {
            if (!((w[4 * x + warp] >> lane) & 1)) continue;
            const int key = (walk.s.tile0 + t) * kTile + x;
            uint32_t seen = 0;      // of a tree: the nodes that see this key
            if (kTree) {
#pragma unroll 1
              for (int i = 0; i < walk.s.q_len; ++i) {
                const uint64_t w = p.a.tree[walk.s.tok0 + i] & node_bits(walk.s.q_len);
                seen |= (uint32_t)tree_sees(w, __popcll(w), key, first_pos, walk.s.len, p.a.window) << i;
              }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const int i = div_small(r, gm), pos = first_pos + i;
              if (kTree ? (seen >> i) & 1 : key <= pos && (p.a.window <= 0 || key > pos - p.a.window))
                acc[r] = NAN;
            }
          }
          // all have read these words before anyone writes the next ones of this parity: S of the
          // tile after this one is there already, so nothing else would hold a fast warp back
          group_sync(2, 128);
        }
      };
      for (int t = walk.a; t < walk.b; ++t, ++it) {
        const uint32_t par = it & 1, st = it % kStages;
        // (the scales and V are read here too; S comes last)
        ok = mbar_wait_sleep(bar_full + 8 * st, (it / kStages) & 1) && ok;
        ok = mbar_wait_sleep(bar_s + 8 * par, (it >> 1) & 1) && ok;
        __syncwarp();
        tc_fence_after();
        const int key0 = (walk.s.tile0 + t) * kTile, key = key0 + tid;
        // some key of the tile is hidden from some row
        const bool masked = key0 + kTile - 1 > low_pos<kTree>(first_pos) ||
                            (p.a.window > 0 && key0 <= walk.s.len - 1 - p.a.window);
        const float* sc = reinterpret_cast<const float*>(sm + C::kOffScale + st * 64);
        float ks = 1.0f, vs = 1.0f;
        if (key < walk.s.len) {
          ks = sc[tid / P];
          vs = sc[8 + tid / P];
        }
        const float lvs = lg2(vs);
        float ivs = __fdividef(1.0f / kPScale, vs);
        float x[NR];
        if (NR <= 16) {
          uint32_t o[C::kN <= 16 ? 16 : 32];
          if constexpr (C::kN <= 16) tmem_ld16(tmem + lane_base + par * C::kN, o);
          else tmem_ld32(tmem + lane_base + par * C::kN, o);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = __uint_as_float(o[r]) + __uint_as_float(o[NR + r]);
        } else {
#pragma unroll
          for (int q = 0; q < NR; q += 16) {
            uint32_t o1[16], o2[16];
            tmem_ld16(tmem + lane_base + par * C::kN + q, o1);
            tmem_ld16(tmem + lane_base + par * C::kN + NR + q, o2);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < 16; ++r) x[q + r] = __uint_as_float(o1[r]) + __uint_as_float(o2[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(qmul + r);
          const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) x[r + e] = kCap ? x[r + e] * (m[e] * ks) : x[r + e] * (m[e] * ks) + lvs;
        }
        if (kCap == kCapPlain) {
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = cap_plain(x[r], to_e, cap, lvs);
        } else if (kCap == kCapExact) {
          float top = 0.0f;
#pragma unroll
          for (int r = 0; r < NR; r += 2) top = max3_abs(top, x[r], x[r + 1]);
          const float2 add = make_float2(lvs, lvs);
          if (__any_sync(0xffffffffu, top * cap.inv >= kCapSmall)) {
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
              const float2 y = cap_any(make_float2(x[r], x[r + 1]), cap, add);
              x[r] = y.x;
              x[r + 1] = y.y;
            }
          } else {
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
              const float2 y = cap_small(make_float2(x[r], x[r + 1]), cap, add);
              x[r] = y.x;
              x[r + 1] = y.y;
            }
          }
        }
        bool hidden_nan = false;
        if (masked) {
          if (!(vs > 0.0f)) ivs = 0.0f;   // (a page without a scale: NaN to the rows that see it only)
          bool all = true, any = false;
          uint32_t seen = 0;        // of a tree: the nodes that see this key
          for (int i = 0; i < walk.s.q_len; ++i) {
            bool see;
            if (kTree) {
              const uint32_t w = __shfl_sync(0xffffffffu, nodes, i);
              see = tree_sees(w, __popc(w), key, first_pos, walk.s.len, p.a.window);
              seen |= (uint32_t)see << i;
            } else {
              const int pos = first_pos + i;
              see = key <= pos && (p.a.window <= 0 || key > pos - p.a.window);
            }
            all = all && see;
            any = any || see;
          }
          unsigned char* vrow = sm + st * kStageBytes + kTile * 128 + (tid >> 3) * 1024 + (tid & 7) * 128;
          if (!any) {
#pragma unroll
            for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(vrow)[c] = make_uint4(0, 0, 0, 0);
          }
          if (walk.s.q_len > 1) {   // NaN channels of a row that some queries see and others do not
            uint32_t bits[4] = {0, 0, 0, 0};
            if (any && !all) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint4* chunk = reinterpret_cast<uint4*>(vrow) + (c ^ (tid & 7));
                const uint4 u = *chunk;
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                uint32_t nan[4], some = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  nan[e] = __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  some |= nan[e];
#pragma unroll
                  for (int b = 0; b < 4; ++b)
                    bits[c >> 1] |= ((nan[e] >> (8 * b)) & 1u) << (16 * (c & 1) + 4 * e + b);
                }
                if (some) *chunk = make_uint4(w[0] & ~nan[0], w[1] & ~nan[1], w[2] & ~nan[2], w[3] & ~nan[3]);
              }
            }
            poison[par * 128 + tid] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
            hidden_nan = (bits[0] | bits[1] | bits[2] | bits[3]) != 0;
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const int i = div_small(r, gm), pos = first_pos + i;
            const bool see = kTree ? (seen >> i) & 1
                                   : key <= pos && (p.a.window <= 0 || key > pos - p.a.window);
            if (!see) x[r] = -INFINITY;
          }
        }
        // ---- the tile's maxima: the warp's by redux, the four warps' through shared memory
        float mine_max = -INFINITY;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float m = warp_max(x[r]);
          if (lane == r) mine_max = m;
        }
        if (lane < NR) wmax[(par * NR + lane) * 4 + warp] = mine_max;
        left = bar_any(1, 128, !ok);
        if (left) break;
        if (lane < NR) {
          const float4 w = *reinterpret_cast<const float4*>(wmax + (par * NR + lane) * 4);
          const float m = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
          const float next = fmaxf(run, m), ref = next == -INFINITY ? 0.0f : next;
          fac[(par * 4 + warp) * NR + lane] =
              make_float4(m == -INFINITY ? 0.0f : m, ex2(run - ref), ex2(m - ref) * (1.0f / kPScale), 0.0f);
          run = next;
        }
        const bool poison_now = masked && walk.s.q_len > 1 && bar_any(2, 128, hidden_nan);
        __syncwarp();
        // ---- numerators and denominators
        const float4* f = fac + (par * 4 + warp) * NR;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float4 c = f[r];
          x[r] = ex2(x[r] - c.x) * kPScale;
          l[r] = l[r] * c.y + x[r] * (ivs * kPScale) * c.z;
        }
        // ---- O of the tile before, whose P operand this one replaces
        if (t > walk.a) add_o(it - 1, t - 1);
        poisoned = poison_now;
        unsigned char* pt = sm + C::kOffP;
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          const uint32_t q1 = e4m3x2(x[r], x[r + 1]);
          const float2 b = from_e4m3x2(q1);
          const uint32_t q2 = e4m3x2(x[r] - b.x, x[r + 1] - b.y);
          pt[tile_off(r, tid)] = (unsigned char)q1;
          pt[tile_off(r + 1, tid)] = (unsigned char)(q1 >> 8);
          pt[tile_off(NR + r, tid)] = (unsigned char)q2;
          pt[tile_off(NR + r + 1, tid)] = (unsigned char)(q2 >> 8);
        }
        tc_fence_before();
        fence_proxy_async();
        mbar_arrive(bar_p);
      }
      if (left) { ok = false; break; }
      add_o(it - 1, walk.b - 1);
      // ---- denominators over the 128 key threads
      // (each step exchanges half of the rows: after log2 NR steps a lane holds row lane * NR / 32)
#pragma unroll
      for (int o = 16, n = NR / 2; o > 0; o >>= 1, n >>= 1) {
        if (n >= 1) {
#pragma unroll
          for (int k = 0; k < n; ++k) {
            const float keep = (lane & o) ? l[k + n] : l[k], send = (lane & o) ? l[k] : l[k + n];
            l[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        }
      }
      if (lane % (32 / NR) == 0) sums[(lane / (32 / NR)) * 4 + warp] = l[0];
      if (bar_any(1, 128, !ok)) { ok = false; break; }
      float den = 0.0f;     // lane r: row r's, the same in every warp
      if (lane < NR) {
        const float4 q = *reinterpret_cast<const float4*>(sums + 4 * lane);
        den = (q.x + q.y) + (q.z + q.w);
      }
      if (walk.a == 0 && walk.b == walk.s.tiles) {   // the whole item: its rows of out and lse
        const float inv_l = den == 0.0f ? 0.0f : 1.0f / den;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float il = __shfl_sync(0xffffffffu, inv_l, r);
          if (r < rows) {
            const int i = div_small(r, gm);
            p.a.out[(int64_t)(walk.s.tok0 + i) * p.a.out_stride + (walk.h * G + r - i * G) * kHeadDim + tid] =
                __float2bfloat16_rn(acc[r] * il);
          }
        }
        if (p.a.lse && warp == 0 && lane < rows) {
          const int i = div_small(lane, gm);
          p.a.lse[(int64_t)(walk.s.tok0 + i) * p.a.heads + walk.h * G + lane - i * G] =
              den == 0.0f ? -INFINITY : (run + lg2(den)) * kLn2;
        }
      } else {
        // slot 0: an item that an earlier CTA began; slot 1: one that this CTA begins
        const bool begins = walk.a == 0;
        float* slot = p.slots + ((int64_t)2 * blockIdx.x + (begins ? 1 : 0)) * kSlotFloats<NR>;
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (r < rows) slot[r * 128 + tid] = acc[r];
        if (warp == 0 && lane < rows) {
          slot[NR * 128 + lane] = run;
          slot[NR * 129 + lane] = den;
        }
        if (begins) {   // the CTA that its last tile lies in, from the cut of the ranges
          const int64_t last = walk.unit_of(walk.s.tiles - 1);
          const int64_t c = ((last + 1) * ranges - 1) / total;
          part.tok0 = walk.s.tok0;
          part.rows = rows;
          part.head0 = walk.h * G;
          part.parts = (int)(c - blockIdx.x) + 1;
        }
      }
      walk = ahead;
    }
    if (!ok && tid == 0) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 315);
    if (!ok) part.parts = 0;
    if (tid == 0) p.desc[blockIdx.x] = part;
  }
  // (beside the prefill kernel: this grid does not end before that one)
  if (blockIdx.x == 0 && warp == 0) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merges the parts of the items that two CTAs of the first kernel began and did not finish: sums and
// denominators by their maxima, in a fixed order.  Eight warps a CTA take NR / 8 rows; as many of
// a row's warps as have work take its parts in turn, 4 channels a lane, four parts in flight.  (One
// sequence of 65536 tokens leaves 76 parts an item: a chain of loads per part would cost more
// than reading the cache.)  Two neighbours' items, since where items have many parts
// only one of them begins any: so all CTAs run at once.
constexpr int kMergeWarps = 8, kInFlight = 4;
template <int NR>
__global__ void __launch_bounds__(32 * kMergeWarps)
    kda_attn_merge_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kPerRow = 64 / NR;     // warps of a row
  __shared__ float4 acc_s[kMergeWarps][32];
  __shared__ float2 ml_s[kMergeWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int4* desc = reinterpret_cast<const int4*>(p.desc + 2 * blockIdx.x);
  const int4 both[2] = {desc[0], desc[1]};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % kPerRow;
  const int r = blockIdx.y * (NR / 8) + warp / kPerRow;
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int4 d4 = j ? both[1] : both[0];
    const PartDesc d = {d4.x, d4.y, d4.z, d4.w};
    if (d.parts == 0) continue;
    const int cta = 2 * blockIdx.x + j;
    const int used = min(kPerRow, (d.parts + kInFlight - 1) / kInFlight);   // warps of a row with work
    const bool live = r < d.rows && w0 < used;
    float m = -INFINITY, den = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // four parts merged into the running maximum, sum and denominator
    auto merge = [&](const float (&mi)[kInFlight], const float (&di)[kInFlight], const float4 (&ai)[kInFlight]) {
      float top = m;
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) top = fmaxf(top, mi[u]);
      const float ref = top == -INFINITY ? 0.0f : top, f = ex2(m - ref);
      m = top;
      den *= f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const float w = ex2(mi[u] - ref);
        den += di[u] * w;
        acc.x += ai[u].x * w;
        acc.y += ai[u].y * w;
        acc.z += ai[u].z * w;
        acc.w += ai[u].w * w;
      }
    };
    if (live) {
      for (int i0 = w0; i0 < d.parts; i0 += used * kInFlight) {
        float mi[kInFlight], di[kInFlight];
        float4 ai[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const int i = i0 + u * used;
          const float* s = p.slots + ((int64_t)2 * (cta + i) + (i == 0 ? 1 : 0)) * kSlotFloats<NR>;
          mi[u] = -INFINITY;
          di[u] = 0.0f;
          ai[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < d.parts) {
            mi[u] = s[NR * 128 + r];
            di[u] = s[NR * 129 + r];
            ai[u] = *reinterpret_cast<const float4*>(s + r * 128 + 4 * lane);
          }
        }
        merge(mi, di, ai);
      }
    }
    if (used > 1) {
      __syncthreads();     // (the item before has been read)
      acc_s[warp][lane] = acc;
      if (lane == 0) ml_s[warp] = make_float2(m, den);
      __syncthreads();
    }
    if (w0 != 0 || !live) continue;
    for (int w = 1; w < used; w += kInFlight) {
      float mi[kInFlight], di[kInFlight];
      float4 ai[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const bool in = w + u < used;
        const float2 ml = in ? ml_s[warp + w + u] : make_float2(-INFINITY, 0.0f);
        mi[u] = ml.x;
        di[u] = ml.y;
        ai[u] = in ? acc_s[warp + w + u][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      merge(mi, di, ai);
    }
    const float il = den == 0.0f ? 0.0f : 1.0f / den;
    const int i = div_small(r, p.group_magic);
    const int64_t tok = d.tok0 + i;
    const int head = d.head0 + r - i * p.group;
    *reinterpret_cast<uint2*>(p.a.out + tok * p.a.out_stride + head * kHeadDim + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * il, acc.y * il), pack_bf16x2(acc.z * il, acc.w * il));
    if (p.a.lse && lane == 0)
      p.a.lse[tok * p.a.heads + head] = den == 0.0f ? -INFINITY : (m + lg2(den)) * kLn2;
  }
}

int decode_ctas(int sms) { return 2 * sms; }

template <int NR, int kCap, bool kTree>
cudaError_t launch_nr(const DecodeParams& d, int sms, cudaStream_t stream) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&]() -> cudaError_t {
    return cudaFuncSetAttribute(kda_attn_decode_kernel<NR, kCap, kTree>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NR>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch(kda_attn_decode_kernel<NR, kCap, kTree>, dim3((unsigned)decode_ctas(sms)), dim3(kThreads),
                Cfg<NR>::kBytes, true, stream, d);
}
template <int NR, bool kTree>
cudaError_t launch_cap(const DecodeParams& d, int sms, cudaStream_t stream) {
  switch (cap_kind(d.a.softcap)) {
    case kNoCap: return launch_nr<NR, kNoCap, kTree>(d, sms, stream);
    case kCapPlain: return launch_nr<NR, kCapPlain, kTree>(d, sms, stream);
    default: return launch_nr<NR, kCapExact, kTree>(d, sms, stream);
  }
}
template <int NR>
cudaError_t launch_mask(const DecodeParams& d, int sms, cudaStream_t stream) {
  return d.a.tree ? launch_cap<NR, true>(d, sms, stream) : launch_cap<NR, false>(d, sms, stream);
}
template <int NR>
cudaError_t launch_merge(const DecodeParams& d, int sms, cudaStream_t stream) {
  return launch(kda_attn_merge_kernel<NR>, dim3((unsigned)(decode_ctas(sms) / 2), 8), dim3(32 * kMergeWarps),
                0, true, stream, d);
}

}  // namespace

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool make_cache_maps(const CacheView& c, CacheMaps* m) {
  EncodeTiled enc = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride,
                                 (cuuint64_t)c.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)kHeadDim, (cuuint32_t)c.page_size, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (enc(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? c.v : c.k, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

size_t decode_workspace_bytes(int sms) {
  const size_t ctas = (size_t)decode_ctas(sms);
  return ctas * sizeof(PartDesc) + ctas * 2 * kSlotFloats<32> * sizeof(float);
}

namespace {
void make_params(const AttnParams& a, int max_rows, int gate, void* work, int sms, DecodeParams* d) {
  d->a = a;
  d->gate = gate;
  d->least = 0;
  d->group = a.heads / a.c.kv_heads;
  d->group_magic = 65535u / (uint32_t)d->group + 1;
  d->min_rows = 1;
  d->max_rows = max_rows;
  d->desc = static_cast<PartDesc*>(work);
  d->slots = reinterpret_cast<float*>(d->desc + decode_ctas(sms));
}
}  // namespace

// The operands are padded to 8, 16 or 32 rows.
cudaError_t launch_attn_decode(const AttnParams& a, const CacheMaps& maps, int max_rows, int64_t least,
                               int gate, void* work, int sms, cudaStream_t stream) {
  DecodeParams d;
  make_params(a, max_rows, gate, work, sms, &d);
  d.maps = maps;
  d.least = least;
  return max_rows <= 8 ? launch_mask<8>(d, sms, stream) : max_rows <= 16 ? launch_mask<16>(d, sms, stream)
                                                                      : launch_mask<32>(d, sms, stream);
}

cudaError_t launch_attn_decode_merge(const AttnParams& a, int max_rows, void* work, int sms,
                                     cudaStream_t stream) {
  DecodeParams d = {};
  make_params(a, max_rows, 0, work, sms, &d);
  return max_rows <= 8    ? launch_merge<8>(d, sms, stream)
         : max_rows <= 16 ? launch_merge<16>(d, sms, stream)
                          : launch_merge<32>(d, sms, stream);
}

}  // namespace attn
}  // namespace kda
