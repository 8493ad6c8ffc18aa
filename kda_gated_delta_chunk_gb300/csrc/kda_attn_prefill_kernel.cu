// Attention over the paged e4m3 cache for many query rows (prefill, long verifies): the rows --
// new tokens x query heads of one kv head, token-major -- are cut into tiles of up to 256 (whole
// tokens), two halves A and B of 128 rows that share the stream of key tiles:
//   S   = q1 K8^T + q2 K8^T   e4m3 on tcgen05, the cache's keys as they lie in memory; a bf16
//                             query is two e4m3 terms (exact to 2^-18 of its row's largest entry,
//                             at the tensor time of one bf16 product)
//   P   = 2^(s + log2 v_scale(page) - m)   two threads a row, written as f16 over S in tensor memory
//   O  += P V                 f16 on tcgen05, P from tensor memory, V widened to f16 by four
//                             warps (an e4m3 value is exact in f16; page scales are in P)
// The row maximum m is brought up only when it grows by more than 2^8, so O is rescaled rarely, and a
// tile's P is computed by the standing m while its own maximum is found; a tile that raises m is
// read again (371 -> 348 us against waiting for the maximum first, at the size below).
// Numerators are 2^7 at the maximum, 2^15 with that slack: f16 then keeps 11 bits down to 2^-21 of
// the maximum and rounds to 2^-31 of it, against bf16's 8 bits.  The denominators take the fp32
// numerators, divided by the page's value scale.
//
// Bound by the tensor cores: 4 x 128 flops per visible (row, key).  4096 tokens at the end of 16384,
// 16 heads over 2: 326.6 us, 1473 TFLOP/s; 289 us with the softmax left out.  With capped scores
// 597 us (three special functions a score; caps above 64 585: nine fp32 operations and one), and a
// tile's maximum before its numerators.  Two halves keep the tensor cores busy: while one half's
// softmax runs, the other half's products do.  The matrix instructions of a CTA
// run in the order they are issued, so S(i+1) of a half may follow its O += P(i) V, whose P it
// overwrites, without a wait.  Key tiles of all (sequence, kv head, row tile) items are laid end
// to end and cut into one equal range per CTA, one CTA per SM (as in the decode kernel; an item
// counts kOver tiles more), and a dependent kernel merges the items that were cut.
//
// Warps: 0-7 / 8-15 softmax of the halves, 16-19 the widening of V, 20 the TMA producer, 21 the MMA
// issuer, 22 the scheduler, which walks the CTA's range and hands its segments to the others
// through a ring in shared memory (23 only gives its registers).  Every wait is bounded.
//
// Masked entries as in the decode kernel: pages before every window are not read, scores by selection,
// V rows that no row of the tile sees as zeros, and a NaN in a V row that only some rows see as zero,
// put back into those rows at the end from the cache itself.
//
// Trees of drafted tokens: what a row sees among the new tokens are the bits of its node's mask, shifted to the
// thread's 64 keys; everything else is as above, and 4 sequences of 64 nodes over 65536 keys, 32 heads over 4,
// take 204 us (1346 TFLOP/s).  Where trees fill half of a row tile or less, the second half would work on
// nothing: there a row tile has 128 rows, and the two halves take its key tiles in turns (even ones A, odd
// ones B), each with a maximum, a denominator and an O of its own, which A merges at the end.  Half as long a
// tile wants more of what feeds it: a producer warp for values beside the one for keys, four places for V,
// and four warps a half to widen it.  16 sequences of 16 nodes over up to 16384 keys, 32 heads over 8: 83 us
// (2.8 TB/s), side by side 104; 8 sequences over 65536, pages of 128, 243 us (4.4 TB/s).  Neither memory (35%)
// nor the tensor cores (27%) bound it but the chain of a half's tile (S, softmax, P, O: 4400 cycles), and at
// the size above two changes of item a CTA, 9 us each.  Measured and not kept: P as two e4m3 terms and V as it
// lies in memory (90 us: the conversions), a third place for widened V in that of two for V (84), the next
// item's queries made by half B while A writes (91).
#include "kda_attn_tc.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kThreadsP = 768, kThreadsTurns = 896;     // (in turns two groups of V warps)
constexpr int kRowsP = 256;
constexpr int kKStages = 3, kVStages = 2, kSegs = 4;
constexpr int kSoftWarps = 16, kRegsSoftmax = 104, kRegsOther = 32;
constexpr int kRegsNeeded = 32 * (kSoftWarps * kRegsSoftmax + (kThreadsP / 32 - kSoftWarps) * kRegsOther);
constexpr int kRegsSoftmaxTurns = 96, kRegsOtherTurns = 40;
constexpr int kRegsNeededTurns =
    32 * (kSoftWarps * kRegsSoftmaxTurns + (kThreadsTurns / 32 - kSoftWarps) * kRegsOtherTurns);
constexpr float kSlack = 8.0f;              // log2 growth of the maximum before O is rescaled
constexpr float kPShift = 7.0f;             // log2 of the numerator at the maximum: at most 2^15 with the slack

// shared memory, from a 1024-byte aligned base
constexpr int kOffQ = 0;                                    // [half][term] 128 x 128 e4m3
constexpr int kOffVB = kOffQ + 4 * 16384;                   // [2] V as f16, two 64-channel blocks
constexpr int kOffK = kOffVB + 2 * 32768;                   // [kKStages] K tiles
constexpr int kOffV8 = kOffK + kKStages * 16384;            // [kVStages] V tiles
constexpr int kOffSc = kOffV8 + kVStages * 16384;           // float4 [4 or 8][8]: k scale, log2 v scale, 1 / v scale
constexpr int kOffQmul = kOffSc + 8 * 8 * 16;               // float [256]
constexpr int kOffMx = kOffQmul + 4 * kRowsP;               // float [2][2][256]: maxima of a row's two threads
constexpr int kOffL = kOffMx + 16 * kRowsP;                 // float [256][2]: denominators
constexpr int kOffSeg = kOffL + 8 * kRowsP;                 // Segment [kSegs]
constexpr int kOffBars = kOffSeg + 64 * 4;
constexpr int kNumBars = 2 * kKStages + 2 * 4 + 2 * 7 + 8 + 2 * kSegs;
constexpr int kOffMiscP = kOffBars + 8 * kNumBars;
constexpr int kSmemP = kOffMiscP + 448 + 1024;
static_assert(kSmemP <= 227 * 1024, "shared memory");

// tensor memory columns
constexpr uint32_t kTS = 0, kTOP = 256;     // S (P) of half h at 128 h, O at 256 + 128 h

// named barriers beside the pairs' (1-8) and the halves' (9, 10)
constexpr uint32_t kIdBoth = 11, kIdMerge = 12;

constexpr int kSlotFloatsP = kRowsP * 130;

struct PartDescP {
  int parts;          // CTAs whose parts make up the item that this CTA begins; 0: none is cut
  int tok0, rows;     // its first token's row of q and out, its query rows
  int head0;          // its first query head
};

// What a launch works on: causal rows; the nodes of trees; the same in row tiles of 128, both halves taking the
// key tiles of one row tile in turn (even ones half A, odd ones half B).
enum { kCausal = 0, kNodesWide = 1, kNodesTurns = 2 };

struct PrefillParams {
  AttnParams a;
  CacheMaps maps;
  int group;                 // query heads of a kv head
  uint32_t group_magic;      // 65535 / group + 1 (div_small)
  int gate;                  // the call's number, when the decode kernel runs beside this one; else 0
  int few, tokens;           // rows of the decode kernel's sequences at most; new tokens per row tile (256 or 128 / group)
  int64_t least;             // units of those below which this kernel takes them too
  PartDescP* desc;
  float* slots;
};

// Row tile rt of a sequence: its tokens, and the key tiles they see.
struct ItemP {
  int tok, cnt;              // tokens [tok, tok + cnt) of the sequence's new ones
  int tile0, tiles;
};
template <bool kTree>
__device__ __forceinline__ ItemP item_of(int q_len, int len, int rt, int tokens, int window) {
  ItemP it;
  it.tok = rt * tokens;
  it.cnt = min(tokens, q_len - it.tok);
  const int p_first = kTree ? low_pos<true>(len - q_len) : len - q_len + it.tok;
  const int p_last = kTree ? len - 1 : p_first + it.cnt - 1;
  it.tile0 = first_seen(p_first, window) / kTile;
  it.tiles = max(1, (max(p_last, -1) + kTile) / kTile - it.tile0);
  return it;
}

// The walk over a CTA's range, in units: an item has kOver of them, then one per key tile.
template <bool kTree>
struct WalkP {
  int64_t pos, end;
  int n, h, rt, off;         // the next item and the units of it that lie before this range
  int min_rows;              // sequences of fewer rows are the decode kernel's
  SeqInfo s;
  ItemP it;
  int a, b;                  // segment: tiles [a, b) of the item
  int ch;                    // its head
  int64_t last;              // unit of the item's last tile
  __device__ __forceinline__ bool next(const PrefillParams& p) {
    while (pos < end) {
      while (s.tiles == 0 || rt * p.tokens >= s.q_len) {   // to the next head or sequence
        if (s.tiles != 0 && h + 1 < p.a.c.kv_heads) {
          ++h;
          rt = 0;
          continue;
        }
        int err;
        if (++n >= p.a.num_seqs) return false;             // (lengths that changed under the kernel)
        s = seq_info<kTree>(p.a, n, min_rows, 0x7fffffff, &err);
        h = rt = 0;
      }
      it = item_of<kTree>(s.q_len, s.len, rt, p.tokens, p.a.window);
      ch = h;
      ++rt;
      const int size = it.tiles + kOver, o = off, o1 = (int)min((int64_t)size, o + (end - pos));
      last = pos - o + size - 1;
      pos += o1 - o;
      off = 0;
      a = max(0, o - kOver);
      b = o1 - kOver;
      if (b > a) return true;                              // (else the range ends before its first tile)
    }
    return false;
  }
};

// What the roles need of a segment: written by the scheduler warp, a ring of kSegs in shared memory.
struct Segment {
  int more;                  // 0: there is none, the CTA is done
  int tok0, cnt;             // its tokens, as rows of q and out
  int head0;                 // first query head
  int p_first, p_last;       // positions of the first and last token (of a tree: bounds, low_pos)
  int key0, key1;            // keys [key0, key1), whole tiles; those past the last position are masked
  int ch;                    // kv head
  int used;                  // pages of the sequence
  int whole, begins;         // the item's tiles are all here / its first one is
  const int32_t* table;      // the sequence's pages
};

template <int kCap, int kKind>
__global__ void __launch_bounds__(kKind == kNodesTurns ? kThreadsTurns : kThreadsP, 1)
    kda_attn_prefill_kernel(const __grid_constant__ PrefillParams p) {
  constexpr bool kTree = kKind != kCausal, kTurns = kKind == kNodesTurns;
  constexpr int kT = kTurns ? kThreadsTurns : kThreadsP;
  constexpr int kSoftRegs = kTurns ? kRegsSoftmaxTurns : kRegsSoftmax;
  constexpr int kOtherRegs = kTurns ? kRegsOtherTurns : kRegsOther;
  constexpr int kScales = kTurns ? 8 : 4;            // tiles whose scales are kept
  // (in turns there is one row tile's queries, and two V tiles in the place of the other's)
  constexpr int kVS = kTurns ? 4 : kVStages;
  auto v8_at = [](uint32_t stage) -> uint32_t {
    return kTurns && stage >= 2 ? kOffQ + 32768 + (stage - 2) * 16384 : kOffV8 + stage * 16384;
  };
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar_kf = sb + kOffBars, bar_ke = bar_kf + 8 * kKStages;
  const uint32_t bar_vf = bar_ke + 8 * kKStages, bar_ve = bar_vf + 8 * kVS;
  const uint32_t bar_be = bar_ve + 8 * kVS;                             // widened V read
  const uint32_t bar_q = bar_be + 16, bar_s = bar_q + 16, bar_p = bar_s + 16, bar_o = bar_p + 16;
  const uint32_t bar_of = bar_o + 16, bar_end = bar_of + 16, bar_sc = bar_end + 16;   // bar_sc: scales
  const uint32_t bar_gf = bar_sc + 64, bar_ge = bar_gf + 8 * kSegs;               // segment ring
  struct Misc {
    long long part[kThreadsTurns / 32];
    long long rest;          // first tile's place in its sequence
    int few[kThreadsTurns / 32];
    int start_n, poison[8];
    int start_h, start_rt, start_off;
    uint32_t tmem;
  };
  Misc* misc = reinterpret_cast<Misc*>(sm + kOffMiscP);
  static_assert(sizeof(Misc) <= 448, "misc");
  const int hk = p.a.c.kv_heads, N = p.a.num_seqs, P = p.a.c.page_size;
  const int G = p.group;
  const uint32_t gm = p.group_magic;

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(bar_kf + 8 * i, 1);
      mbar_init(bar_ke + 8 * i, 1);
    }
    for (int i = 0; i < kVS; ++i) {
      mbar_init(bar_vf + 8 * i, 1);
      mbar_init(bar_ve + 8 * i, 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_be + 8 * i, 1);
      mbar_init(bar_q + 8 * i, kSoftWarps / 2);
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, kSoftWarps / 2 + 4);   // and the four V warps
      mbar_init(bar_o + 8 * i, 1);
      mbar_init(bar_of + 8 * i, kSoftWarps / 2);
      mbar_init(bar_end + 8 * i, 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(bar_sc + 8 * i, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar_gf + 8 * i, 1);
      mbar_init(bar_ge + 8 * i, kSoftWarps + (kTurns ? 11 : 6));   // softmax, V, producer(s), MMA
    }
    mbar_fence_init();
    for (int i = 0; i < 8; ++i) misc->poison[i] = 0;
    tma_prefetch_desc(&p.maps.k);
    tma_prefetch_desc(&p.maps.v);
  }
  if (warp == kSoftWarps + 5) {
    tmem_alloc(smem_u32(&misc->tmem), 512);
    tmem_relinquish();
  }
  // (launched as a programmatic dependent of the work before this call)
  pdl_wait();
  if (p.gate && tid == 0 && blockIdx.x == 0) st_release_gpu(p.a.status + kGateWord, p.gate);
  pdl_launch_dependents();
  if (tid == 0 && blockIdx.x == 0 && p.a.cu_seqlens[0] != 0) record_error(p.a.status, KDA_ERR_BAD_CU_SEQLENS, 330);

  // ---- this CTA's range.  A thread reads its sequence's lengths; the warp adds up the row
  // tiles of each of its sequences together.
  auto cost = [&](int n, bool report, int& few) -> long long {   // units of sequence n (all heads)
    int q_len = 0, len = 0;
    few = 0;                 // ... of one that the decode kernel may take
    if (n < N) {
      int err;
      const SeqInfo s = seq_info<kTree>(p.a, n, 1, 0x7fffffff, &err);
      if (err != KDA_OK && report && blockIdx.x == 0) record_error(p.a.status, err, 331);
      if (s.tiles && (int64_t)s.q_len * G <= p.few) {
        few = (int)min((long long)(s.tiles + kOver) * hk, 1ll << 24);   // (as the decode kernel counts)
      } else if (s.tiles) {
        q_len = s.q_len;
        len = s.len;
      }
    }
    // a lane its own sequence when it has few row tiles, else the warp together
    long long mine = 0;
    const int rts = (q_len + p.tokens - 1) / p.tokens;
    if (rts <= 32)
      for (int rt = 0; rt < rts; ++rt) mine += item_of<kTree>(q_len, len, rt, p.tokens, p.a.window).tiles + kOver;
    uint32_t todo = __ballot_sync(0xffffffffu, rts > 32);
    while (todo) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const int ql = __shfl_sync(0xffffffffu, q_len, k), ln = __shfl_sync(0xffffffffu, len, k);
      int sum = 0;
      for (int rt = lane; rt * p.tokens < ql; rt += 32) sum += item_of<kTree>(ql, ln, rt, p.tokens, p.a.window).tiles + kOver;
      // (millions of new tokens over as many keys: the warp's sum passes 31 bits)
      const long long all = __reduce_add_sync(0xffffffffu, (unsigned)sum & 0xffffu) +
                            ((long long)__reduce_add_sync(0xffffffffu, (unsigned)sum >> 16) << 16);
      if (lane == k) mine = all;
    }
    mine *= hk;
    return mine;
  };
  long long mine = 0, first = 0;
  int few = 0, first_few = 0;
  for (int n0 = 0; n0 < N; n0 += kT) {
    int f;
    const long long w = cost(n0 + tid, true, f);
    if (n0 == 0) {
      first = w;
      first_few = f;
    }
    mine += w;
    few = min(few + f, 1 << 24);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  few = __reduce_add_sync(0xffffffffu, few);
  if (lane == 0) {
    misc->part[warp] = mine;
    misc->few[warp] = few;
  }
  __syncthreads();
  long long total = 0, total_few = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    total += misc->part[w];
    total_few += misc->few[w];
  }
  __syncthreads();
  const bool all = total_few < p.least;
  if (all) total += total_few;
  WalkP<kTree> walk;
  walk.min_rows = all ? 1 : p.few + 1;
  // (no more ranges than units: between two CTAs of an item there is none without a part)
  const int ranges = (int)min((long long)gridDim.x, total);
  walk.pos = walk.end = 0;
  if ((int)blockIdx.x < ranges) {
    walk.pos = (int64_t)blockIdx.x * total / ranges;
    walk.end = (int64_t)(blockIdx.x + 1) * total / ranges;
  }
  if (walk.pos < walk.end) {
    long long before = 0;
    for (int n0 = 0; n0 < N; n0 += kT) {
      int f = first_few;
      long long w = n0 == 0 ? first : cost(n0 + tid, false, f);
      if (all) w += f;
      long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 31) misc->part[warp] = inc;
      __syncthreads();
      // the warps' sums scanned by every warp, a lane each
      const long long mine_w = lane < kT / 32 ? misc->part[lane] : 0;
      long long scan = mine_w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += u;
      }
      const long long off = before + __shfl_sync(0xffffffffu, scan - mine_w, warp);
      if (w > 0 && walk.pos >= off + inc - w && walk.pos < off + inc) {
        const long long x = walk.pos - (off + inc - w);
        misc->start_n = n0 + tid;
        if (w >> 32 == 0) {            // (64-bit division takes hundreds of cycles)
          const uint32_t per_head = (uint32_t)w / (uint32_t)hk;
          misc->start_h = (int)((uint32_t)x / per_head);
          misc->rest = (uint32_t)x % per_head;
        } else {
          const long long per_head = w / hk;
          misc->start_h = (int)(x / per_head);
          misc->rest = x % per_head;
        }
      }
      before += __shfl_sync(0xffffffffu, scan, 31);
      __syncthreads();
      if (before > walk.pos) break;
    }
    walk.n = misc->start_n;
    walk.h = misc->start_h;
    int err;
    walk.s = seq_info<kTree>(p.a, walk.n, walk.min_rows, 0x7fffffff, &err);
    if (warp == 0) {     // the row tile: 32 at a time
      long long left = misc->rest;
      for (int r0 = 0;; r0 += 32) {
        const int rt = r0 + lane;
        const int c = rt * p.tokens < walk.s.q_len
                          ? item_of<kTree>(walk.s.q_len, walk.s.len, rt, p.tokens, p.a.window).tiles + kOver : 0;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, left < inc && left >= inc - c);
        if (here) {
          if (lane == __ffs(here) - 1) {
            misc->start_rt = rt;
            misc->start_off = (int)(left - (inc - c));
          }
          break;
        }
        if (r0 * p.tokens >= walk.s.q_len) break;   // (lengths that changed under the kernel)
        left -= __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  if (walk.pos < walk.end) {
    walk.rt = misc->start_rt;
    walk.off = misc->start_off;
  }

  const Segment* ring = reinterpret_cast<const Segment*>(sm + kOffSeg);
  static_assert(sizeof(Segment) <= 64 && kSegs <= 4, "segment ring");
  // The next segment (`ok`: none of the warp's waits gave up), and done with one.
  auto seg_wait = [&](uint32_t seg, bool& ok) -> const Segment* {
    ok = ok && mbar_wait_sleep(bar_gf + 8 * (seg % kSegs), (seg / kSegs) & 1);
    ok = __all_sync(0xffffffffu, ok);
    return ring + seg % kSegs;
  };
  auto seg_done = [&](uint32_t seg) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_ge + 8 * (seg % kSegs));
  };

  if (warp >= kSoftWarps + 4 && warp < kSoftWarps + 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftWarps + 4 || (kTurns && warp == kSoftWarps + 7)) {
      // ================= producer; a tile's pages and scales are looked up one tile ahead.  In turns the
      // values have a warp of their own: a tile is half as long there, and keys that waited for a place of
      // the values before them came late (tile 2350 -> 1400 cycles, with four places for values)
      const bool feeds_k = warp == kSoftWarps + 4, feeds_v = !kTurns || !feeds_k;
      uint32_t it = 0, seg = 0;
      bool ok = true;
      const int per = P / 16;                            // 16-key groups per page
      // lanes 0-7: the page that holds keys 16 lane .. of a tile (its first lane loads it); one wholly
      // before every window is not looked up: its entry may be stale
      auto page_of = [&](const Segment& g, int key) -> int {
        const int b = (key + 16 * lane) / P;
        if (lane >= 8 || key >= g.key1 || b >= g.used || (b + 1) * P <= first_seen(g.p_first, p.a.window))
          return -2;
        const int pg = g.table[b];
        if (pg < 0 || pg >= p.a.c.num_pages) {
          record_error(p.a.status, KDA_ERR_BAD_CACHE_INDEX, 332);
          return p.a.c.num_pages;                        // outside the map: the load gives zeros
        }
        return pg;
      };
      while (true) {
        const Segment g = *seg_wait(seg, ok);
        if (!ok || !g.more) break;
        seg_done(seg++);
        auto scale_of = [&](const float* sc, int pg) -> float {
          return pg >= 0 && pg < p.a.c.num_pages ? sc[(int64_t)pg * p.a.c.scale_stride + g.ch] : 1.0f;
        };
        int pg = page_of(g, g.key0);
        for (int key = g.key0; key < g.key1; key += kTile, ++it) {
          const uint32_t sk = it % kKStages, sv = it % kVS;
          const bool loads = pg != -2 && lane % per == 0;
          const int row = lane * 16;
          int pg_next = 0;
          if (feeds_k) {
            const float ks = scale_of(p.a.c.k_scale, pg), vs = scale_of(p.a.c.v_scale, pg);
            pg_next = page_of(g, key + kTile);
            if (it >= kKStages) ok = mbar_wait_sleep(bar_ke + 8 * sk, (it / kKStages - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // (slot it % 4 was last read for tile it - 4, whose P precedes the products of tile
            // it - 3 that the wait above saw done; in turns slot it % 8 for tile it - 8, whose P precedes that
            // of tile it - 6, which precedes those products)
            if (lane < 8)   // (a page without a scale is NaN to the rows that see it, and nothing to the others)
              reinterpret_cast<float4*>(sm + kOffSc)[(it % kScales) * 8 + lane] =
                  make_float4(ks, vs > 0.0f ? lg2(vs) : NAN, vs > 0.0f ? __fdividef(1.0f, vs) : 0.0f, 0.0f);
          }
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, loads)) * P * kHeadDim;
          __syncwarp();
          if (feeds_k) {
            if (lane == 0) {
              mbar_arrive(bar_sc + 8 * (it % kScales));
              mbar_expect_tx(bar_kf + 8 * sk, bytes);
            }
            __syncwarp();
            if (loads) tma_load_4d(sb + kOffK + sk * 16384 + row * 128, &p.maps.k, 0, 0, g.ch, pg, bar_kf + 8 * sk);
          } else {
            pg_next = page_of(g, key + kTile);
          }
          if (feeds_v) {
            if (it >= kVS) ok = mbar_wait_sleep(bar_ve + 8 * sv, (it / kVS - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(bar_vf + 8 * sv, bytes);
            __syncwarp();
            if (loads) tma_load_4d(sb + v8_at(sv) + row * 128, &p.maps.v, 0, 0, g.ch, pg, bar_vf + 8 * sv);
          }
          pg = pg_next;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 333);
      // the copies in flight end before the CTA does (a failed wait left at most one K behind)
      if (feeds_k)
        for (uint32_t i = it > kKStages ? it - kKStages : 0; i < it + (ok ? 0 : 1); ++i)
          mbar_wait_sleep(bar_kf + 8 * (i % kKStages), (i / kKStages) & 1);
      if (feeds_v)
        for (uint32_t i = it > kVS ? it - kVS : 0; i < it; ++i)
          mbar_wait_sleep(bar_vf + 8 * (i % kVS), (i / kVS) & 1);
    } else if (warp == kSoftWarps + 5) {
      // ================= MMA issuer (the warp stays together; one lane issues)
      constexpr uint32_t id_s = idesc_e4m3(128, 128, 0, 0), id_o = idesc_f16(128, 128, 0, 1);
      const uint32_t lead = elect_one() ? 1u : 0u;
      const uint64_t dq = kmajor8(sb + kOffQ, 0), dk0 = kmajor8(sb + kOffK, 0);
      const uint64_t dv0 = sdesc_sw128(sb + kOffVB, 16384, 1024);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      uint32_t sk = 0;                                   // stage of the next keys
      auto qk = [&](int h) {                             // S of half h from the keys of stage sk
        const uint64_t dk = dk0 + sk * (16384 >> 4), q = dq + (kTurns ? 0 : h * (32768 >> 4));
#pragma unroll
        for (int x = 0; x < 8; ++x)
          mma_e4m3_on(lead, tmem + kTS + 128 * h, q + ((x >> 2) * 16384 + (x & 3) * 32) / 16,
                      dk + (x & 3) * 32 / 16, id_s, x > 0);
        mma_commit_on(lead, bar_s + 8 * h);
      };
      auto pv = [&](uint32_t i, int h, bool first_tile, bool last_tile) {   // O of half h += P(i) V(i)
        // (the segment before has read its O)
        if (first_tile && seg > 0) ok = ok && mbar_wait_sleep(bar_of + 8 * h, (seg - 1) & 1);
        // P(i), V(i) and the keys of the half's next tile
        ok = ok && mbar_wait_sleep(bar_p + 8 * h, (kTurns ? i >> 1 : i) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dv = dv0 + (i & 1) * (32768 >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ts_on(lead, tmem + kTOP + 128 * h, tmem + kTS + 128 * h + 8 * ks, dv + 2048 * ks / 16,
                        id_o, !(first_tile && ks == 0));
        if (last_tile) mma_commit_on(lead, bar_o + 8 * h);
      };
      while (true) {
        const Segment* sg = seg_wait(seg, ok);
        if (!ok || !sg->more) break;
        const int tiles = (sg->key1 - sg->key0) / kTile;
        seg_done(seg);
        if (kTurns) {
          // tile i is half i & 1's: S of the first two, then O of a tile and S of the half's next
          ok = mbar_wait_sleep(bar_q, seg & 1);
          const uint32_t end = it + tiles;
          for (uint32_t i = it; ok && i < end && i < it + 2; ++i) {
            sk = i % kKStages;
            ok = mbar_wait_sleep(bar_kf + 8 * sk, (i / kKStages) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            qk(i & 1);
            mma_commit_on(lead, bar_ke + 8 * sk);
          }
          ok = __all_sync(0xffffffffu, ok);
          const uint32_t start = it;
          for (; ok && it < end; ++it) {
            if (it + 2 < end)
              ok = mbar_wait_sleep(bar_kf + 8 * ((it + 2) % kKStages), ((it + 2) / kKStages) & 1);
            ok = __all_sync(0xffffffffu, ok);
            pv(it, it & 1, it < start + 2, it + 2 >= end);
            if (!ok) break;
            mma_commit_on(lead, bar_be + 8 * (it & 1));
            if (it + 2 < end) {
              sk = (it + 2) % kKStages;
              qk(it & 1);
              mma_commit_on(lead, bar_ke + 8 * sk);
            }
          }
          if (ok && tiles == 1) {      // the other half's O of nothing
            const int h = it & 1;
            if (seg > 0) ok = mbar_wait_sleep(bar_of + 8 * h, (seg - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            mma_commit_on(lead, bar_o + 8 * h);
          }
          ++seg;
          if (!ok) break;
          continue;
        }
        ok = mbar_wait_sleep(bar_kf + 8 * sk, (it / kKStages) & 1);
        for (int h = 0; h < 2; ++h) {
          ok = ok && mbar_wait_sleep(bar_q + 8 * h, seg & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          qk(h);
        }
        for (int t = 1; ok; ++t) {
          // O of the tile before, S of this one, half by half
          mma_commit_on(lead, bar_ke + 8 * sk);
          if (++sk == kKStages) sk = 0;
          ++it;
          const bool more = t < tiles;
          pv(it - 1, 0, t == 1, !more);
          if (!ok) break;
          if (more) qk(0);
          pv(it - 1, 1, t == 1, !more);
          if (!ok) break;
          mma_commit_on(lead, bar_be + 8 * ((it - 1) & 1));
          if (!more) break;
          qk(1);
        }
        ++seg;
        if (!ok) break;
      }
      if (!ok && lead) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 334);
      // what was issued ends, its arrivals included, before shared and tensor memory go
      mma_commit_on(lead, bar_end);
      mbar_wait_sleep(bar_end, 0);
      for (uint32_t i = it > kKStages ? it - kKStages : 0; ok && i < it; ++i)
        mbar_wait_sleep(bar_ke + 8 * (i % kKStages), (i / kKStages) & 1);
      for (uint32_t i = it > 2 ? it - 2 : 0; ok && i < it; ++i)
        mbar_wait_sleep(bar_be + 8 * (i & 1), (i >> 1) & 1);
      __syncwarp();
    } else if (warp == kSoftWarps + 6) {
      // ================= scheduler: this CTA's segments, one after the other
      PartDescP part = {0, 0, 0, 0};
      bool ok = true;
      for (uint32_t seg = 0;; ++seg) {
        const bool more = walk.next(p);
        const int tok0 = walk.s.tok0 + walk.it.tok;
        if (seg >= kSegs) ok = mbar_wait_sleep(bar_ge + 8 * (seg % kSegs), (seg / kSegs - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          Segment* g = reinterpret_cast<Segment*>(sm + kOffSeg) + seg % kSegs;
          g->more = more;
          if (more) {
            g->tok0 = tok0;
            g->cnt = walk.it.cnt;
            g->head0 = walk.ch * G;
            g->p_first = kTree ? low_pos<true>(walk.s.len - walk.s.q_len)
                               : walk.s.len - walk.s.q_len + walk.it.tok;
            g->p_last = kTree ? walk.s.len - 1 : g->p_first + walk.it.cnt - 1;
            g->key0 = (walk.it.tile0 + walk.a) * kTile;
            g->key1 = (walk.it.tile0 + walk.b) * kTile;
            g->ch = walk.ch;
            g->used = (walk.s.len + P - 1) / P;
            g->whole = walk.a == 0 && walk.b == walk.it.tiles;
            g->begins = walk.a == 0;
            g->table = p.a.c.block_table + walk.n * p.a.c.table_stride;
          }
          mbar_arrive(bar_gf + 8 * (seg % kSegs));
        }
        if (!more) break;
        if (seg > 0)    // its queries towards L2 (the first's are wanted at once)
          for (int i = lane; i < walk.it.cnt * ((G + 15) / 16); i += 32) {
            const int t = i / ((G + 15) / 16), h = (i % ((G + 15) / 16)) * 16;
            l2_prefetch(p.a.q + (int64_t)(tok0 + t) * p.a.q_stride + (walk.ch * G + h) * kHeadDim,
                        min(16, G - h) * kHeadDim * 2);
          }
        if (walk.a == 0 && walk.b < walk.it.tiles) {   // the CTA that the item's last tile lies in
          part.tok0 = tok0;
          part.rows = walk.it.cnt * G;
          part.head0 = walk.ch * G;
          part.parts = (int)(((walk.last + 1) * ranges - 1) / total - blockIdx.x) + 1;
        }
      }
      if (lane == 0) {
        if (!ok) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 337);
        p.desc[blockIdx.x] = part;
      }
      __syncwarp();
    }
  } else if (warp >= kSoftWarps) {
    // ================= V to f16, MN-major, 64-channel blocks 16 KB apart.  In turns four warps a half: a tile takes
    // them longer than the tensor cores
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int vt = (tid - 32 * kSoftWarps) & 127, c = vt & 7;        // 16-channel chunk of this thread
    const uint32_t vh = warp >= kSoftWarps + 8 ? 1 : 0;
    uint32_t it = 0, seg = 0;
    bool ok = true;
    while (true) {
      const Segment* sg = seg_wait(seg, ok);
      if (!ok || !sg->more) break;
      const int p_first = sg->p_first, p_last = sg->p_last, key1 = sg->key1;
      int key0 = sg->key0;
      // (last read four segments ago; before this segment's place is given back, or the other four warps
      // might be there already)
      if (vt == 0 && vh == 0) misc->poison[(seg + 4) & 7] = 0;
      seg_done(seg);
      for (; key0 < key1; key0 += kTile, ++it) {
        if (kTurns && (it & 1) != vh) continue;
        const uint32_t sv = it % kVS, vb = it & 1;
        ok = mbar_wait_sleep(bar_vf + 8 * sv, (it / kVS) & 1);
        if (it >= 2) ok = ok && mbar_wait_sleep(bar_be + 8 * vb, ((it >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned char* src = sm + v8_at(sv);
        unsigned char* dst = sm + kOffVB + vb * 32768 + (c >> 2) * 16384;
        const int seen0 = first_seen(p_first, p.a.window);   // no row of the tile sees an earlier key
        const bool masked = key0 + kTile - 1 > p_first || key0 < first_seen(p_last, p.a.window);
#pragma unroll 2
        for (int j = 0; j < 8; ++j) {
          const int row = (vt >> 3) + 16 * j, key = key0 + row;
          uint4 u = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
          // seen by no row of the tile: whatever is there reads as zero
          if (masked && (key > p_last || key < seen0))
            u = make_uint4(0, 0, 0, 0);
          uint32_t w[4] = {u.x, u.y, u.z, u.w}, o[8];
          if (masked) {     // NaN entries (rare) of a row that only some may see: noted, read as zero
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t m = __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              if (m) misc->poison[seg & 7] = 1;
              w[e] &= ~m;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = f16x2_of_e4m3x2(w[e] & 0xffff);
            o[2 * e + 1] = f16x2_of_e4m3x2(w[e] >> 16);
          }
          unsigned char* d = dst + (row >> 3) * 1024 + (row & 7) * 128;
          // the eight lanes of a row write even chunks of one block and odd ones of the other at a
          // time, which is every bank once
          const int k0 = (2 * c) & 7, odd = c >> 2;
          *reinterpret_cast<uint4*>(d + (((k0 + odd) ^ (row & 7)) << 4)) =
              odd ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d + (((k0 + 1 - odd) ^ (row & 7)) << 4)) =
              odd ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async();
        mbar_arrive(bar_ve + 8 * sv);
        // This warp's arrival on the barriers of P(it) tells the MMA issuer that V(it) is there, and
        // the next keys: it then has one thing to wait for (a wait behind matrix instructions takes
        // until they have left its queue).  Not before P(it - 1), whose phase it would count in.
        if (kTurns) {
          // (P(it - 2) is done: its products are, which the wait above saw.  The issuer waits for keys itself:
          // of three stages those of neighbouring tiles share one, and a half's warps see every second)
          if (lane == 0) mbar_arrive(bar_p + 8 * vh);
          continue;
        }
        if (it > 0) ok = mbar_wait_sleep(bar_p, (it - 1) & 1) && mbar_wait_sleep(bar_p + 8, (it - 1) & 1);
        if (key0 + kTile < key1) ok = ok && mbar_wait_sleep(bar_kf + 8 * ((it + 1) % kKStages), ((it + 1) / kKStages) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive(bar_p);
          mbar_arrive(bar_p + 8);
        }
      }
      ++seg;
      if (!ok) break;
    }
    if (!ok && vt == 0) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 335);
  } else {
    // ================= softmax: two threads a row, 64 keys (64 channels of O) each.  A wait that
    // gives up clears `ok`, after which nothing is waited for any more but every barrier is met.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int half = warp >> 3, cg = (warp >> 2) & 1, place = 128 * half + 32 * (warp & 3) + lane;
    const int row = kTurns ? place & 127 : place;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + kTS + 128 * half + lanes;
    const uint32_t to = tmem + kTOP + 128 * half + 64 * cg + lanes;
    const uint32_t id_pair = 1 + 4 * half + (warp & 3), id_half = 9 + half;
    const Cap cap = kCap ? cap_of(p.a.softcap) : Cap{0.0f, 0.0f};
    const float sign = p.a.scale < 0.0f ? -1.0f : 1.0f;  // (the row maximum is taken before the scale)
    float* qmul_s = reinterpret_cast<float*>(sm + kOffQmul);
    float* mx_s = reinterpret_cast<float*>(sm + kOffMx) + place;
    float* l_s = reinterpret_cast<float*>(sm + kOffL) + 2 * place;
    uint32_t it = 0, seg = 0;
    bool ok = true;
    while (true) {
      const Segment* sg = seg_wait(seg, ok);
      // (the half's threads go on or leave together; its staging of the segment before is over)
      // (in turns: both halves', whose merge is a barrier)
      if (bar_any(kTurns ? kIdBoth : id_half, kTurns ? 512 : 256, !ok)) {
        ok = false;
        break;
      }
      if (!sg->more) break;
      const int rows = sg->cnt * G;
      if (kTurns && half == 1) {      // (the other half's, for both)
        ok = ok && mbar_wait_sleep(bar_q, seg & 1);
        __syncwarp();
      } else {   // ---- queries as two e4m3 terms: 16 lanes a row, 16 rows a warp
        const int c = lane & 15, r0 = 128 * half + 16 * (warp & 7) + (lane >> 4);
        const __nv_bfloat16* src = p.a.q + (int64_t)sg->tok0 * p.a.q_stride + sg->head0 * kHeadDim + 8 * c;
        uint4 u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + 2 * j;
          u[j] = make_uint4(0, 0, 0, 0);
          const int i = div_small(r, gm);
          if (r < rows)
            u[j] = *reinterpret_cast<const uint4*>(src + (int64_t)i * p.a.q_stride + (r - i * G) * kHeadDim);
        }
        unsigned char* q1 = sm + kOffQ + half * 32768;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + 2 * j;
          float x[8], top = 0.0f;
          unpack8(u[j], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
          // a power of two that brings the row's largest entry into (224, 448]
          const int e2 = (int)((__float_as_uint(top) >> 23) & 255) - 127 - 8 +
                         ((__float_as_uint(top) & 0x7fffffu) > 0x600000u ? 1 : 0);
          const int e2c = max(e2, -100);
          const float inv = sign * __uint_as_float((uint32_t)(127 - e2c) << 23);
          uint32_t t1[4], t2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_e4m3x2(x[2 * e] * inv, x[2 * e + 1] * inv, t1[e], t2[e]);
          const uint32_t w1[2] = {t1[0] | (t1[1] << 16), t1[2] | (t1[3] << 16)};
          const uint32_t w2[2] = {t2[0] | (t2[1] << 16), t2[2] | (t2[3] << 16)};
          *reinterpret_cast<uint2*>(q1 + tile_off(r & 127, 8 * c)) = make_uint2(w1[0], w1[1]);
          *reinterpret_cast<uint2*>(q1 + 16384 + tile_off(r & 127, 8 * c)) = make_uint2(w2[0], w2[1]);
          if (c == 0) {   // a non-finite query makes its row NaN
            const float sq = top <= 3.402823466e38f ? __uint_as_float((uint32_t)(127 + e2c) << 23) : NAN;
            qmul_s[r] = sq * fabsf(p.a.scale) * kLog2e;
          }
        }
        fence_proxy_async();
        group_sync(id_half, 256);
        if (lane == 0) mbar_arrive(bar_q + 8 * half);
      }
      const float qmul = qmul_s[row];
      // relative to the tile's first key: this row's position, and those of the half's first and last
      const int last = sg->cnt - 1, rel = sg->p_first - sg->key0;
      int hi = rel + (row < rows ? div_small(row, gm) : last) - 64 * cg;
      int p_lo = rel + min(div_small(128 * half, gm), last);
      int p_hi = rel + div_small(max(min(rows, 128 * half + 128) - 1, 0), gm);
      // of a tree: this row's mask, and the cached tokens before the new ones from its first key on
      uint64_t node = 0;
      if (kTree) {
        node = p.a.tree[sg->tok0 + (row < rows ? div_small(row, gm) : last)] &
               node_bits(sg->p_last - sg->p_first);
        hi = rel + 1 - 64 * cg;
        p_lo = rel;
        p_hi = sg->p_last - sg->key0;
      }
      const int tiles = (sg->key1 - sg->key0) / kTile;
      float m = -INFINITY, l = 0.0f;
      // in turns every second tile, from the segment's first or second on
      constexpr int kStep = kTurns ? 2 : 1;
      const uint32_t after = it + tiles;
      const int skip = kTurns ? (int)((it ^ half) & 1) : 0;
      it += skip;
      hi -= skip * kTile;
      p_lo -= skip * kTile;
      p_hi -= skip * kTile;
      for (int t = 0; it < after; ++t, it += kStep, hi -= kStep * kTile, p_lo -= kStep * kTile, p_hi -= kStep * kTile) {
        const uint32_t turn = kTurns ? it >> 1 : it;      // the half's tiles before
        // (a wait costs over 100 cycles even when it need not wait: S, the last to come, last)
        ok = ok && mbar_wait_sleep(bar_sc + 8 * (it % kScales), (it / kScales) & 1);
        // (S was issued behind the O of the tile before, so that is there as well)
        ok = ok && mbar_wait_sleep(bar_s + 8 * half, turn & 1);
        __syncwarp();
        tc_fence_after();
        if (kTurns && row - lane >= rows) {      // none of the warp's rows: whatever lies there is its P
          tc_fence_before();
          if (lane == 0) mbar_arrive(bar_p + 8 * half);
          continue;
        }
        uint32_t s[64];
        uint32_t (&s_hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(s + 32);
        tmem_ld32(ts + 64 * cg, *reinterpret_cast<uint32_t(*)[32]>(s));
        tmem_wait_ld_of(*reinterpret_cast<uint32_t(*)[32]>(s));
        tmem_ld32(ts + 64 * cg + 32, s_hi);    // on its way while the first keys are worked on
        const float4* sc = reinterpret_cast<const float4*>(sm + kOffSc) + (it % kScales) * 8 + 4 * cg;
        const bool masked = kTile - 1 > p_lo || (p.a.window > 0 && p.a.window <= p_hi);
        const bool scaled = kCap || masked;    // s holds the finished exponents (else raw products)
        float mt = -INFINITY;
        // P of the group's 16 keys, and their part of the denominator
        auto p_of = [&](int g, float mul, float add, uint32_t (&pk)[32]) -> float {
          const float2 mul2 = make_float2(mul, mul), add_2 = make_float2(add, add);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int e = 16 * g; e < 16 * g + 16; e += 2) {
            float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), mul2, add_2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum = add2(sum, x);
            pk[e >> 1] = f16x2_of(x.x, x.y);
          }
          return sum.x + sum.y;
        };
        auto max_of = [&](int g) -> float {    // of the group's raw products
          float a = __uint_as_float(s[16 * g]), b = __uint_as_float(s[16 * g + 1]);
#pragma unroll
          for (int e = 16 * g + 2; e < 16 * g + 14; e += 4) {
            a = max3(a, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            b = max3(b, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          }
          a = max3(a, __uint_as_float(s[16 * g + 14]), __uint_as_float(s[16 * g + 15]));
          return fmaxf(a, b);
        };
        auto with_pair = [&] {        // the row's other 64 keys
          mx_s[((turn & 1) * 2 + cg) * kRowsP] = mt;
          group_sync(id_pair, 64);    // (also: both have S in registers, P may go over it)
          mt = fmaxf(mt, mx_s[((turn & 1) * 2 + (cg ^ 1)) * kRowsP]);
        };
        uint32_t pk[32];
        bool keep = false;
        const bool ahead = !scaled && t > 0;
        if (ahead) {
          // most tiles leave the reference where it is: P by it, the maximum beside that
          const float ref = (m == -INFINITY ? 0.0f : m) - kPShift;
          float sum = l;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 f = sc[g];
            const float mul = qmul * f.x;
            if (g == 2) tmem_wait_ld_of(s_hi);
            mt = fmaxf(mt, fmaf(max_of(g), mul, f.y));
            sum = fmaf(p_of(g, mul, f.y - ref, pk), f.z, sum);
          }
          with_pair();
          keep = !__any_sync(0xffffffffu, mt > m + kSlack);
          if (keep) l = sum;
        } else {
          tmem_wait_ld_of(s_hi);
        }
        if (!keep) {
          if (ahead) {
            tmem_ld32(ts + 64 * cg, *reinterpret_cast<uint32_t(*)[32]>(s));
            tmem_ld32(ts + 64 * cg + 32, s_hi);
            tmem_wait_ld();
            group_sync(id_pair, 64);
          } else if (scaled) {
            // bits of the 64 keys that this row sees: lo <= e <= hi
            // (below hi < 0 the difference may wrap: nothing is seen then)
            int lo = p.a.window > 0 ? (int)((uint32_t)hi - (uint32_t)p.a.window + 1u) : 0;
            uint64_t upto = hi < 0 ? 0 : (hi >= 63 ? ~0ull : (2ull << hi) - 1);
            if (kTree) {     // hi cached keys, then the new ones (the window has room for those seen)
              lo = p.a.window > 0 && hi > 0 ? hi + __popcll(node) - p.a.window : 0;
              upto = hi >= 64 ? ~0ull
                     : hi >= 0 ? ((1ull << hi) - 1) | (node << hi)
                               : (hi > -64 ? node >> -hi : 0);
            }
            const uint64_t see = lo <= 0 ? upto : (lo >= 64 ? 0 : upto & (~0ull << lo));
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float4 f = sc[g];
              const float mul = qmul * f.x, add = f.y;
              const uint32_t bits = (uint32_t)(see >> (32 * (g >> 1))) >> (16 * (g & 1));
              if (kCap == kCapExact) {
                float top = 0.0f;
#pragma unroll
                for (int e = 16 * g; e < 16 * g + 16; e += 2)
                  top = max3_abs(top, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                const float2 mul_2 = make_float2(mul, mul), add_2 = make_float2(add, add);
                if (__any_sync(0xffffffffu, top * mul * cap.inv >= kCapSmall)) {
#pragma unroll
                  for (int e = 16 * g; e < 16 * g + 16; e += 2) {
                    const float2 t = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), mul_2);
                    const float2 y = cap_any(t, cap, add_2);
                    s[e] = __float_as_uint(y.x);
                    s[e + 1] = __float_as_uint(y.y);
                  }
                } else {
#pragma unroll
                  for (int e = 16 * g; e < 16 * g + 16; e += 2) {
                    const float2 t = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), mul_2);
                    const float2 y = cap_small(t, cap, add_2);
                    s[e] = __float_as_uint(y.x);
                    s[e + 1] = __float_as_uint(y.y);
                  }
                }
              }
              if (kCap == kCapExact && !masked) {
                mt = fmaxf(mt, max_of(g));
                continue;
              }
              const float mul_e = mul * (2.0f * kLog2e * cap.inv);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x = __uint_as_float(s[16 * g + e]);
                if (kCap != kCapExact) x = kCap ? cap_plain(x, mul_e, cap, add) : fmaf(x, mul, add);
                if (!((bits >> e) & 1)) x = -INFINITY;
                mt = fmaxf(mt, x);
                s[16 * g + e] = __float_as_uint(x);
              }
            }
            with_pair();
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) mt = fmaxf(mt, fmaf(max_of(g), qmul * sc[g].x, sc[g].y));
            with_pair();
          }
          if (__any_sync(0xffffffffu, mt > m + kSlack)) {
            const float next = fmaxf(m, mt), f = ex2(m - (next == -INFINITY ? 0.0f : next));
            if (t > 0) {       // O, the tile before included, by the factor
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t o[16];
                tmem_ld16(to + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(to + 16 * c, o);
              }
            }
            l *= f;
            m = next;
          }
          const float ref = (m == -INFINITY ? 0.0f : m) - kPShift;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 f = sc[g];
            l = fmaf(p_of(g, scaled ? 1.0f : qmul * f.x, scaled ? -ref : f.y - ref, pk), f.z, l);
          }
        }
        // P over the columns of S
        tmem_st32(ts + 32 * cg, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 8 * half);
      }
      it = after;
      ok = ok && mbar_wait_sleep(bar_o + 8 * half, seg & 1);
      m -= kPShift;       // (the numerators' reference)
      l_s[cg] = l;
      group_sync(id_pair, 64);
      l = l_s[0] + l_s[1];
      tc_fence_after();
      // ---- in turns: half A takes half B's maxima and denominators, and its sums from tensor memory (the rows of
      // a warp are the same lanes there)
      float mine = 1.0f, other = 0.0f;
      if (kTurns) {
        if (half == 1) {
          if (cg == 0) {
            mx_s[0] = m;
            l_s[0] = l;
          }
          group_sync(kIdMerge, 512);
          seg_done(seg);
          ++seg;
          continue;
        }
        ok = ok && mbar_wait_sleep(bar_o + 8, seg & 1);
        group_sync(kIdMerge, 512);
        tc_fence_after();
        const float m1 = mx_s[128], l1 = l_s[256], top = fmaxf(m, m1), ref = top == -INFINITY ? 0.0f : top;
        mine = ex2(m - ref);
        other = ex2(m1 - ref);
        m = top;
        l = l * mine + l1 * other;
      }
      // ---- the segment's rows out: 128 bytes of a row at a time through this warp's 4 KB of the
      // query area (all products of the half are done), so that the stores are whole lines
      const bool poisoned = *reinterpret_cast<volatile int*>(&misc->poison[seg & 7]) != 0;
      const bool live = row < rows, whole = sg->whole;
      const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
      const int i_tok = live ? div_small(row, gm) : last, head = sg->head0 + (live ? row - i_tok * G : 0);
      const int64_t tok = sg->tok0 + i_tok;
      float* slot = p.slots + ((int64_t)2 * blockIdx.x + (sg->begins ? 1 : 0)) * kSlotFloatsP;
      unsigned char* stage = sm + kOffQ + half * 32768 + (warp & 7) * 4096;
      uint64_t dst = whole ? reinterpret_cast<uint64_t>(p.a.out + tok * p.a.out_stride + head * kHeadDim + 64 * cg)
                           : reinterpret_cast<uint64_t>(slot + row * 128 + 64 * cg);
      if (!live) dst = 0;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {     // 32 channels
        uint32_t o[32];
        tmem_ld32(to + 32 * c, o);
        tmem_wait_ld();
        if (kTurns) {
          // (a half without a tile, or without a key that the row sees, has nothing to add, whatever lies there)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t x[16];
            tmem_ld16(to + 128 + 32 * c + 16 * g, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a = mine > 0.0f ? __uint_as_float(o[16 * g + e]) * mine : 0.0f;
              o[16 * g + e] = __float_as_uint(other > 0.0f ? fmaf(__uint_as_float(x[e]), other, a) : a);
            }
          }
        }
        if (poisoned && live) {    // NaN entries that this row sees, in tiles that some rows do not
          const int p0 = sg->p_first, p1 = sg->p_last, pos = kTree ? p1 : p0 + i_tok;
          const int cnt = __popcll(node);
          for (int key0 = sg->key0; key0 < sg->key1; key0 += kTile) {
            if (!(key0 + kTile - 1 > p0 || key0 < first_seen(p1, p.a.window))) continue;
            for (int key = kTree ? key0 : max(key0, first_seen(pos, p.a.window));
                 key <= min(key0 + kTile - 1, pos); ++key) {
              if (kTree && !tree_sees(node, cnt, key, p0 + 1, p1 + 1, p.a.window)) continue;
              const int pg = sg->table[key / P];
              if (pg < 0 || pg >= p.a.c.num_pages) continue;
              const uint8_t* v = p.a.c.v + pg * p.a.c.page_stride + sg->ch * p.a.c.head_stride +
                                 (key % P) * p.a.c.token_stride + 64 * cg + 32 * c;
#pragma unroll 1
              for (int e = 0; e < 32; ++e)
                if ((v[e] & 0x7f) == 0x7f) {
#pragma unroll
                  for (int f = 0; f < 32; ++f)
                    if (f == e) o[f] = 0x7fffffffu;
                }
            }
          }
        }
        const int sw = lane & 7;
        if (whole) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * g + e]) * inv_l;
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + g) ^ sw) << 4)) = pack8(x);
          }
          if (c == 0) continue;    // a row's 64 channels are 128 bytes of bf16
        } else {
#pragma unroll
          for (int g = 0; g < 8; ++g)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((g ^ sw) << 4)) =
                make_uint4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 4 * j + (lane >> 3), g = lane & 7;
          const uint64_t d = __shfl_sync(0xffffffffu, dst, r);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((g ^ (r & 7)) << 4));
          if (d) *reinterpret_cast<uint4*>(d + (whole ? 0 : 128 * c) + 16 * g) = v;
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_of + 8 * half);
        if (kTurns) mbar_arrive(bar_of + 8);
      }
      if (live && cg == 0) {
        if (!whole) {
          slot[kRowsP * 128 + row] = m;
          slot[kRowsP * 129 + row] = l;
        } else if (p.a.lse) {
          p.a.lse[tok * p.a.heads + head] = l == 0.0f ? -INFINITY : (m + lg2(l)) * kLn2;
        }
      }
      seg_done(seg);
      ++seg;
    }
    if (!ok && lane == 0) record_error(p.a.status, KDA_ERR_DEVICE_TIMEOUT, 336);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merges the parts of the item that CTA blockIdx.x began and did not finish, in CTA order: a warp
// a row, a lane 4 channels.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows)
    kda_attn_prefill_merge_kernel(const __grid_constant__ PrefillParams p) {
  pdl_wait();
  pdl_launch_dependents();
  if (p.gate && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) p.a.status[kGateWord] = 0;
  const int4 d4 = *reinterpret_cast<const int4*>(p.desc + blockIdx.x);
  const PartDescP d = {d4.x, d4.y, d4.z, d4.w};
  const int lane = threadIdx.x & 31, r = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
  if (d.parts == 0 || r >= d.rows) return;
  // four parts in flight, merged into the running maximum, sum and denominator
  constexpr int kInFlight = 4;
  float m = -INFINITY, den = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < d.parts; i0 += kInFlight) {
    float mi[kInFlight], di[kInFlight], top = m;
    float4 ai[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int i = i0 + u;
      const float* s = p.slots + ((int64_t)2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kSlotFloatsP;
      mi[u] = -INFINITY;
      di[u] = 0.0f;
      ai[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < d.parts) {
        mi[u] = s[kRowsP * 128 + r];
        di[u] = s[kRowsP * 129 + r];
        ai[u] = *reinterpret_cast<const float4*>(s + r * 128 + 4 * lane);
      }
    }
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
  }
  const float il = den == 0.0f ? 0.0f : 1.0f / den;
  const int i_tok = div_small(r, p.group_magic);
  const int64_t tok = d.tok0 + i_tok;
  const int head = d.head0 + r - i_tok * p.group;
  const uint2 o2 = make_uint2(pack_bf16x2(acc.x * il, acc.y * il), pack_bf16x2(acc.z * il, acc.w * il));
  *reinterpret_cast<uint2*>(p.a.out + tok * p.a.out_stride + head * kHeadDim + 4 * lane) = o2;
  if (p.a.lse && lane == 0)
    p.a.lse[tok * p.a.heads + head] = den == 0.0f ? -INFINITY : (m + lg2(den)) * kLn2;
}

template <int kCap, int kKind>
cudaError_t launch_kernel(const PrefillParams& d, int sms, cudaStream_t stream) {
  constexpr int threads = kKind == kNodesTurns ? kThreadsTurns : kThreadsP;
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&]() -> cudaError_t {
    cudaFuncAttributes at;
    cudaError_t x = cudaFuncGetAttributes(&at, kda_attn_prefill_kernel<kCap, kKind>);
    if (x != cudaSuccess) return x;
    // the warpgroups' register shares must fit what the block is launched with
    if ((at.numRegs + 7) / 8 * 8 * threads < (kKind == kNodesTurns ? kRegsNeededTurns : kRegsNeeded))
      return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kda_attn_prefill_kernel<kCap, kKind>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemP);
  });
  if (e != cudaSuccess) return e;
  return launch(kda_attn_prefill_kernel<kCap, kKind>, dim3((unsigned)sms), dim3(threads), kSmemP, true,
                stream, d);
}
// Trees whose rows fill no more than half of a tile of 256, on average over the batch (the lengths are on the
// device), take the halves in turns.  32 heads over 8, 16 sequences of up to 16384 keys, in turns against side by
// side: 16 nodes (64 rows) 83 : 104 us, 40 nodes 146 : 108, 64 nodes 154 : 112; 64 sequences of 1 to 31
// nodes, 16 heads over 2, a window of 2048 and capped scores 47 : 55.
bool in_turns(const AttnParams& a) {
  const int group = a.heads / a.c.kv_heads;
  return a.tree && group <= kRowsP / 2 && (int64_t)a.max_q_len * group <= kRowsP &&
         a.total_tokens * group <= (int64_t)a.num_seqs * (kRowsP / 2);
}
template <int kCap>
cudaError_t launch_cap(const PrefillParams& d, int sms, cudaStream_t stream) {
  if (!d.a.tree) return launch_kernel<kCap, kCausal>(d, sms, stream);
  return in_turns(d.a) ? launch_kernel<kCap, kNodesTurns>(d, sms, stream)
                       : launch_kernel<kCap, kNodesWide>(d, sms, stream);
}

}  // namespace

size_t prefill_workspace_bytes(int sms) {
  return (size_t)sms * sizeof(PartDescP) + (size_t)sms * 2 * kSlotFloatsP * sizeof(float);
}

namespace {
void make_params(const AttnParams& a, int few, int64_t least, int gate, void* work, int sms, PrefillParams* d) {
  d->a = a;
  d->gate = gate;
  d->few = few;
  d->least = least;
  d->group = a.heads / a.c.kv_heads;
  d->group_magic = 65535u / (uint32_t)d->group + 1;
  d->tokens = (in_turns(a) ? kRowsP / 2 : kRowsP) / d->group;
  d->desc = static_cast<PartDescP*>(work);
  d->slots = reinterpret_cast<float*>(d->desc + sms);
}
}  // namespace

cudaError_t launch_attn_prefill(const AttnParams& a, const CacheMaps& maps, int few, int64_t least,
                                int gate, void* work, int sms, cudaStream_t stream) {
  PrefillParams d;
  make_params(a, few, least, gate, work, sms, &d);
  d.maps = maps;
  switch (cap_kind(a.softcap)) {
    case kNoCap: return launch_cap<kNoCap>(d, sms, stream);
    case kCapPlain: return launch_cap<kCapPlain>(d, sms, stream);
    default: return launch_cap<kCapExact>(d, sms, stream);
  }
}

cudaError_t launch_attn_prefill_merge(const AttnParams& a, int gate, void* work, int sms,
                                      cudaStream_t stream) {
  PrefillParams d = {};
  make_params(a, 0, 0, gate, work, sms, &d);
  return launch(kda_attn_prefill_merge_kernel, dim3((unsigned)sms, kRowsP / kMergeRows),
                dim3(32 * kMergeRows), 0, true, stream, d);
}

}  // namespace attn
}  // namespace kda
