// The accepted branch of a drafted tree moved together in the paged cache: the branch's e-th node
// sits in cache position start + node (start: the cached tokens before the nodes) and goes to
// start + e.  A page that takes entries gets the largest scale of the pages that its kept entries come from
// (its own where it holds cached text), so no entry outgrows e4m3; entries whose scale changes are
// requantised, which for kda_rope_append's powers of two only shifts exponents.
//
// A CTA takes a (sequence, kv head, keys or values) and a page at a time, in order: it reads the entries
// that go there into registers (8 threads an entry of 128 bytes), and writes them after a barrier.  The e-th
// node is never before position start + e, so no page is read after it was written, but for entries of the
// page in work.  A branch that lies together already moves nothing.  Bound by a chain of dependent loads
// (lengths, parents, table, scales and entries), not by bytes: 1.9 us for one sequence, 5.8 for 128 sequences of
// up to 64 nodes, 8 kv heads, pages of 16.
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

using attn::e4m3x4;
using attn::from_e4m3x2;

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;             // entries at a time, 16 bytes a thread
constexpr int kPer = kNodes / kGroups;            // entries of a group at most

__device__ __forceinline__ uint32_t requant(uint32_t w, float f) {
  const float2 a = from_e4m3x2(w & 0xffff), b = from_e4m3x2(w >> 16);
  return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ uint4 requant(const uint4& u, float f) {
  return make_uint4(requant(u.x, f), requant(u.y, f), requant(u.z, f), requant(u.w, f));
}

__global__ void __launch_bounds__(kThreads) kda_tree_accept_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ int links[kNodes], node_s[kNodes], page_s[kNodes];
  __shared__ float scale_s[kNodes];
  const int tid = threadIdx.x, hk = p.c.kv_heads, P = p.c.page_size;
  const int side = blockIdx.x & 1, h = (blockIdx.x >> 1) % hk, seq = (blockIdx.x >> 1) / hk;
  const bool lead = (blockIdx.x >> 1) % hk == 0 && side == 0;      // reports, and writes the length
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  Nodes s;
  int err;
  bool ok = nodes_of(p.cu_seqlens, seq, p.total_tokens, p.max_q_len, &s, &err);
  const int len = p.c.kv_lens[seq];
  const int node = p.accepted[seq];
  if (ok && (len < s.n || (int64_t)len > (int64_t)p.c.max_blocks * P)) {
    err = KDA_ERR_BAD_CACHE_INDEX;
    ok = false;
  }
  if (ok && s.n > 0 && (node < -1 || node >= s.n)) {
    err = KDA_ERR_BAD_TREE;
    ok = false;
  }
  if (!ok || s.n == 0) {
    if (lead && tid == 0) {
      if (!ok) record_error(p.status, err, 410);
      p.lens_out[seq] = len;
    }
    return;
  }
  const uint64_t on = branch_of(p.parents, s, node, links, p.status, lead);
  const int L = __popcll(on), start = len - s.n;
  if (lead && tid == 0) p.lens_out[seq] = start + L;
  // the branch's first nodes that are in place already: those whose lower nodes are all on it
  const int still = on == ~0ull ? kNodes : __ffsll((long long)~on) - 1;
  if (still >= L) return;
  const int32_t* table = p.c.block_table + (int64_t)seq * p.c.table_stride;
  float* scales = side ? p.c.v_scale : p.c.k_scale;
  uint8_t* base = (side ? p.c.v : p.c.k) + h * p.c.head_stride;
  auto page_at = [&](int blk) -> int {       // -1 (reported) for one outside the pool
    const int pg = table[blk];
    if (pg >= 0 && pg < p.c.num_pages) return pg;
    if (lead) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 411);
    return -1;
  };
  // the branch's nodes, the pages they are in and those pages' scales (before any changes)
  if (tid < s.n && ((on >> tid) & 1)) {
    const int e = __popcll(on & ((1ull << tid) - 1)), pg = page_at((start + tid) / P);
    node_s[e] = tid;
    page_s[e] = pg;
    scale_s[e] = pg < 0 ? 0.0f : scales[(int64_t)pg * p.c.scale_stride + h];
  }
  __syncthreads();
  const int g = tid >> 3, c = (tid & 7) * 16;
  for (int blk = (start + still) / P; blk <= (start + L - 1) / P; ++blk) {
    const int first = max(0, blk * P - start), last = min(L, (blk + 1) * P - start);   // entries [first, last)
    const int kept = max(0, start - blk * P);                                          // cached text's
    const int to = page_at(blk);
    float own = 1.0f, top = 0.0f;
    if (to >= 0) own = scales[(int64_t)to * p.c.scale_stride + h];
    if (kept > 0) top = own;
    for (int e = first; e < last; ++e) top = fmaxf(top, scale_s[e]);
    uint4 u[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = first + g + kGroups * j;
      if (e < last && page_s[e] >= 0)
        u[j] = *reinterpret_cast<const uint4*>(base + (int64_t)page_s[e] * p.c.page_stride +
                                               (int64_t)((start + node_s[e]) % P) * p.c.token_stride + c);
    }
    __syncthreads();       // (and everybody has the page's scale)
    if (to >= 0) {
      uint8_t* dst = base + (int64_t)to * p.c.page_stride;
      if (own != top) {
        for (int i = g; i < kept; i += kGroups) {
          uint4* w = reinterpret_cast<uint4*>(dst + (int64_t)i * p.c.token_stride + c);
          *w = requant(*w, own / top);
        }
        if (tid == 0) scales[(int64_t)to * p.c.scale_stride + h] = top;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = first + g + kGroups * j;
        if (e < last && page_s[e] >= 0)
          *reinterpret_cast<uint4*>(dst + (int64_t)((start + e) % P) * p.c.token_stride + c) =
              scale_s[e] == top ? u[j] : requant(u[j], scale_s[e] / top);
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t stream) {
  const int64_t ctas = (int64_t)p.num_seqs * p.c.kv_heads * 2;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return attn::launch(kda_tree_accept_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, true, stream, p);
}

}  // namespace tree
}  // namespace kda
