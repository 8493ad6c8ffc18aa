// Masks and positions of drafted trees:
//   mask_i = bit i | mask_parent(i)        position_i = kv_len - n + depth_i,  depth_i = |mask_i| - 1
// A warp takes a sequence, a lane two of its nodes.  Masks double: after k steps a node's mask holds
// itself and its 2^k - 1 nearest ancestors, and its link the 2^k-th; a chain of 64 nodes then takes six
// steps instead of 63.  Nothing to read or write that counts (16 bytes a node): bound by the launch and
// three dependent loads (cu_seqlens, parents, the steps in shared memory): 1.2 us for one tree of 8 nodes, 1.8 for
// 512 trees of up to 64.
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

constexpr int kWarps = 4;      // sequences of a CTA

__global__ void __launch_bounds__(32 * kWarps) kda_tree_plan_kernel(const PlanParams p) {
  __shared__ uint64_t masks[kWarps][kNodes];
  __shared__ int links[kWarps][kNodes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seq = blockIdx.x * kWarps + warp;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  if (seq >= p.num_seqs) return;
  Nodes s;
  int err;
  bool ok = nodes_of(p.cu_seqlens, seq, p.total_tokens, p.max_q_len, &s, &err);
  const int len = p.kv_lens[seq];
  if (ok && len < s.n) {
    err = KDA_ERR_BAD_CACHE_INDEX;
    ok = false;
  }
  if (!ok) {
    if (lane == 0) record_error(p.status, err, 401);
    return;
  }
  uint64_t m[2];
  int up[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    m[j] = 1ull << i;
    up[j] = i < s.n ? parent_of(p.parents, s, i, p.status, true) : -1;
  }
  while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      masks[warp][lane + 32 * j] = m[j];
      links[warp][lane + 32 * j] = up[j];
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (up[j] >= 0) {
        m[j] |= masks[warp][up[j]];
        up[j] = links[warp][up[j]];
      }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    if (i >= s.n) continue;
    p.mask[s.tok0 + i] = m[j];
    p.positions[s.tok0 + i] = len - s.n + __popcll(m[j]) - 1;
  }
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  return attn::launch(kda_tree_plan_kernel, dim3((unsigned)((p.num_seqs + kWarps - 1) / kWarps)),
                      dim3(32 * kWarps), 0, true, stream, p);
}

}  // namespace tree
}  // namespace kda
