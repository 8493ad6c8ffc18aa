// Trees of drafted tokens: what the operators on them share.  A tree's nodes are a sequence's new
// tokens, at most KDA_TREE_NODES; node i follows node parents[i] < i of the same sequence, or the
// cached text (-1).
#pragma once

#include "kda_attn.cuh"

namespace kda {
namespace tree {

constexpr int kNodes = KDA_TREE_NODES;

// The nodes of one sequence of a batch.
struct Nodes {
  int tok0, n;        // first row, nodes
};
// False, with the code to record in *err, for a malformed sequence.
__device__ __forceinline__ bool nodes_of(const int32_t* cu, int seq, int64_t total, int max_q_len,
                                         Nodes* s, int* err) {
  const int t0 = cu[seq], t1 = cu[seq + 1];
  s->tok0 = t0;
  s->n = t1 - t0;
  *err = KDA_OK;
  if (t0 < 0 || t1 < t0 || (int64_t)t1 > total || (seq == 0 && t0 != 0)) *err = KDA_ERR_BAD_CU_SEQLENS;
  else if (s->n > max_q_len) *err = KDA_ERR_INVALID_ARG;
  return *err == KDA_OK;
}
// Node i's parent, -1 for one out of range.
__device__ __forceinline__ int parent_of(const int32_t* parents, const Nodes& s, int i, int* status,
                                         bool report) {
  const int p = parents[s.tok0 + i];
  if (p >= -1 && p < i) return p;
  if (report) record_error(status, KDA_ERR_BAD_TREE, 400);
  return -1;
}

struct PlanParams {
  const int32_t* parents;
  const int32_t* cu_seqlens;
  const int32_t* kv_lens;
  uint64_t* mask;
  int32_t* positions;
  int* status;
  int64_t total_tokens;
  int32_t num_seqs, max_q_len;
};
cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream);

// A sequence's accepted branch, for a CTA's threads: parents into `links` (shared, kNodes ints), then
// the nodes from the cached text to `node` as bits.  Every warp walks by itself.  Barriers inside.
__device__ __forceinline__ uint64_t branch_of(const int32_t* parents, const Nodes& s, int node, int* links,
                                              int* status, bool report) {
  for (int i = threadIdx.x; i < s.n; i += blockDim.x) links[i] = parent_of(parents, s, i, status, report);
  __syncthreads();
  uint64_t on = 0;
  for (int i = node; i >= 0; i = links[i]) on |= 1ull << i;
  return on;
}

struct AcceptParams {
  attn::CacheView c;
  const int32_t* cu_seqlens;
  const int32_t* parents;
  const int32_t* accepted;
  int32_t* lens_out;
  int* status;
  int64_t total_tokens;
  int32_t num_seqs, max_q_len;
};
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t stream);

// The KDA recurrence along trees.  q, k, v, g, beta: bf16, a token's heads dense, strides between tokens.
struct RecurParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* g;
  const __nv_bfloat16* beta;
  int64_t s_q, s_k, s_v, s_g, s_beta;
  const float* A_log;
  const float* dt_bias;
  float lower_bound, scale;
  const void* initial_state;   // [num_seqs, heads, 128, 128] or null (zeros)
  int state_bf16;
  const int32_t* cu_seqlens;
  const int32_t* parents;
  __nv_bfloat16* out;          // [total_tokens, heads, 128]
  float* u;                    // [total_tokens, heads, 128]
  const int32_t* accepted;     // commit: [num_seqs]
  void* final_state;           // commit
  int* status;
  int64_t total_tokens;
  int32_t num_seqs, heads, max_q_len;
};
cudaError_t launch_recur(const RecurParams& p, int sms, cudaStream_t stream);
cudaError_t launch_commit(const RecurParams& p, cudaStream_t stream);

}  // namespace tree
}  // namespace kda
