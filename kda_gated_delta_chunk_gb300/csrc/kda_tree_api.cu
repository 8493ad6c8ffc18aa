// C entry points of the operators on drafted trees: argument checks and dispatch.  Declared in
// include/kda.h.
#include "kda_checks.cuh"
#include "kda_tree.cuh"

using namespace kda::checks;

namespace {

// What every call on trees is checked for.
int check_trees(const void* cu_seqlens, const void* parents, const void* workspace, int64_t total_tokens,
                int32_t num_seqs, int32_t max_q_len, size_t workspace_bytes) {
  if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0 || !cu_seqlens || !workspace)
    return KDA_ERR_INVALID_ARG;
  if (max_q_len < 0 || max_q_len > KDA_TREE_NODES) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!parents || max_q_len < 1)) return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(cu_seqlens, 4) || !aligned(parents, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_tree_plan(const int32_t* parents, const int32_t* cu_seqlens, const int32_t* kv_lens,
                  void* mask, int32_t* positions, void* workspace, kda_stream_t stream,
                  int64_t total_tokens, int32_t num_seqs, int32_t max_q_len, size_t workspace_bytes) {
  int rc = check_trees(cu_seqlens, parents, workspace, total_tokens, num_seqs, max_q_len, workspace_bytes);
  if (rc != KDA_OK) return rc;
  if (num_seqs > 0 && !kv_lens) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!mask || !positions)) return KDA_ERR_INVALID_ARG;
  if (!aligned(kv_lens, 4) || !aligned(mask, 8) || !aligned(positions, 4)) return KDA_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device(&sms);
  if (rc != KDA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
  kda::tree::PlanParams p{};
  p.parents = parents;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = kv_lens;
  p.mask = static_cast<uint64_t*>(mask);
  p.positions = positions;
  p.status = static_cast<int*>(workspace);
  p.total_tokens = total_tokens;
  p.num_seqs = num_seqs;
  p.max_q_len = max_q_len;
  return launched(kda::tree::launch_plan(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
