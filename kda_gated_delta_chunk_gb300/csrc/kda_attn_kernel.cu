// Attention over the paged e4m3 cache: which kernel takes which sequences of a call.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kDecodeRows = 32;    // query rows per kv head that the decode kernel takes at most

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    sms = kDefaultSmCount;
  }
  return sms;
}

// Rows (new tokens x heads per kv head) of a sequence that go to the decode kernel: up to 32.
int decode_rows(int64_t rows, int group) {
  return group > kDecodeRows ? 0 : (int)(rows < kDecodeRows ? rows : kDecodeRows);
}

}  // namespace

size_t attn_workspace_bytes(int32_t num_seqs, int32_t heads, int32_t kv_heads, int32_t max_q_len) {
  (void)num_seqs;
  const int sms = device_sms(), group = heads / kv_heads;
  const int64_t rows = (int64_t)max_q_len * group;
  size_t need = 0;
  if (decode_rows(rows, group) > 0) need = decode_workspace_bytes(sms);
  if (rows > decode_rows(rows, group)) need = need > prefill_workspace_bytes(sms) ? need : prefill_workspace_bytes(sms);
  return (size_t)kWorkspaceBytes + need;
}

// Sequences with at most 32 rows per kv head take the decode kernel, the others of the same call
// the prefill kernel; a launch is left out when max_q_len says that no sequence can need it.  The
// two run one after the other and share the area for partial results.
cudaError_t launch_attn(const AttnParams& p, int sms, cudaStream_t stream) {
  const int group = p.heads / p.c.kv_heads;
  const int64_t rows = (int64_t)p.max_q_len * group;
  const int few = decode_rows(rows, group);
  char* work = reinterpret_cast<char*>(p.status) + kWorkspaceBytes;
  if (few > 0) {
    const cudaError_t e = launch_attn_decode(p, 1, few, work, sms, stream);
    if (e != cudaSuccess) return e;
  }
  return rows > few ? launch_attn_prefill(p, few + 1, work, sms, stream) : cudaSuccess;
}

}  // namespace attn
}  // namespace kda
