// Attention over the paged e4m3 cache: which kernel takes which sequences of a call.
#include "kda_attn_tc.cuh"

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

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

// Rows (new tokens x heads per kv head) of a sequence that go to the decode kernel: up to 32.
int decode_rows(int64_t rows, int group) {
  return group > kDecodeRows ? 0 : (int)(rows < kDecodeRows ? rows : kDecodeRows);
}

}  // namespace

size_t attn_workspace_bytes(int32_t num_seqs, int32_t heads, int32_t kv_heads, int32_t max_q_len) {
  (void)num_seqs;
  const int sms = device_sms(), group = heads / kv_heads;
  const int64_t rows = (int64_t)max_q_len * group;
  const int few = decode_rows(rows, group);
  return (size_t)kWorkspaceBytes + (few > 0 ? align16(decode_workspace_bytes(sms)) : 0) +
         (rows > few ? prefill_workspace_bytes(sms) : 0);
}

// Sequences with at most 32 rows per kv head take the decode kernel, the others of the same call
// the prefill kernel.  A launch is left out when the sizes say that no sequence can need it: none
// can have more rows than max_q_len gives, and with num_seqs * max_q_len tokens in the batch all
// have that many.  With both, the prefill kernel is launched as the decode kernel's dependent and
// waits for nothing (its CTAs start as SMs come free), the first merge is an ordinary launch
// behind both, and the second one runs beside it.
cudaError_t launch_attn(const AttnParams& p, int sms, cudaStream_t stream) {
  const int group = p.heads / p.c.kv_heads;
  const int64_t rows = (int64_t)p.max_q_len * group;
  const int most = decode_rows(rows, group);
  const bool many = rows > most;
  const int few = many && p.total_tokens == (int64_t)p.num_seqs * p.max_q_len ? 0 : most;
  char* work = reinterpret_cast<char*>(p.status) + kWorkspaceBytes;
  char* work2 = work + (most > 0 ? align16(decode_workspace_bytes(sms)) : 0);
  CacheMaps maps;
  if (!make_cache_maps(p.c, &maps)) return cudaErrorNotSupported;
  cudaError_t e = cudaSuccess;
  if (few > 0 && (e = launch_attn_decode(p, maps, few, work, sms, stream)) != cudaSuccess) return e;
  if (many && (e = launch_attn_prefill(p, maps, few + 1, work2, sms, few > 0, stream)) != cudaSuccess) return e;
  if (few > 0 && (e = launch_attn_decode_merge(p, few, work, sms, !many, stream)) != cudaSuccess) return e;
  return many ? launch_attn_prefill_merge(p, few + 1, work2, sms, few == 0, stream) : cudaSuccess;
}

}  // namespace attn
}  // namespace kda
