// Attention over the paged e4m3 cache: which kernel takes which sequences of a call.
#include <atomic>

#include "kda_attn_tc.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kDecodeRows = 32;    // query rows per kv head that the decode kernel takes at most
// Units (key tiles, and kOver an item) of such sequences per SM below which the prefill kernel takes
// them with its own.  A tile of few rows takes it over twice the decode kernel's time, but a decode
// kernel on the same SMs costs about ten microseconds of launch, start and end.  16 heads over 4, with one
// prefill of 1024 tokens | four over 4096 keys each, decode kernel against prefill kernel: 16
// sequences of 4096 tokens (14.7 units per SM) 63.6 : 57.8 us | 153.5 : 144.3 us, 32 (29.5 units)
// 80.9 : 88.5 | 169.2 : 166.0, 64 (59 units) 113.7 : 139.8 | 202.0 : 210.8.
constexpr int kFewUnits = 20;

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    sms = kDefaultSmCount;
  }
  return sms;
}

// Numbers calls that run both kernels, from 1.
int call_number() {
  static std::atomic<unsigned> calls{0};
  return (int)(calls.fetch_add(1) & 0x3fffffffu) + 1;
}

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

// Rows (new tokens x heads per kv head) of a sequence that go to the decode kernel: up to 32.
int decode_rows(int64_t rows, int group) {
  return group > kDecodeRows ? 0 : (int)(rows < kDecodeRows ? rows : kDecodeRows);
}

}  // namespace

// The parts that some call with at most these sizes lays out: one with fewer heads or kv heads
// may have a larger group and need what this one does not.
size_t attn_workspace_bytes(int32_t heads, int32_t max_q_len) {
  const int sms = device_sms();
  return (size_t)kWorkspaceBytes + (max_q_len > 0 ? align16(decode_workspace_bytes(sms)) : 0) +
         ((int64_t)heads * max_q_len > kDecodeRows ? prefill_workspace_bytes(sms) : 0);
}

size_t attn_call_bytes(int32_t heads, int32_t kv_heads, int32_t max_q_len) {
  const int sms = device_sms(), group = heads / kv_heads;
  const int64_t rows = (int64_t)max_q_len * group;
  const int few = decode_rows(rows, group);
  return (size_t)kWorkspaceBytes + (few > 0 ? align16(decode_workspace_bytes(sms)) : 0) +
         (rows > few ? prefill_workspace_bytes(sms) : 0);
}

// Sequences with at most 32 rows per kv head take the decode kernel, the others of the same call
// the prefill kernel, which takes the first ones too when they are few (both kernels find that out
// from the lengths on the device).  A launch is left out when the sizes say that no sequence can
// need it: none can have more rows than max_q_len gives, and with num_seqs * max_q_len tokens in
// the batch all have that many.  With both, the decode kernel runs beside the prefill kernel
// (kda_attn_tc.cuh; its CTAs start as SMs come free) and does not end before that has; the first merge
// waits for the decode kernel and so for both, the second one for the first.  Decode kernel after the
// prefill kernel's end, 16 heads over 4: 16 ragged sequences 85.5 us against 81.2, without a window
// 128.9 : 123.1, 64 of 4096 to 8192 keys 453.5 : 438.0.
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
  const bool both = many && few > 0;
  const int64_t least = both ? (int64_t)kFewUnits * sms : 0;
  const int gate = both ? call_number() : 0;
  if (many && (e = launch_attn_prefill(p, maps, few, least, gate, work2, sms, stream)) != cudaSuccess) return e;
  if (few > 0 && (e = launch_attn_decode(p, maps, few, least, gate, work, sms, stream)) != cudaSuccess) return e;
  if (few > 0 && (e = launch_attn_decode_merge(p, few, work, sms, stream)) != cudaSuccess) return e;
  return many ? launch_attn_prefill_merge(p, gate, work2, sms, stream) : cudaSuccess;
}

}  // namespace attn
}  // namespace kda
