// Pages of the cache given back, shared, copied and reserved, on the device, so that a decode loop
// with a changing batch can be captured whole.
//
// The pool's state is the count of rows that hold each page; a free page has 0.  Whoever needs pages gets the
// lowest free ones, in the order of rows and blocks: the outcome does not depend on the order in
// which threads run, and there is no list of free pages to keep.  The search is one CTA's scan over the
// counts, 16384 at a time, which ends at the page that serves the last request; a page that is
// found knows its rank, and the rank the request (a binary search over the requests' prefix sums in
// shared memory).  The first counts are on their way while the requests are counted (the next ones
// as well: 19.4 us; an SM's loads bound the scan).  Counts go up
// and down by atomics on integers, whose order does not show.
//
// Nothing here moves bytes that count; each call is a launch and a chain of dependent loads.  64 rows ended,
// forked from 16 prompts of up to 65535 tokens, their last pages copied (2 kv heads, pages of 64) and 64 tokens a
// row reserved, in a pool of 24000 pages: 18.4 us for the four calls, about 3, 5.6, 2 and 7.6 (0.6 of the last for the
// counts of the pages that take new tokens).  Where the low pages are held the search walks over them: a page for each
// of 64 rows takes 8 us if the free ones are the last of 24000, 26 of 150,000 and 140 of a million, and a fork the same.
#include "kda_pages.cuh"

namespace kda {
namespace pages {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// Exclusive prefix of v over the CTA, and the sum; `part` has kWarps + 1 ints.  Barriers inside.
__device__ __forceinline__ int block_scan(int v, int* part, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();       // (the sums of the scan before have been read)
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = part[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    part[lane] = s - w;
    if (lane == 31) part[kWarps] = s;
  }
  __syncthreads();
  *sum = part[kWarps];
  return part[warp] + inc - v;
}

// Exclusive prefix over the CTA's warps of a number that a warp's lanes have in common, and the sum.
__device__ __forceinline__ int warp_scan(int v, int* part, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();       // (the sums of the scan before have been read)
  if (lane == 0) part[warp] = v;
  __syncthreads();
  const int w = part[lane];
  int inc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  *sum = __shfl_sync(0xffffffffu, inc, 31);
  return __shfl_sync(0xffffffffu, inc - w, warp);
}

// A CTA's look at the counts: warp w takes 512 pages from 512 w on, 32 at a time.
constexpr int kLooks = 16, kChunk = kWarps * 32 * kLooks;
struct Counts {
  int32_t r[kLooks];
  __device__ __forceinline__ void load(const int32_t* refs, int num_pages, int64_t p0) {
    const int64_t base = p0 + (threadIdx.x >> 5) * (32 * kLooks) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < kLooks; ++j) r[j] = base + 32 * j < num_pages ? refs[base + 32 * j] : 1;
  }
};
// Calls give(rank, page) for the first `total` free pages; false when there are fewer.  For a whole CTA, with
// the counts of the first kChunk pages loaded.  (A lane a page: with 16 neighbouring pages a thread a few
// threads gave all of them, one after the other.)
template <class Give>
__device__ bool find_free(const int32_t* refs, int num_pages, int total, int* part, Counts& c, Give give) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int64_t p0 = 0; p0 < num_pages && before < total; p0 += kChunk) {
    if (p0 > 0) c.load(refs, num_pages, p0);
    uint32_t free[kLooks];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kLooks; ++j) {
      free[j] = __ballot_sync(0xffffffffu, c.r[j] == 0);
      mine += __popc(free[j]);
    }
    int found;
    int rank = before + warp_scan(mine, part, &found);
    const int64_t base = p0 + warp * (32 * kLooks) + lane;
#pragma unroll
    for (int j = 0; j < kLooks; ++j) {
      const int r = rank + __popc(free[j] & ((1u << lane) - 1));
      if (((free[j] >> lane) & 1) && r < total) give(r, (int)(base + 32 * j));
      rank += __popc(free[j]);
    }
    before += found;
  }
  return before >= total;
}

// The request that takes rank r: the last i with first[i] <= r (first[0] = 0, non-decreasing).
__device__ __forceinline__ int request_of(const int* first, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

constexpr int kFreeThreads = 256;
__global__ void __launch_bounds__(kFreeThreads)
    kda_pages_free_kernel(const Pool p, const int32_t* rows) {
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int row = rows ? rows[blockIdx.x] : (int)blockIdx.x;
  if (row < 0 || row >= p.num_rows) {
    if (threadIdx.x == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 420);
    return;
  }
  int first = 0;
  if (rows) {
    if (threadIdx.x == 0) p.kv_lens[row] = 0;
  } else {
    const int len = p.kv_lens[row];
    if (len < 0 || (int64_t)len > (int64_t)p.max_blocks * p.page_size) {
      if (threadIdx.x == 0) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 421);
      return;
    }
    first = (len + p.page_size - 1) / p.page_size;
  }
  int32_t* table = p.table + (int64_t)row * p.table_stride;
  // (four entries of a thread in flight: each takes three trips to memory)
  constexpr int kAhead = 4;
  for (int b0 = first + threadIdx.x; b0 < p.max_blocks; b0 += kFreeThreads * kAhead) {
    int pg[kAhead], held[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      pg[j] = b0 + kFreeThreads * j < p.max_blocks ? table[b0 + kFreeThreads * j] : -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)        // (a row that is named twice gives its pages once)
      if (pg[j] != -1) pg[j] = atomicExch(table + b0 + kFreeThreads * j, -1);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      held[j] = 1;
      if (pg[j] >= 0 && pg[j] < p.num_pages) held[j] = atomicSub(p.refs + pg[j], 1);
      else if (pg[j] != -1) record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 422);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (held[j] <= 0) {                    // nobody held it
        atomicAdd(p.refs + pg[j], 1);
        record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 423);
      }
  }
}

// One CTA: requests counted and scanned, then served.
__global__ void __launch_bounds__(kThreads)
    kda_pages_reserve_kernel(const Pool p, const int32_t* new_tokens) {
  extern __shared__ int smem[];
  int* first = smem;                 // [num_rows] prefix sums of the requests
  int* start = smem + p.num_rows;    // [num_rows] first block of each
  __shared__ int part[kWarps + 1];
  const int lane = threadIdx.x & 31;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  Counts counts;
  counts.load(p.refs, p.num_pages, 0);
  int total = 0;
  for (int r0 = 0; r0 < p.num_rows; r0 += kThreads) {
    const int row = r0 + threadIdx.x;
    int b = 0, end = 0, bad = 0;
    bool begun = false;         // the first block holds cached text
    if (row < p.num_rows) {
      const int64_t len = p.kv_lens[row], add = new_tokens[row];
      const int64_t need = (len + add + p.page_size - 1) / p.page_size;
      if (len < 0 || add < 0 || need > p.max_blocks) {
        bad = 1;
      } else if (add > 0) {
        b = (int)(len / p.page_size);
        end = (int)need;
        begun = len % p.page_size != 0;
      }
    }
    // empty blocks from the first empty one on: a lane its own row, or the warp a long one together.  A page
    // before them takes new tokens: it has to be this row's alone (kv_lens may have been set back into one that
    // a fork shares).
    auto others = [&](int pg) { return pg < 0 || pg >= p.num_pages || p.refs[pg] != 1; };
    int at = b;
    const int32_t* table = p.table + (int64_t)row * p.table_stride;
    const bool far = end - b > 8;
    if (!far) {
      uint32_t empty = 0;
      int pg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pg[j] = b + j < end ? table[b + j] : -1;
        empty |= (uint32_t)(b + j < end && pg[j] == -1) << j;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) bad |= pg[j] != -1 && others(pg[j]);
      at = empty ? b + __ffs(empty) - 1 : end;
      bad |= at < end && (empty >> (at - b)) != (1u << (end - at)) - 1;      // a page behind an empty block
    }
    uint32_t todo = __ballot_sync(0xffffffffu, far);
    while (todo) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const int bk = __shfl_sync(0xffffffffu, b, k), ek = __shfl_sync(0xffffffffu, end, k);
      const int32_t* t = p.table + (int64_t)(row - lane + k) * p.table_stride;
      int found = ek, wrong = 0;
      for (int i0 = bk; i0 < ek; i0 += 32) {
        const bool in = i0 + lane < ek;
        const int pg = in ? t[i0 + lane] : -1;
        const bool empty = in && pg == -1;
        const uint32_t e = __ballot_sync(0xffffffffu, empty), f = __ballot_sync(0xffffffffu, in && !empty);
        if (__any_sync(0xffffffffu, in && !empty && others(pg))) wrong = 1;
        if (found == ek && e) found = i0 + __ffs(e) - 1;
        // a page behind an empty block
        if (found < ek && (f >> max(0, found - i0)) != 0 && i0 + 31 >= found) wrong = 1;
      }
      if (lane == k) {
        at = found;
        bad |= wrong;
      }
    }
    // (an empty page in the place of cached text, as after a fork that found none, would pass for it)
    if (bad || (begun && at == b)) {
      record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 424);
      at = end;
    }
    int sum;
    const int before = total + block_scan(end - at, part, &sum);
    if (row < p.num_rows) {
      first[row] = before;
      start[row] = at;
    }
    total += sum;
  }
  __syncthreads();
  const bool enough = find_free(p.refs, p.num_pages, total, part, counts, [&](int rank, int page) {
    const int row = request_of(first, p.num_rows, rank);
    p.table[(int64_t)row * p.table_stride + start[row] + rank - first[row]] = page;
    p.refs[page] = 1;
  });
  if (!enough && threadIdx.x == 0) record_error(p.status, KDA_ERR_OUT_OF_PAGES, 425);
}

// CTA 0 finds the pages for the partial last ones; the others share whole pages, a row each.  A pair is in
// order when its rows exist, its source's length fits the table, and no other pair writes to its dst
// or reads from it: then nothing that one CTA reads is another's to write.
constexpr int kIsSource = 1 << 30;
__global__ void __launch_bounds__(kThreads)
    kda_pages_fork_kernel(const Pool p, const int32_t* src, const int32_t* dst, int num, int32_t* from,
                          int32_t* to) {
  extern __shared__ int smem[];
  int* found = smem;                 // [num] the pages that were found, in order
  int* rank = smem + num;            // [num] which of them is a pair's, or -1
  int* uses = smem + 2 * num;        // [num_rows] pairs that write to the row, and whether one reads it
  __shared__ int part[kWarps + 1];
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  if (blockIdx.x > 0) {
    const int i = blockIdx.x - 1;
    const int s = src[i], d = dst[i];
    bool mine = true;
    for (int j = threadIdx.x; j < num; j += kThreads) mine = mine && src[j] != d && (j == i || dst[j] != d);
    if (!__syncthreads_and(mine) || s < 0 || s >= p.num_rows || d < 0 || d >= p.num_rows) return;
    const int len = p.kv_lens[s];
    if (len < 0 || (int64_t)len > (int64_t)p.max_blocks * p.page_size) return;
    const int whole = len / p.page_size, tail = len % p.page_size > 0 ? whole : -1;
    const int32_t* a = p.table + (int64_t)s * p.table_stride;
    int32_t* b = p.table + (int64_t)d * p.table_stride;
    for (int x = threadIdx.x; x < p.max_blocks; x += kThreads) {
      if (x == tail) continue;
      int pg = -1;
      if (x < whole) {
        pg = a[x];
        if (pg < 0 || pg >= p.num_pages) {
          record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 426);
          pg = -1;
        } else {
          atomicAdd(p.refs + pg, 1);
        }
      }
      b[x] = pg;
    }
    return;
  }
  Counts counts;        // (a page that the other CTAs share is held by its source already)
  counts.load(p.refs, p.num_pages, 0);
  for (int r = threadIdx.x; r < p.num_rows; r += kThreads) uses[r] = 0;
  __syncthreads();
  // a pair's rows, its source's length (-1: out of range) and last page; the first ones loaded at once
  auto load = [&](int i, int& s, int& d, int& len, int& last) {
    s = d = len = last = -1;
    if (i >= num) return;
    s = src[i];
    d = dst[i];
    if (s < 0 || s >= p.num_rows) return;
    len = p.kv_lens[s];
    if ((int64_t)len > (int64_t)p.max_blocks * p.page_size) len = -1;
    if (len > 0 && len % p.page_size) last = p.table[(int64_t)s * p.table_stride + len / p.page_size];
  };
  int s, d, len, last;
  load(threadIdx.x, s, d, len, last);
  for (int i = threadIdx.x; i < num; i += kThreads) {
    const int a = src[i], b = dst[i];
    if (a >= 0 && a < p.num_rows) atomicOr(uses + a, kIsSource);
    if (b >= 0 && b < p.num_rows) atomicAdd(uses + b, 1);
  }
  __syncthreads();
  int total = 0;
  for (int i0 = 0; i0 < num; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < num) {
      int pg = -1;
      if (i0 > 0) load(i, s, d, len, last);
      if (!(len >= 0 && d >= 0 && d < p.num_rows && uses[d] == 1)) {
        record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 427);
      } else {
        p.kv_lens[d] = len;
        if (len % p.page_size) {
          pg = last;
          need = 1;
          p.table[(int64_t)d * p.table_stride + len / p.page_size] = -1;
          if (pg < 0 || pg >= p.num_pages) {
            record_error(p.status, KDA_ERR_BAD_CACHE_INDEX, 428);
            need = 0;
            pg = -1;
          }
        }
      }
      from[i] = pg;
    }
    int sum;
    const int before = total + block_scan(need, part, &sum);
    if (i < num) {
      rank[i] = need ? before : -1;
      found[i] = -1;
    }
    total += sum;
  }
  __syncthreads();
  const bool enough = find_free(p.refs, p.num_pages, total, part, counts, [&](int r, int page) {
    found[r] = page;
    p.refs[page] = 1;
  });
  __syncthreads();
  // (a thread with one pair has its rows still)
  for (int i = threadIdx.x; i < num; i += kThreads) {
    const int page = rank[i] >= 0 ? found[rank[i]] : -1;
    to[i] = page;
    if (page < 0) continue;
    if (num > kThreads) load(i, s, d, len, last);
    p.table[(int64_t)d * p.table_stride + len / p.page_size] = page;
  }
  if (!enough && threadIdx.x == 0) record_error(p.status, KDA_ERR_OUT_OF_PAGES, 429);
}

// A CTA copies one side of one head of a page: page_size rows of 128 bytes, eight threads a row.
constexpr int kCopyThreads = 128;
__global__ void __launch_bounds__(kCopyThreads)
    kda_pages_copy_kernel(const __grid_constant__ attn::CacheView c, const int32_t* from, const int32_t* to,
                          int* status) {
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int units = 2 * c.kv_heads, i = blockIdx.x / units, h = (blockIdx.x % units) >> 1, side = blockIdx.x & 1;
  const int a = from[i], b = to[i];
  if (a < 0 || b < 0 || a == b) return;
  if (a >= c.num_pages || b >= c.num_pages) {
    if (threadIdx.x == 0) record_error(status, KDA_ERR_BAD_CACHE_INDEX, 430);
    return;
  }
  uint8_t* base = (side ? c.v : c.k) + h * c.head_stride + (threadIdx.x & 7) * 16;
  const uint8_t* src = base + (int64_t)a * c.page_stride;
  uint8_t* dst = base + (int64_t)b * c.page_stride;
  constexpr int kRows = kCopyThreads / 8, kAhead = 4;
  for (int r0 = threadIdx.x >> 3; r0 < c.page_size; r0 += kRows * kAhead) {
    uint4 u[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (r0 + kRows * j < c.page_size)
        u[j] = *reinterpret_cast<const uint4*>(src + (int64_t)(r0 + kRows * j) * c.token_stride);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (r0 + kRows * j < c.page_size)
        *reinterpret_cast<uint4*>(dst + (int64_t)(r0 + kRows * j) * c.token_stride) = u[j];
  }
  if (threadIdx.x == 0) {
    float* s = side ? c.v_scale : c.k_scale;
    s[(int64_t)b * c.scale_stride + h] = s[(int64_t)a * c.scale_stride + h];
  }
}

cudaError_t allow_smem(const void* kernel, PerDeviceOnce& once, int bytes) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once.run(dev, [&]() -> cudaError_t {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

}  // namespace

cudaError_t launch_free(const Pool& p, const int32_t* rows, int32_t num, cudaStream_t stream) {
  return attn::launch(kda_pages_free_kernel, dim3((unsigned)(rows ? num : p.num_rows)), dim3(kFreeThreads), 0,
                      true, stream, p, rows);
}

cudaError_t launch_reserve(const Pool& p, const int32_t* new_tokens, cudaStream_t stream) {
  static PerDeviceOnce once;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kda_pages_reserve_kernel), once,
                                   kMaxRows * 8);
  if (e != cudaSuccess) return e;
  return attn::launch(kda_pages_reserve_kernel, dim3(1), dim3(kThreads), (size_t)p.num_rows * 8, true, stream,
                      p, new_tokens);
}

cudaError_t launch_fork(const Pool& p, const int32_t* src, const int32_t* dst, int32_t num, int32_t* from,
                        int32_t* to, cudaStream_t stream) {
  static PerDeviceOnce once;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kda_pages_fork_kernel), once, kMaxRows * 12);
  if (e != cudaSuccess) return e;
  return attn::launch(kda_pages_fork_kernel, dim3((unsigned)num + 1), dim3(kThreads), (size_t)(2 * num + p.num_rows) * 4, true,
                      stream, p, src, dst, num, from, to);
}

cudaError_t launch_copy(const attn::CacheView& c, const int32_t* from, const int32_t* to, int64_t num,
                        int* status, cudaStream_t stream) {
  const int64_t ctas = num * c.kv_heads * 2;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return attn::launch(kda_pages_copy_kernel, dim3((unsigned)ctas), dim3(kCopyThreads), 0, true, stream, c, from,
                      to, status);
}

}  // namespace pages
}  // namespace kda
