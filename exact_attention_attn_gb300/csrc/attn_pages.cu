// Pages of a KV cache: block tables and slot maps from request lengths, and
// pages given back, without the host knowing a length.
//
// assign: request r holds len_r tokens in ceil(len_r / P) pages and gets new_r
//   more.  need_r = ceil((len_r + new_r) / P) - ceil(len_r / P); with exclusive
//   sums over the requests, its pages are the free stack's entries
//   count - 1 - (sum need before r) - j, and its tokens are numbers
//   cu_r = sum new before r, ... of the step.  Token n of request r at
//   position p = len_r + n - cu_r lives in slot table[r][p / P] * P + p % P.
// release: request r keeps keep_r tokens; its pages from ceil(keep_r / P) on
//   go back on the stack in request order.
//
// Both are one launch of one thread-block cluster (1 to 8 CTAs, by the size
// of what is written).  Every CTA scans all requests itself -- a few thousand
// integers from L2 -- and reaches the same verdict, so no CTA waits for
// another's sums and no workspace is kept; one cluster barrier separates the
// reads of the state from its update, which makes updates in place safe.
// Latency bound: the scan, then a search in shared memory per four tokens, and
// one more past each run of idle requests between them (a decode step of 64
// requests 4.6 us from a graph, 512 slots of which two are active 5.5, 16384 of
// them 26; 512 prompts of 44 Ki tokens 9.8 us on 8 SMs, 12.0 with CTAs of 512
// threads, 8.1 with clusters of 16, which not every device grants: below the 11 us
// that the host's call takes anyway; release of 16384 pages of 64 requests 31 us,
// of 512 requests 15.5).
#include <stdint.h>
#include <string.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;

struct PagesParams {
  int *table;
  int64_t table_stride;
  int max_pages, P, shift;
  const int *lens;
  int *lens_out;
  const int *arg;  // new lengths (assign) or kept lengths (release)
  int *free_pages;
  int free_capacity;
  const int *free_count;
  int *free_count_out;
  int B, max_tokens;
  int *cu, *slots, *positions, *info;
  const int *after;  // info of a call that must not have been refused, or nullptr
};

// Inclusive sums of v over the warp's lanes.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive sums of (a, b) over the block's threads; the block totals in ta,
// tb.  The warps' totals are summed by every warp, one a lane.
__device__ __forceinline__ void block_scan(long long &a, long long &b, long long &ta, long long &tb) {
  __shared__ long long wa[kMaxWarps], wb[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const long long ia = warp_scan(a, lane), ib = warp_scan(b, lane);
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  const long long sa = warp_scan(lane < warps ? wa[lane] : 0, lane), sb = warp_scan(lane < warps ? wb[lane] : 0, lane);
  const int before = (warp - 1) & 31;  // (the first warp has none)
  const long long pa = __shfl_sync(0xffffffffu, sa, before), pb = __shfl_sync(0xffffffffu, sb, before);
  ta = __shfl_sync(0xffffffffu, sa, 31);
  tb = __shfl_sync(0xffffffffu, sb, 31);
  __syncthreads();
  a = (warp ? pa : 0) + ia - a;
  b = (warp ? pb : 0) + ib - b;
}

// The last r in [0, n) with sums[r] <= x (sums ascending, sums[0] <= x); of
// equal sums the last, which is the request that is not empty.
__device__ __forceinline__ int find_last(const int *sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool ASSIGN>
__global__ void __launch_bounds__(kMaxThreads) attn_pages_kernel(const PagesParams p) {
  extern __shared__ int sm[];
  __shared__ int verdict;
  int *tok = sm, *pg = sm + p.B, *len = sm + 2 * p.B;  // first token, first page, length of each request
  const int ncta = gridDim.x, cta = blockIdx.x;
  const int threads = blockDim.x, gt = cta * threads + threadIdx.x, gn = ncta * threads;
  const int count = *p.free_count;
  const int64_t room = (int64_t)p.max_pages << p.shift;
  int bad = (count < 0 || count > p.free_capacity) ? ATTN_PAGES_BAD_COUNT : 0;
  if (p.after && *p.after) bad |= ATTN_PAGES_AFTER_REFUSAL;
  long long tokens = 0, pages = 0;
  for (int base = 0; base < p.B; base += threads) {
    const int r = base + threadIdx.x;
    long long a = 0, b = 0;
    if (r < p.B) {
      const int l = p.lens[r], g = p.arg[r];
      len[r] = l;
      if (ASSIGN) {
        if (l < 0 || g < 0 || (int64_t)l + g > room) {
          bad |= ATTN_PAGES_BAD_LENGTH;
        } else {
          a = g;
          b = (((int64_t)l + g + p.P - 1) >> p.shift) - (((int64_t)l + p.P - 1) >> p.shift);
        }
      } else {
        if (l < 0 || l > room)
          bad |= ATTN_PAGES_BAD_LENGTH;
        else if (g >= 0 && g < l)
          b = (((int64_t)l + p.P - 1) >> p.shift) - (((int64_t)g + p.P - 1) >> p.shift);
      }
    }
    long long ta, tb;
    block_scan(a, b, ta, tb);
    if (r < p.B) {
      // sums past the limits below are refused before they are used
      tok[r] = (int)min(tokens + a, (long long)0x7fffffff);
      pg[r] = (int)min(pages + b, (long long)0x7fffffff);
    }
    tokens += ta;
    pages += tb;
  }
  if (ASSIGN) {
    if (tokens > p.max_tokens) bad |= ATTN_PAGES_TOO_MANY_TOKENS;
    if (pages > count) bad |= ATTN_PAGES_NO_FREE_PAGES;
  } else if (count + pages > p.free_capacity) {
    bad |= ATTN_PAGES_NO_FREE_PAGES;
  }
  if (threadIdx.x == 0) verdict = 0;
  __syncthreads();
  if (bad) atomicOr(&verdict, bad);
  __syncthreads();
  bad = verdict;
  // every CTA has read the state that is updated below
  ptx::cluster_sync_all();
  const int total = bad ? 0 : (int)tokens, moved = bad ? 0 : (int)pages;

  for (int r = gt; r < p.B; r += gn) {
    const int l = len[r], g = p.arg[r];
    p.lens_out[r] = bad ? l : ASSIGN ? l + g : (g >= 0 && g < l ? g : l);
    if (ASSIGN) p.cu[r] = bad ? 0 : tok[r];
  }
  if (gt == 0) {
    *p.free_count_out = ASSIGN ? count - moved : count + moved;
    if (ASSIGN) p.cu[p.B] = total;
    p.info[0] = bad;
    p.info[1] = ASSIGN ? total : moved;
  }
  for (int64_t n = gt; n < moved; n += gn) {
    const int i = (int)n, r = find_last(pg, p.B, i);
    int *row = p.table + (int64_t)r * p.table_stride;
    if (ASSIGN) {
      const int have = (int)(((int64_t)len[r] + p.P - 1) >> p.shift);
      row[have + i - pg[r]] = p.free_pages[count - 1 - i];
    } else {
      const int keep = (int)(((int64_t)p.arg[r] + p.P - 1) >> p.shift);
      int *e = row + keep + i - pg[r];
      p.free_pages[count + i] = *e;
      *e = -1;
    }
  }
  if constexpr (ASSIGN) {
    // Four tokens a thread, so that their four page loads overlap: the first
    // one's request by a search, the others' from there; 16-byte stores where the
    // buffers allow them.
    const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
    for (int64_t i0 = (int64_t)gt * 4; i0 < p.max_tokens; i0 += (int64_t)gn * 4) {
      int slot[4], pos[4];
      int r = i0 < total ? find_last(tok, p.B, (int)i0) : 0;
      const int *from[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u;
        pos[u] = 0;
        from[u] = nullptr;
        if (i < total) {
          // usually the same request or the next one; past a run of idle ones by a search
          if (r + 1 < p.B && tok[r + 1] <= i) {
            ++r;
            if (r + 1 < p.B && tok[r + 1] <= i) r += find_last(tok + r, p.B - r, (int)i);
          }
          pos[u] = len[r] + (int)(i - tok[r]);
          const int j = pos[u] >> p.shift, have = (int)(((int64_t)len[r] + p.P - 1) >> p.shift);
          // a page of this step comes from the stack: its table entry may not be written yet
          from[u] = j < have ? p.table + (int64_t)r * p.table_stride + j
                             : p.free_pages + (count - 1 - (pg[r] + j - have));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) slot[u] = from[u] ? *from[u] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (from[u])  // -2: what the table or the stack holds has no 32-bit slot
          slot[u] = (unsigned)slot[u] > (0x7fffffffu >> p.shift) ? -2 : slot[u] * p.P + (pos[u] & (p.P - 1));
      if (wide && i0 + 4 <= p.max_tokens) {
        *reinterpret_cast<int4 *>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4 *>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i0 + u < p.max_tokens) {
            p.slots[i0 + u] = slot[u];
            p.positions[i0 + u] = pos[u];
          }
      }
    }
  }
}

template <bool ASSIGN>
int launch_pages(PagesParams &p, cudaStream_t st) {
  int device = 0, sms = 0;
  int *status = nullptr;
  const int rc = current_device(&device, &sms, &status);
  if (rc != ATTN_OK) return rc;
  const size_t smem = (size_t)p.B * 3 * sizeof(int);
  cudaError_t e;
  if (smem > 40 * 1024) {
    e = cudaFuncSetAttribute(attn_pages_kernel<ASSIGN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(ATTN_PAGES_MAX_REQUESTS * 3 * sizeof(int)));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  // one CTA of 256 threads for a decode step's few tokens, else CTAs of 1024,
  // one for each 2 Ki written entries, at most 8
  const int64_t entries = ASSIGN ? (int64_t)p.max_tokens + p.B : (int64_t)4 * p.B;
  const int threads = p.B <= 256 && entries <= 1024 ? 256 : kMaxThreads;
  int64_t n = entries / 2048;
  n = n < 1 ? 1 : n > 8 ? 8 : n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)n;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_pages_kernel<ASSIGN>, p);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_pages_assign(int *block_table, long long table_stride, int max_pages, const int *lens, const int *new_lens,
                      int B, int page_size, const int *free_pages, int free_capacity, const int *free_count,
                      int *lens_out, int *free_count_out, int *cu, int *slots, int *positions, int max_tokens,
                      int *info, attn_stream_t stream) {
  return attn_pages_assign_after(nullptr, block_table, table_stride, max_pages, lens, new_lens, B, page_size, free_pages,
                                 free_capacity, free_count, lens_out, free_count_out, cu, slots, positions, max_tokens,
                                 info, stream);
}

int attn_pages_assign_after(const int *after, int *block_table, long long table_stride, int max_pages, const int *lens,
                            const int *new_lens, int B, int page_size, const int *free_pages, int free_capacity,
                            const int *free_count, int *lens_out, int *free_count_out, int *cu, int *slots,
                            int *positions, int max_tokens, int *info, attn_stream_t stream) {
  using namespace attn;
  const int shift = kv4_page_shift(page_size);
  if (shift < 0 || B < 0 || B > ATTN_PAGES_MAX_REQUESTS || max_pages < 0 || free_capacity < 0 || max_tokens < 0)
    return ATTN_ERR_ARG;
  if (max_pages > (0x7fffffff >> shift) || table_stride < max_pages) return ATTN_ERR_ARG;
  if (!free_count || !free_count_out || !cu || !info) return ATTN_ERR_ARG;
  if (B > 0 && (!lens || !new_lens || !lens_out)) return ATTN_ERR_ARG;
  if (B > 0 && max_pages > 0 && !block_table) return ATTN_ERR_ARG;
  if (free_capacity > 0 && !free_pages) return ATTN_ERR_ARG;
  if (max_tokens > 0 && (!slots || !positions)) return ATTN_ERR_ARG;
  PagesParams p{};
  p.table = block_table; p.table_stride = table_stride; p.max_pages = max_pages; p.P = page_size; p.shift = shift;
  p.lens = lens; p.lens_out = lens_out; p.arg = new_lens; p.after = after;
  p.free_pages = const_cast<int *>(free_pages);  // only read by this kernel
  p.free_capacity = free_capacity; p.free_count = free_count; p.free_count_out = free_count_out;
  p.B = B; p.max_tokens = max_tokens;
  p.cu = cu; p.slots = slots; p.positions = positions; p.info = info;
  return launch_pages<true>(p, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_release(int *block_table, long long table_stride, int max_pages, const int *lens, const int *keep_lens,
                       int B, int page_size, int *free_pages, int free_capacity, const int *free_count, int *lens_out,
                       int *free_count_out, int *info, attn_stream_t stream) {
  using namespace attn;
  const int shift = kv4_page_shift(page_size);
  if (shift < 0 || B < 0 || B > ATTN_PAGES_MAX_REQUESTS || max_pages < 0 || free_capacity < 0) return ATTN_ERR_ARG;
  if (max_pages > (0x7fffffff >> shift) || table_stride < max_pages) return ATTN_ERR_ARG;
  if (!free_count || !free_count_out || !info) return ATTN_ERR_ARG;
  if (B > 0 && (!lens || !keep_lens || !lens_out)) return ATTN_ERR_ARG;
  if (B > 0 && max_pages > 0 && !block_table) return ATTN_ERR_ARG;
  if (free_capacity > 0 && !free_pages) return ATTN_ERR_ARG;
  PagesParams p{};
  p.table = block_table; p.table_stride = table_stride; p.max_pages = max_pages; p.P = page_size; p.shift = shift;
  p.lens = lens; p.lens_out = lens_out; p.arg = keep_lens;
  p.free_pages = free_pages; p.free_capacity = free_capacity; p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.B = B; p.info = info;
  return launch_pages<false>(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
