// Pages that several requests share: taken over, given back, made one's own before a
// write, moved, and their contents copied.
//
// shares[p] is the number of table rows that name page p beyond the first: 0 for a free
// page and for one with a single owner, so attn_pages_assign needs no change.
//
// fork:    row r becomes a copy of row parents[r] (as it was before the call), or
//          empty.  Every entry that a row loses counts its page down, every entry that
//          it gains counts it up (whole numbers: the order does not matter); a page
//          whose count ends at -1 has no row left.  Those are found by going over all
//          pages, so they come onto the stack once each and in the order of their ids.
// release: the same for the entries behind the kept tokens.
// own:     a row about to be written whose last page is partly filled and shared gets
//          a page from the stack, as if rows were served one after the other: with w
//          rows that write and s shares all w get one if w <= s, else all but the last.
// compact: with n pages of which c are free, used pages with ids >= n - c take the
//          places of the free ones below, both in the order of their ids.
//
// All but copy are one launch of one thread-block cluster (1 to 8 CTAs), its phases
// separated by cluster barriers; what one phase writes to global memory and the next
// reads is read past L1.  A call that cannot be served takes its counts back and
// changes nothing.  Latency bound: some six dependent passes through L2, with several
// entries of each thread in flight (one at a time: fork of 512 rows 28 us, compact of
// 65536 pages 40).  Measured (us; floor: the bytes at 6.80 TB/s, under 0.3 but where
// given): fork of 8 rows of up to 300 tokens 4.5, of 512 rows of up to 8192 15.6, own
// of 256 rows 5.3 (one CTA), compact of 1000 pages 10.4, of 65536 30, copy of 15700
// pages of 2 KB 12.5 (9.6: HBM).
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
constexpr int kMostCtas = 8;
constexpr int kHeld = 8;  // table entries that a thread holds between reading and writing them
constexpr int kUnchanged = -2;

struct SharedPagesParams {
  int *table, *table_out;
  int64_t table_stride, out_stride;
  int max_pages, P, shift;
  const int *lens;
  int *lens_out;
  const int *arg;  // parents, kept lengths or new lengths
  const int *after;  // own: info of a call that must not have been refused, or nullptr
  int *shares, *shares_out;
  int num_pages;
  int *free_pages, *free_out;
  int free_capacity;
  const int *free_count;
  int *free_count_out;
  int B, max_moves;
  int *src, *dst, *map, *info;
};

__device__ __forceinline__ int ld_dsmem(const int *local, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa_shared(ptx::smem_u32(local), rank)) : "memory");
  return v;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive sum of v over the block's threads; its total in `total`.
__device__ __forceinline__ int block_scan(int v, int &total) {
  __shared__ int sums[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int inc = warp_scan(v, lane);
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  const int s = warp_scan(lane < warps ? sums[lane] : 0, lane);
  const int before = __shfl_sync(0xffffffffu, s, (warp - 1) & 31);
  total = __shfl_sync(0xffffffffu, s, 31);
  __syncthreads();
  return (warp ? before : 0) + inc - v;
}

__device__ __forceinline__ void cluster_barrier() {
  if (gridDim.x == 1)
    __syncthreads();
  else
    ptx::cluster_sync_all();
}

// What the CTAs of the cluster tell each other: words that are zero at the start, each used by one exchange.
struct Exchange {
  int any[4];
  int sums[2];
};

// The OR of `bits` over the cluster, which all of it reaches.
__device__ __forceinline__ int cluster_or(int *word, int bits) {
  if (gridDim.x == 1) {
    if (!__syncthreads_or(bits)) return 0;
    if (bits) atomicOr(word, bits);
    __syncthreads();
    return *word;
  }
  if (bits) atomicOr(word, bits);
  ptx::cluster_sync_all();
  int all = 0;
  for (int c = 0; c < (int)gridDim.x; ++c) all |= ld_dsmem(word, c);
  return all;
}

// Sums of (a, b) over the CTAs before this one, and over all, from each CTA's.
__device__ __forceinline__ void cluster_sums(int *mine, int a, int b, int2 &before, int2 &all) {
  before = make_int2(0, 0);
  all = make_int2(a, b);
  if (gridDim.x == 1) return;
  if (threadIdx.x == 0) {
    mine[0] = a;
    mine[1] = b;
  }
  ptx::cluster_sync_all();
  all = make_int2(0, 0);
  for (int c = 0; c < (int)gridDim.x; ++c) {
    const int x = ld_dsmem(&mine[0], c), y = ld_dsmem(&mine[1], c);
    if (c < (int)blockIdx.x) before.x += x, before.y += y;
    all.x += x;
    all.y += y;
  }
}

// load(i), then use(i, what it gave), for i = first, first + step, ... below last: U of them in flight.
template <int U, typename L, typename F>
__device__ __forceinline__ void in_flight(int64_t first, int64_t last, int64_t step, L &&load, F &&use) {
  for (int64_t i0 = first; i0 < last; i0 += step * U) {
    decltype(load(0)) v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * step < last) v[u] = load((int)(i0 + u * step));
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * step < last) use((int)(i0 + u * step), v[u]);
  }
}

__device__ __forceinline__ int pages_of(int len, int P, int shift) { return (int)(((int64_t)len + P - 1) >> shift); }

constexpr int kChunk = 256;  // columns of a row that a warp goes over at a time

// Counts the changed rows' entries: lost ones by -sign, gained ones by +sign.
// Returns ATTN_PAGES_BAD_PAGE where an entry is no page (it is not counted).
template <bool FORK>
__device__ __forceinline__ int count_entries(const SharedPagesParams &p, const int *len, const int *arg, int columns, int sign) {
  constexpr int U = kChunk / 32;
  const int lane = threadIdx.x & 31, warps = (gridDim.x * blockDim.x) >> 5;
  const int chunks = (columns + kChunk - 1) / kChunk;
  const int64_t tasks = (int64_t)p.B * chunks;
  int bad = 0;
  for (int64_t task = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; task < tasks; task += warps) {
    const int r = (int)(task / chunks), start = (int)(task % chunks) * kChunk, c0 = start + lane;
    if (arg[r] == kUnchanged) continue;
    const int had = pages_of(len[r], p.P, p.shift);
    const int *row = p.table + (int64_t)r * p.table_stride;
    const int first = FORK ? 0 : pages_of(arg[r], p.P, p.shift);
    const int has = FORK && arg[r] >= 0 ? pages_of(len[arg[r]], p.P, p.shift) : 0;
    const int *from = FORK && arg[r] >= 0 ? p.table + (int64_t)arg[r] * p.table_stride : row;
    if (start >= had && start >= has) continue;
    int lost[U], got[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + 32 * i;
      lost[i] = c >= first && c < had ? row[c] : 0;
      got[i] = FORK && c < has ? from[c] : 0;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + 32 * i;
      const bool loses = c >= first && c < had, gains = FORK && c < has;
      const bool lost_ok = (unsigned)lost[i] < (unsigned)p.num_pages, got_ok = (unsigned)got[i] < (unsigned)p.num_pages;
      if ((loses && !lost_ok) || (gains && !got_ok)) bad = ATTN_PAGES_BAD_PAGE;
      if (loses && gains && lost[i] == got[i]) continue;  // a page that both rows name
      if (loses && lost_ok) atomicAdd(p.shares + lost[i], -sign);
      if (gains && got_ok) atomicAdd(p.shares + got[i], sign);
    }
  }
  return bad;
}

template <bool FORK>
__global__ void __launch_bounds__(kMaxThreads) attn_pages_fork_kernel(const SharedPagesParams p) {
  extern __shared__ int sm[];
  __shared__ Exchange ex;
  __shared__ int widest, chained;
  int *len = sm, *arg = sm + p.B;
  const int threads = blockDim.x, gt = blockIdx.x * threads + threadIdx.x, gn = gridDim.x * threads;
  const int count = *p.free_count;
  const int64_t room = (int64_t)p.max_pages << p.shift;
  int bad = count < 0 || count > p.free_capacity ? ATTN_PAGES_BAD_COUNT : 0;
  if (threadIdx.x < 4) ex.any[threadIdx.x] = 0;
  if (threadIdx.x == 0) widest = chained = 0;
  in_flight<2>(
      threadIdx.x, p.B, threads, [&](int r) { return make_int2(p.lens[r], p.arg[r]); },
      [&](int r, int2 v) {
        const int l = v.x, a = v.y;
        len[r] = l;
        if (l < 0 || l > room) bad |= ATTN_PAGES_BAD_LENGTH;
        if (FORK) {
          if (a < -1 || a >= p.B) bad |= ATTN_PAGES_BAD_LENGTH;
          arg[r] = a == r ? kUnchanged : a;
        } else {
          arg[r] = a >= 0 && a < l ? a : kUnchanged;
        }
      });
  __syncthreads();
  bad = cluster_or(&ex.any[0], bad);
  if (!bad) {
    // columns that any changed row has, before or after; whether a row is taken over that changes itself
    int most = 0, chain = 0;
    for (int r = threadIdx.x; r < p.B; r += threads) {
      if (arg[r] == kUnchanged) continue;
      most = max(most, pages_of(len[r], p.P, p.shift));
      if (FORK && arg[r] >= 0) {
        most = max(most, pages_of(len[arg[r]], p.P, p.shift));
        chain |= arg[arg[r]] != kUnchanged;
      }
    }
    if (most) atomicMax(&widest, most);
    if (chain) chained = 1;
    __syncthreads();
  }
  const int columns = widest;
  int freed = 0;
  // a CTA's pages: a multiple of 4, so that threads take four each
  const int per = ((p.num_pages + (int)gridDim.x * 4 - 1) / ((int)gridDim.x * 4)) * 4;
  const int first_page = (int)min((int64_t)blockIdx.x * per, (int64_t)p.num_pages);
  const int last_page = (int)min((int64_t)first_page + per, (int64_t)p.num_pages);
  if (!bad && columns > 0) {
    bad = cluster_or(&ex.any[1], count_entries<FORK>(p, len, arg, columns, 1));
    if (gridDim.x == 1) __syncthreads();
    // pages without a row
    int mine = 0, odd = 0;
    in_flight<8>(
        first_page + threadIdx.x, last_page, threads, [&](int i) { return __ldcg(p.shares + i); },
        [&](int, int s) {
          mine += s == -1;
          if (s < -1) odd = ATTN_PAGES_BAD_SHARES;
        });
    int total;
    int2 before, all;
    block_scan(mine, total);
    cluster_sums(ex.sums, total, 0, before, all);
    freed = all.x;
    odd = cluster_or(&ex.any[2], odd | ((int64_t)count + freed > p.free_capacity ? ATTN_PAGES_NO_FREE_PAGES : 0));
    if (!bad) bad = odd;
    if (bad) {
      count_entries<FORK>(p, len, arg, columns, -1);
    } else {
      int at = count + before.x;
      for (int base = first_page; base < last_page && total > 0; base += threads * 4) {
        int gone[4], n = 0;
        const int i0 = base + threadIdx.x * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          gone[k] = i0 + k < last_page && __ldcg(p.shares + i0 + k) == -1;
          n += gone[k];
        }
        int here;
        int to = at + block_scan(n, here);
        at += here;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (gone[k]) {
            p.free_pages[to++] = i0 + k;
            p.shares[i0 + k] = 0;
          }
      }
      if (FORK && chained) {
        // in place, some columns at a time: all of their entries are read before one is written
        const int wide = max(1, min(columns, gn * kHeld / p.B));
        for (int c0 = 0; c0 < columns; c0 += wide) {
          const int w = min(wide, columns - c0);
          int held[kHeld];
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            held[k] = kUnchanged;
            const int e = gt + k * gn, r = e / w, c = c0 + e % w;
            if (r >= p.B || arg[r] == kUnchanged) continue;
            if (arg[r] >= 0 && c < pages_of(len[arg[r]], p.P, p.shift))
              held[k] = p.table[(int64_t)arg[r] * p.table_stride + c];
            else if (c < pages_of(len[r], p.P, p.shift))
              held[k] = -1;
          }
          cluster_barrier();
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            const int e = gt + k * gn, r = e / w, c = c0 + e % w;
            if (held[k] != kUnchanged) p.table[(int64_t)r * p.table_stride + c] = held[k];
          }
        }
      } else {
        // no row that changes is read: row by row
        constexpr int U = kChunk / 32;
        const int lane = threadIdx.x & 31, chunks = (columns + kChunk - 1) / kChunk;
        const int64_t tasks = (int64_t)p.B * chunks;
        for (int64_t task = gt >> 5; task < tasks; task += gn >> 5) {
          const int r = (int)(task / chunks), c0 = (int)(task % chunks) * kChunk + lane;
          if (arg[r] == kUnchanged) continue;
          const int had = pages_of(len[r], p.P, p.shift);
          const int kept = !FORK ? pages_of(arg[r], p.P, p.shift) : arg[r] < 0 ? 0 : pages_of(len[arg[r]], p.P, p.shift);
          int *row = p.table + (int64_t)r * p.table_stride;
          const int *from = FORK && arg[r] >= 0 ? p.table + (int64_t)arg[r] * p.table_stride : row;
          int v[U];
#pragma unroll
          for (int i = 0; i < U; ++i) v[i] = FORK && c0 + 32 * i < kept ? from[c0 + 32 * i] : -1;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int c = c0 + 32 * i;
            if (c < kept ? FORK : c < had) row[c] = v[i];
          }
        }
      }
    }
  }
  for (int r = gt; r < p.B; r += gn) {
    const int a = arg[r];
    p.lens_out[r] = bad || a == kUnchanged ? len[r] : !FORK ? a : a < 0 ? 0 : len[a];
  }
  if (gt == 0) {
    *p.free_count_out = bad ? count : count + freed;
    p.info[0] = bad;
    p.info[1] = bad ? 0 : freed;
  }
  if (gridDim.x > 1) ptx::cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// One CTA: each row is one entry.
__global__ void __launch_bounds__(kMaxThreads) attn_pages_own_kernel(const SharedPagesParams p) {
  extern __shared__ int page[];  // the page that each row is about to write into and shares, or kUnchanged
  __shared__ int word;
  const int threads = blockDim.x;
  const int count = *p.free_count;
  const int64_t room = (int64_t)p.max_pages << p.shift;
  auto all = [&](int bits) {
    __syncthreads();
    if (threadIdx.x == 0) word = 0;
    __syncthreads();
    if (bits) atomicOr(&word, bits);
    __syncthreads();
    return word;
  };
  int bad = count < 0 || count > p.free_capacity ? ATTN_PAGES_BAD_COUNT : 0;
  if (p.after && *p.after) bad |= ATTN_PAGES_AFTER_REFUSAL;
  for (int r = threadIdx.x; r < p.B; r += threads) {
    const int l = p.lens[r], n = p.arg[r];
    page[r] = kUnchanged;
    if (l < 0 || n < 0 || l > room) {
      bad |= ATTN_PAGES_BAD_LENGTH;
    } else if (n > 0 && (l & (p.P - 1))) {
      const int pg = p.table[(int64_t)r * p.table_stride + (l >> p.shift)];
      if ((unsigned)pg >= (unsigned)p.num_pages)
        bad |= ATTN_PAGES_BAD_PAGE;
      else
        page[r] = pg;
    }
  }
  bad = all(bad);
  int moved = 0;
  if (!bad) {
    for (int r = threadIdx.x; r < p.B; r += threads)
      if (page[r] >= 0) atomicAdd(p.shares + page[r], -1);
    __syncthreads();
    // shares - writers: below 0 where every row that names the page writes
    int odd = 0;
    uint32_t contested = 0;  // of the thread's rows (16 at most)
    int k = 0;
    for (int r = threadIdx.x; r < p.B; r += threads, ++k)
      if (page[r] >= 0) {
        const int s = __ldcg(p.shares + page[r]);
        if (s < -1) odd = ATTN_PAGES_BAD_SHARES;
        if (s < 0) contested |= 1u << k;
      }
    bad = all(odd);
    if (bad) {
      for (int r = threadIdx.x; r < p.B; r += threads)
        if (page[r] >= 0) atomicAdd(p.shares + page[r], 1);
    } else {
      // the last of them keeps the page: the smallest of -2 - r
      k = 0;
      for (int r = threadIdx.x; r < p.B; r += threads, ++k)
        if (contested >> k & 1) atomicMin(p.shares + page[r], -2 - r);
      __syncthreads();
      uint32_t keeps = 0;
      k = 0;
      for (int r = threadIdx.x; r < p.B; r += threads, ++k)
        if ((contested >> k & 1) && __ldcg(p.shares + page[r]) == -2 - r) keeps |= 1u << k;
      __syncthreads();
      k = 0;
      for (int r = threadIdx.x; r < p.B; r += threads, ++k)
        if (keeps >> k & 1) p.shares[page[r]] = -1;
      __syncthreads();
      int total = 0;
      for (int base = 0, j = 0; base < p.B; base += threads, ++j) {
        const int r = base + threadIdx.x;
        int here;
        block_scan(r < p.B && page[r] >= 0 && !(keeps >> j & 1), here);
        total += here;
      }
      int wrong = total > count ? ATTN_PAGES_NO_FREE_PAGES : 0;
      if (!wrong)
        for (int i = threadIdx.x; i < total; i += threads)
          if ((unsigned)p.free_pages[count - 1 - i] >= (unsigned)p.num_pages) wrong = ATTN_PAGES_BAD_PAGE;
      bad = all(wrong);
      if (bad) {
        for (int r = threadIdx.x; r < p.B; r += threads)
          if (page[r] >= 0) atomicAdd(p.shares + page[r], 1);
      } else {
        int before = 0;
        for (int base = 0, j = 0; base < p.B; base += threads, ++j) {
          const int r = base + threadIdx.x;
          const bool moves = r < p.B && page[r] >= 0 && !(keeps >> j & 1);
          int here;
          const int i = before + block_scan(moves, here);
          before += here;
          if (r >= p.B) continue;
          int to = -1;
          if (moves) {
            to = p.free_pages[count - 1 - i];
            p.table[(int64_t)r * p.table_stride + (p.lens[r] >> p.shift)] = to;
            p.shares[to] = 0;
          } else if (keeps >> j & 1) {
            p.shares[page[r]] = 0;
          }
          p.src[r] = moves ? page[r] : -1;
          p.dst[r] = to;
        }
        moved = total;
      }
    }
  }
  if (bad)
    for (int r = threadIdx.x; r < p.B; r += threads) p.src[r] = p.dst[r] = -1;
  if (threadIdx.x == 0) {
    *p.free_count_out = count - moved;
    p.info[0] = bad;
    p.info[1] = moved;
  }
}

__global__ void __launch_bounds__(kMaxThreads) attn_pages_compact_kernel(const SharedPagesParams p) {
  __shared__ Exchange ex;
  const int lane = threadIdx.x & 31, threads = blockDim.x, gt = blockIdx.x * threads + threadIdx.x, gn = gridDim.x * threads;
  const int count = *p.free_count, n = p.num_pages, end = n - count;
  const int64_t room = (int64_t)p.max_pages << p.shift;
  int bad = count < 0 || count > p.free_capacity || count > n ? ATTN_PAGES_BAD_COUNT : 0;
  if (threadIdx.x < 4) ex.any[threadIdx.x] = 0;
  for (int r = gt; r < p.B; r += gn)
    if (p.lens[r] < 0 || p.lens[r] > room) bad |= ATTN_PAGES_BAD_LENGTH;
  for (int i = gt; i < n; i += gn) p.map[i] = i;
  __syncthreads();
  bad = cluster_or(&ex.any[0], bad);
  if (!bad) {
    int odd = 0;
    in_flight<4>(
        gt, count, gn, [&](int i) { return p.free_pages[i]; },
        [&](int, int e) {
          if ((unsigned)e >= (unsigned)n || atomicExch(p.map + e, -1) == -1) odd = ATTN_PAGES_BAD_PAGE;  // no page, or twice
        });
    bad = cluster_or(&ex.any[1], odd);
    if (gridDim.x == 1) __syncthreads();
  }
  const int per = ((n + (int)gridDim.x * 4 - 1) / ((int)gridDim.x * 4)) * 4;
  const int first_page = (int)min((int64_t)blockIdx.x * per, (int64_t)n);
  const int last_page = (int)min((int64_t)first_page + per, (int64_t)n);
  const int chunks = (p.max_pages + kChunk - 1) / kChunk;
  const int64_t tasks = (int64_t)p.B * chunks;
  constexpr int U = kChunk / 32;
  int moved = 0;
  if (!bad) {
    int moves = 0, holes = 0, odd = 0;
    in_flight<8>(
        first_page + threadIdx.x, last_page, threads, [&](int i) { return __ldcg(p.map + i); },
        [&](int i, int to) {
          moves += to >= 0 && i >= end;
          holes += to < 0 && i < end;
        });
    for (int64_t task = gt >> 5; task < tasks; task += gn >> 5) {
      const int r = (int)(task / chunks), start = (int)(task % chunks) * kChunk, had = pages_of(p.lens[r], p.P, p.shift);
      if (start >= had) continue;
      int e[U], to[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = start + lane + 32 * i;
        e[i] = c < had ? p.table[(int64_t)r * p.table_stride + c] : kUnchanged;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) to[i] = (unsigned)e[i] < (unsigned)n ? __ldcg(p.map + e[i]) : -1;
#pragma unroll
      for (int i = 0; i < U; ++i)  // no page, or a free one
        if (start + lane + 32 * i < had && to[i] < 0) odd = ATTN_PAGES_BAD_PAGE;
    }
    int total_moves, total_holes;
    int2 before, all;
    block_scan(moves, total_moves);
    block_scan(holes, total_holes);
    cluster_sums(ex.sums, total_moves, total_holes, before, all);
    moved = all.x;
    bad = cluster_or(&ex.any[2], odd | (moved > p.max_moves ? ATTN_PAGES_TOO_MANY_MOVES : 0));
    if (!bad) {
      int move_at = before.x, hole_at = before.y;
      for (int base = first_page; base < last_page; base += threads * 4) {
        const int i0 = base + threadIdx.x * 4;
        int to[4], a = 0, b = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = i0 + k < last_page ? __ldcg(p.map + i0 + k) : 0;
        bool is_move[4], is_hole[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k;
          is_move[k] = i < last_page && to[k] >= 0 && i >= end;
          is_hole[k] = i < last_page && to[k] < 0 && i < end;
          a += is_move[k];
          b += is_hole[k];
        }
        int ta, tb;
        int x = move_at + block_scan(a, ta), y = hole_at + block_scan(b, tb);
        move_at += ta;
        hole_at += tb;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (is_move[k]) p.src[x++] = i0 + k;
          if (is_hole[k]) p.dst[y++] = i0 + k;
        }
      }
    }
  }
  const int from = bad ? 0 : moved;
  for (int i = from + gt; i < p.max_moves; i += gn) p.src[i] = p.dst[i] = -1;
  cluster_barrier();
  if (!bad) {
    in_flight<4>(
        gt, moved, gn, [&](int i) { return make_int2(__ldcg(p.src + i), __ldcg(p.dst + i)); }, [&](int, int2 m) { p.map[m.x] = m.y; });
    cluster_barrier();
  }
  in_flight<8>(
      gt, n, gn, [&](int i) { return make_int2(__ldcg(p.map + i), p.shares[i]); },
      [&](int i, int2 v) {
        const int to = bad ? i : v.x;
        if (to == i) {
          if (p.shares_out != p.shares) p.shares_out[i] = v.y;
        } else if (to >= 0) {
          p.shares_out[to] = v.y;
          p.shares_out[i] = 0;
        } else if (i >= end) {
          p.shares_out[i] = 0;  // (a free page below `end` gets its count from the page that moves there)
        }
        if (bad) p.map[i] = i;
      });
  const bool other_stack = p.free_out != p.free_pages;
  in_flight<4>(
      gt, p.free_capacity, gn, [&](int i) { return other_stack && (bad || i >= count) ? p.free_pages[i] : n - 1 - i; },
      [&](int i, int v) {
        if (other_stack || (!bad && i < count)) p.free_out[i] = v;
      });
  const bool other = p.table_out != p.table;
  for (int64_t task = gt >> 5; task < tasks; task += gn >> 5) {
    const int r = (int)(task / chunks), start = (int)(task % chunks) * kChunk;
    const int had = bad ? 0 : pages_of(p.lens[r], p.P, p.shift);
    if (start >= had && !other) continue;
    int e[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = start + lane + 32 * i;
      e[i] = c < (other ? p.max_pages : had) ? p.table[(int64_t)r * p.table_stride + c] : 0;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (start + lane + 32 * i < had) e[i] = __ldcg(p.map + e[i]);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = start + lane + 32 * i;
      if (c < (other ? p.max_pages : had)) p.table_out[(int64_t)r * p.out_stride + c] = e[i];
    }
  }
  if (gt == 0) {
    p.info[0] = bad;
    p.info[1] = bad ? 0 : moved;
  }
  if (gridDim.x > 1) ptx::cluster_sync_all();
}

// ---------------------------------------------------------------- contents

struct CopyParams {
  uint8_t *cache;
  int64_t page_bytes, layer_stride;
  int layers, num_pages, n;
  const int *src, *dst;
  int parts, part_bytes;  // a page in parts of at most 2 KB, a warp each
  int *status;
};

constexpr int kCopyThreads = 256;

// Four 16-byte words a lane in flight; a warp's parts lie a grid apart, so that the
// pages of neighbouring entries are copied at the same time.
__global__ void __launch_bounds__(kCopyThreads) attn_pages_copy_kernel(const CopyParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32), all = (int64_t)p.n * p.layers * p.parts;
  for (int64_t w = ((int64_t)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; w < all; w += warps) {
    const int64_t e = w / p.parts;
    const int part = (int)(w - e * p.parts), i = (int)(e / p.layers), layer = (int)(e - (int64_t)i * p.layers);
    const int s = p.src[i], d = p.dst[i];
    if (s == -1) continue;
    if ((unsigned)s >= (unsigned)p.num_pages || (unsigned)d >= (unsigned)p.num_pages) {
      if (lane == 0) atomicCAS(p.status, 0, kStatusDevice);
      continue;
    }
    uint8_t *base = p.cache + layer * p.layer_stride;
    const int64_t off = (int64_t)part * p.part_bytes;
    const int words = (int)(min((int64_t)p.part_bytes, p.page_bytes - off) / 16);
    const uint4 *from = reinterpret_cast<const uint4 *>(base + s * p.page_bytes + off);
    uint4 *to = reinterpret_cast<uint4 *>(base + d * p.page_bytes + off);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (lane + 32 * k < words) v[k] = from[lane + 32 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (lane + 32 * k < words) to[lane + 32 * k] = v[k];
  }
}

// ---------------------------------------------------------------- launches

// One CTA of 256 threads for a few rows and pages, else CTAs of 1024: one for each
// 32 pieces of rows (a warp each) or 4 Ki pages, at most 8.  256 threads / 1, 2, 4, 8 CTAs of 1024, us: fork of 8 rows
// 4.6 / 5.3, 7.7, 7.9, 8.9, of 256 rows of up to 512 tokens 42 / 19.7, 15.9, 12.6, 11.8, of 512 rows of up to 8192
// 146 / 61, 36, 22, 15.6; compact of 1000 pages 10.1 / 10.5, 13.8, 13.9, 14.9, of 65536 321 / 142, 82, 46, 30.
template <typename K>
int launch_cluster(K kernel, const SharedPagesParams &p, size_t smem, cudaStream_t st) {
  int device = 0, sms = 0;
  int *status = nullptr;
  const int rc = current_device(&device, &sms, &status);
  if (rc != ATTN_OK) return rc;
  cudaError_t e;
  if (smem > 40 * 1024) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(ATTN_PAGES_MAX_REQUESTS * 2 * sizeof(int)));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  const int64_t pieces = (int64_t)p.B * ((p.max_pages + kChunk - 1) / kChunk);
  const int threads = pieces <= 8 && p.num_pages <= 2048 ? 256 : kMaxThreads;
  int64_t n = (pieces + kMaxWarps - 1) / kMaxWarps;
  if (n < p.num_pages / 4096) n = p.num_pages / 4096;
  n = n < 1 ? 1 : n > kMostCtas ? kMostCtas : n;
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
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

// The checks that all calls on a page state share.
int check_state(const int *table, long long stride, int max_pages, const int *lens, int B, int P, const int *shares,
                int num_pages, const int *free_pages, int capacity, const int *count, const int *info) {
  const int shift = kv4_page_shift(P);
  if (shift < 0 || B < 0 || B > ATTN_PAGES_MAX_REQUESTS || max_pages < 0 || capacity < 0 || num_pages < 0)
    return ATTN_ERR_ARG;
  if (max_pages > (0x7fffffff >> shift) || stride < max_pages) return ATTN_ERR_ARG;
  if (num_pages > 0x7fffffff - 65536 || capacity > 0x7fffffff - 65536) return ATTN_ERR_ARG;  // threads are numbered past them
  if (!count || !info || (num_pages > 0 && !shares) || (capacity > 0 && !free_pages)) return ATTN_ERR_ARG;
  if (B > 0 && (!lens || (max_pages > 0 && !table))) return ATTN_ERR_ARG;
  return ATTN_OK;
}

int change_rows(bool fork, int *table, long long stride, int max_pages, const int *lens, const int *arg, int B, int P, int *shares,
                int num_pages, int *free_pages, int capacity, const int *count, int *lens_out, int *count_out, int *info,
                cudaStream_t st) {
  const int rc = check_state(table, stride, max_pages, lens, B, P, shares, num_pages, free_pages, capacity, count, info);
  if (rc != ATTN_OK) return rc;
  if (!count_out || (B > 0 && (!arg || !lens_out))) return ATTN_ERR_ARG;
  SharedPagesParams p{};
  p.table = table; p.table_stride = stride; p.max_pages = max_pages; p.P = P; p.shift = kv4_page_shift(P);
  p.lens = lens; p.lens_out = lens_out; p.arg = arg;
  p.shares = shares; p.num_pages = num_pages;
  p.free_pages = free_pages; p.free_capacity = capacity; p.free_count = count; p.free_count_out = count_out;
  p.B = B; p.info = info;
  const size_t smem = (size_t)B * 2 * sizeof(int);
  return fork ? launch_cluster(attn_pages_fork_kernel<true>, p, smem, st)
              : launch_cluster(attn_pages_fork_kernel<false>, p, smem, st);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_pages_fork(int *block_table, long long table_stride, int max_pages, const int *lens, const int *parents, int B,
                    int page_size, int *shares, int num_pages, int *free_pages, int free_capacity, const int *free_count,
                    int *lens_out, int *free_count_out, int *info, attn_stream_t stream) {
  return attn::change_rows(true, block_table, table_stride, max_pages, lens, parents, B, page_size, shares, num_pages,
                           free_pages, free_capacity, free_count, lens_out, free_count_out, info,
                           reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_release_shared(int *block_table, long long table_stride, int max_pages, const int *lens,
                              const int *keep_lens, int B, int page_size, int *shares, int num_pages, int *free_pages,
                              int free_capacity, const int *free_count, int *lens_out, int *free_count_out, int *info,
                              attn_stream_t stream) {
  return attn::change_rows(false, block_table, table_stride, max_pages, lens, keep_lens, B, page_size, shares, num_pages,
                           free_pages, free_capacity, free_count, lens_out, free_count_out, info,
                           reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_own(int *block_table, long long table_stride, int max_pages, const int *lens, const int *new_lens, int B,
                   int page_size, int *shares, int num_pages, const int *free_pages, int free_capacity,
                   const int *free_count, int *free_count_out, int *src, int *dst, int *info, attn_stream_t stream) {
  return attn_pages_own_after(nullptr, block_table, table_stride, max_pages, lens, new_lens, B, page_size, shares, num_pages,
                              free_pages, free_capacity, free_count, free_count_out, src, dst, info, stream);
}

int attn_pages_own_after(const int *after, int *block_table, long long table_stride, int max_pages, const int *lens,
                         const int *new_lens, int B, int page_size, int *shares, int num_pages, const int *free_pages,
                         int free_capacity, const int *free_count, int *free_count_out, int *src, int *dst, int *info,
                         attn_stream_t stream) {
  using namespace attn;
  int rc = check_state(block_table, table_stride, max_pages, lens, B, page_size, shares, num_pages, free_pages, free_capacity,
                       free_count, info);
  if (rc != ATTN_OK) return rc;
  if (!free_count_out || (B > 0 && (!new_lens || !src || !dst))) return ATTN_ERR_ARG;
  SharedPagesParams p{};
  p.table = block_table; p.table_stride = table_stride; p.max_pages = max_pages; p.P = page_size;
  p.shift = kv4_page_shift(page_size);
  p.lens = lens; p.arg = new_lens; p.after = after;
  p.shares = shares; p.num_pages = num_pages;
  p.free_pages = const_cast<int *>(free_pages);  // only read by this kernel
  p.free_capacity = free_capacity; p.free_count = free_count; p.free_count_out = free_count_out;
  p.B = B; p.src = src; p.dst = dst; p.info = info;
  int device = 0, sms = 0;
  int *status = nullptr;
  if ((rc = current_device(&device, &sms, &status)) != ATTN_OK) return rc;
  const size_t smem = (size_t)B * sizeof(int);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(attn_pages_own_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(ATTN_PAGES_MAX_REQUESTS * sizeof(int)));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  // 1024 threads for more than 256 rows: then a thread has 16 at most.  256 / 1024 threads, us: 8 rows 3.1 / 4.1, 32 4.4 /
  // 5.5, 256 5.0 / 6.0.
  attn_pages_own_kernel<<<1, B <= 256 ? 256 : kMaxThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

int attn_pages_compact(const int *block_table, long long table_stride, int *table_out, long long table_out_stride,
                       int max_pages, const int *lens, int B, int page_size, const int *shares, int *shares_out,
                       int num_pages, const int *free_pages, int *free_pages_out, int free_capacity,
                       const int *free_count, int *src, int *dst, int max_moves, int *map, int *info,
                       attn_stream_t stream) {
  using namespace attn;
  const int rc = check_state(block_table, table_stride, max_pages, lens, B, page_size, shares, num_pages, free_pages,
                             free_capacity, free_count, info);
  if (rc != ATTN_OK) return rc;
  if (max_moves < 0 || max_moves > 0x7fffffff - 65536 || table_out_stride < max_pages) return ATTN_ERR_ARG;
  if ((num_pages > 0 && (!shares_out || !map)) || (free_capacity > 0 && !free_pages_out) || (max_moves > 0 && (!src || !dst)))
    return ATTN_ERR_ARG;
  if (B > 0 && max_pages > 0 && !table_out) return ATTN_ERR_ARG;
  if (table_out == block_table && table_out_stride != table_stride) return ATTN_ERR_ARG;
  SharedPagesParams p{};
  // (what is const is written only where it is also the output)
  p.table = const_cast<int *>(block_table); p.table_stride = table_stride; p.table_out = table_out;
  p.out_stride = table_out_stride; p.max_pages = max_pages; p.P = page_size; p.shift = kv4_page_shift(page_size);
  p.lens = lens;
  p.shares = const_cast<int *>(shares); p.shares_out = shares_out; p.num_pages = num_pages;
  p.free_pages = const_cast<int *>(free_pages); p.free_out = free_pages_out; p.free_capacity = free_capacity;
  p.free_count = free_count;
  p.B = B; p.max_moves = max_moves; p.src = src; p.dst = dst; p.map = map; p.info = info;
  return launch_cluster(attn_pages_compact_kernel, p, 0, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_copy(void *cache, long long page_bytes, int num_pages, int layers, long long layer_stride, const int *src,
                    const int *dst, int n, attn_stream_t stream) {
  using namespace attn;
  if (page_bytes < 0 || num_pages < 0 || layers < 0 || layer_stride < 0 || n < 0) return ATTN_ERR_ARG;
  if (page_bytes > ((long long)1 << 40) || layer_stride > ((long long)1 << 44)) return ATTN_ERR_ARG;
  if (n == 0 || layers == 0 || page_bytes == 0) return ATTN_OK;
  const long long parts = (page_bytes + 2047) / 2048;
  if (parts > 0x7fffffff || (long long)n * layers > ((long long)1 << 62) / parts) return ATTN_ERR_ARG;
  if (!src || !dst || (num_pages > 0 && !cache)) return ATTN_ERR_ARG;
  if (page_bytes % 16 || layer_stride % 16 || (reinterpret_cast<uintptr_t>(cache) & 15u)) return ATTN_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3u) return ATTN_ERR_ALIGN;
  int device = 0, sms = 0;
  CopyParams p{};
  const int rc = current_device(&device, &sms, &p.status);
  if (rc != ATTN_OK) return rc;
  p.cache = static_cast<uint8_t *>(cache);
  p.page_bytes = page_bytes; p.layer_stride = layer_stride; p.layers = layers; p.num_pages = num_pages; p.n = n;
  p.src = src; p.dst = dst;
  p.parts = (int)parts;
  p.part_bytes = (int)((page_bytes / 16 + parts - 1) / parts * 16);
  const int64_t ctas = ((int64_t)n * layers * parts + kCopyThreads / 32 - 1) / (kCopyThreads / 32), most = 8 * (int64_t)sms;
  attn_pages_copy_kernel<<<(unsigned)(ctas < most ? ctas : most), kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // extern "C"
