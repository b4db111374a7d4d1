// Attention over the 4-bit paged cache: O = softmax(scale Q K^T) V and its LSE
// for requests of any length with a few query tokens each (decoding, drafted
// tokens), K and V read from the pages as they are held.
//
// With K_jd = s_jg c_jd + m_jg (g the group of 64 dims that d is in),
//     S_j = scale * sum_g ( s_jg (q_g . c_jg) + m_jg sum(q_g) ),
//     O   = sum_j p_j V_j = sum_j (p_j s'_jg) c'_jd + sum_j p_j m'_jg,
// so the products run on the codes, and scales and minima join per token and
// group, not per value.
//
// Codes as half precision without arithmetic.  A nibble in bits 0-3 (4-7) of
// a 16-bit word, all other bits zero, is the half-precision subnormal
// c * 2^-24 (c * 2^-20); the tensor cores take subnormals exactly.  So four
// ANDs and one shift turn a word of eight codes into four operand registers;
// the factors 2^24 and 1/16 are folded into Q (whose rows are scaled by a power
// of two so that half precision holds bfloat16's 8 bits down to 2^-25 of the
// row's largest value) and, for V, into the output.
//
// Products (mma m16n8k16): K and V codes are the 16-row operand, the query
// rows (query token x head of the kv head's group) are the 8 columns, so that
// a decode step's 4 or 8 rows leave nothing or half of the tile unused:
// S^T[token, row] = K Q^T and O^T[dim, row] = V^T P^T.  P^T is S^T's
// accumulator transposed through movmatrix.  ldmatrix hands every lane the
// word of K's row that it multiplies, and, transposed as 16-bit elements (four
// codes of one token), V's words with two tokens side by side, which is how
// the second product wants them.  The order of the dims in a product is free.
//
// Softmax.  p = 2^(y - ref), ref a per-row reference 10 above which the warp
// rescales only when some y exceeds ref + 15; P s' is rounded to half
// precision (2^-11 relative; bfloat16's 2^-8 would be as large as the output's own
// rounding) times a power of two per group that brings the largest scale s' seen
// below 1.  That keeps the products' roundings below 2^-28 of their sum while
// scales lie within 2^6 of each other.  A warp that meets others (a token of huge
// V which some rows do not see, or give no weight, would take the bits of the
// rest) begins its item again in a second form of the loop, with a power of two
// for each row and group that goes by the products the row really has: up to
// twice the time (64 requests of 1 to 8192 tokens: 50 us; 58 with one such token a
// request, 77 with one in a hundred).  Taking that form always cost 3 to 5 % of
// every call.  l and the sums of p m' are in float32.
//
// Work split.  The tiles of all (request, kv head, row tile) items form one
// line, cut into equal pieces, one per resident warp: lengths are read on the
// device, and no warp has more than another but for a tile.  An item's
// beginning and end cost a warp about as much as START tiles, so each item is
// START units longer than its tiles in that line (64 requests of 1 to 8192
// tokens: 49.4 us with 4, 55.4 with 2, 62.0 with 1).  A warp works alone -- it
// copies its own tiles, keeps its own softmax and writes its own result -- so
// that the latencies of an SM's warps overlap and short requests cost no
// barrier.  An item cut by a piece's border leaves partial (ref, l, O) in a
// workspace, which a second kernel -- launched early, its wait overlapping the
// first's end -- merges in the order of the tokens.  Where one item covers all
// the pieces of a CTA its warps' parts are merged in shared memory first.
// Where the items are few and short by the sizes alone (no more than SMs, a few
// tiles a warp), each has a cluster of 1 to 8 CTAs, whose parts are merged
// through distributed shared memory, and there is no workspace and no second
// kernel: one request of 129 tokens 7.1 us against 9.2, 8 requests of 1000 10.1
// against 14.1, 4 of 4000 12.9 against 16.4.
//
// Memory.  Each warp owns a ring of stages of one tile (whole pages, 16 bytes
// a lane and copy), and asks for the next tile as soon as a stage is read.
//
// Bound.  More tokens cost what HBM takes to copy them (Hq 32, Hkv 8, D 128: 228
// requests of 1024 tokens to 2048, 269 MB more, cost 40.0 us more: 6.7 TB/s); a
// call's beginning (finding the piece, the first pages, Q), the items' ends and
// the merge are latency: 16 us in those calls, 19 us over the bytes' time in 64
// requests of 1 to 8192 tokens (49.4 us, 4.2 TB/s), 17.5 us in one of 131072
// (39.8 us, 3.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <mutex>
#include <type_traits>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int kMostParts = 64;    // CTAs that one item is cut into, at most
constexpr int kLeastUnits = 2;    // units of a piece, at least
constexpr int kClusterSizes = 3;  // clusters of 2, 4 and 8 CTAs
constexpr int kMostCluster = 1 << kClusterSizes;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -1e37f;  // reference of a row that has seen no key
constexpr int kMostSig = 126;     // exponent of a row's power of two before its first product
constexpr int kLeastTop = 4;      // a row's products reach 2^(kLeastTop - 1) before their rounding, at least
// What multiplies the weights (up to 2^15) in O's sums, so that these do not
// overflow before they are divided by l.  A smaller one would cost values near
// 2^-126 their bits: a term's rounding of 2^-150 over a largest weight of 2^-15
// is 2^-135, less than half of bfloat16's last place.
constexpr float kDown = 0x1p-25f;
constexpr uint32_t kBias = 4000;  // added to exponents, so that they are not negative
constexpr int kMaxRequests = ATTN_KV4_MAX_REQUESTS;

struct Kv4Params {
  const __nv_bfloat16 *q;
  int64_t qt, qh;  // element strides of token and head
  __nv_bfloat16 *o;
  float *lse;
  const int *cu, *lens, *table;
  int64_t table_stride;
  const uint8_t *cache;
  int num_pages, max_pages, B, T, H, group, shift, causal;
  float scale_log2;  // scale * log2 e
  int pieces;        // warps of the grid; 0: a cluster of CTAs for each item, no item is cut
  int cluster;       // CTAs of a cluster
  float *ws_o;       // partial O of cut items: [pieces][2][R][D]
  float2 *ws_ml;     // their reference and l: [pieces][2][R]
  int4 *ws_cut;      // [pieces][2]: the item that each piece leaves unfinished
  int *status;
};

// A variant: G groups of 64 dims, R query rows a tile, pages of P tokens.
template <int G_, int R_, int P_>
struct Shape {
  static constexpr int G = G_, R = R_, P = P_;
  static constexpr int D = G * kKv4Group;
  static constexpr int NT = R / 8;                     // n8 tiles of rows
  // tokens per tile (a stage of a warp's ring): whole pages, two of 16 tokens
  static constexpr int TK = P > 32 ? P : 32;
  static constexpr int PAGES = TK / P;
  static constexpr int PAGE_BYTES = kv4_page_bytes(G, P);
  static constexpr int STAGE = PAGES * PAGE_BYTES;
  // Warps of a CTA (one CTA per SM), as the registers allow: 128 a thread for
  // 64 dims, 168 for 128 dims or 16 rows of 64, 255 for more.
  static constexpr int WARPS = G == 1 ? (R == 8 ? 16 : 12) : G == 2 && R == 8 ? 12 : G == 4 && P == 64 ? 6 : 8;
  static constexpr int THREADS = WARPS * 32;
  // as many stages as the SM's shared memory holds, 8 at most
  static constexpr int FIT = 221184 / (WARPS * STAGE);
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = WARPS * STAGES * STAGE;
  // An item's beginning and end cost a warp about as much as this many tiles.
  static constexpr int START = TK == 32 ? 4 : 2;
  // offset of group j's K rows and pairs of a stage's 16 tokens number i
  static constexpr __host__ __device__ int code_row(int i, int j) {
    return P == 16 ? i * PAGE_BYTES + j * P * kKv4RowBytes : (j * P + i * 16) * kKv4RowBytes;
  }
  static constexpr __host__ __device__ int pair_row(int i, int j) {
    return P == 16 ? i * PAGE_BYTES + j * P * kKv4PairBytes : (j * P + i * 16) * kKv4PairBytes;
  }
  static_assert(STAGES >= 2, "a warp reads one stage while another fills");
  static_assert(STAGES * STAGE >= 2 * R * D * 4, "a warp's part of a shared item, and the CTA's, fit its ring");
};

// a / b for a >= 0, b > 0; in 32 bits where both fit, a third of the operations.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return (a | b) >> 31 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The tiles of a request whose cu descends: it has no row, and no other request
// has as many.  Where cu descends, requests could share query tokens and the line
// of units be longer than the host took it to be, so the line is left empty.
constexpr int kDescends = 1 << 30;

// What a request's tiles look like, from the device arrays, with whatever
// they hold brought into range (reported once through the status word).
struct Request {
  int t0, nq, len;   // first query token, query tokens, cached tokens
  int tiles, rt;     // tiles of tokens (at least one), row tiles
  __device__ __forceinline__ int64_t units(int H, int start) const { return (int64_t)H * rt * (tiles + start); }
};

template <typename S>
__device__ __forceinline__ Request load_request(const Kv4Params &p, int r) {
  Request q;
  const int a = p.cu[r], b = p.cu[r + 1], l = p.lens[r];
  const int room = p.max_pages << p.shift;
  q.t0 = min(max(a, 0), p.T);
  const int t1 = min(max(b, q.t0), p.T);
  q.nq = t1 - q.t0;
  q.len = min(max(l, 0), room);
  if (q.t0 != a || t1 != b || q.len != l) atomicCAS(p.status, 0, kStatusDevice);
  q.tiles = b < a ? kDescends : max(1, (q.len + S::TK - 1) / S::TK);
  q.rt = (int)(((int64_t)q.nq * p.group + S::R - 1) / S::R);
  return q;
}

// A place in the line of units: unit `off` of the item (request r, head h, row tile rt).
struct Place {
  int r, h, rt, off;
};

// A warp's piece of the line of units, and the item that holds the first unit
// of its CTA's pieces.
struct Piece {
  int64_t begin, end, chunk, total;
  Place at;         // of unit `begin`
  int64_t cta_begin, cta_end, item_begin, item_end;
  int warps;        // pieces of a CTA
  // one item covers the CTA, and more than one warp has a part of it
  __device__ __forceinline__ bool shared() const { return item_end >= cta_end && cta_begin + chunk < cta_end; }
  // ... and all of the item's tiles are in this CTA
  __device__ __forceinline__ bool complete(int start) const {
    return item_begin + start >= cta_begin && item_end == cta_end;
  }
};

// One cluster of CTAs for each item (few and short ones: spreading them further
// would cost more in merging than it saves): the cluster's warps share the item's
// tiles, and its parts are merged in shared memory, without a workspace or a
// second kernel.
template <typename S>
__device__ __forceinline__ void find_item(const Kv4Params &p, Piece &pc) {
  __shared__ Place found;
  __shared__ int tiles;
  __shared__ int64_t wsum[S::WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = (int)blockIdx.x / p.cluster, rank = (int)blockIdx.x % p.cluster;
  // The warp whose requests have the item: the first where 32 lanes hold them all, else each warp has a range of them
  // and they are counted first.
  int64_t before = 0;
  int r0 = 0, r1 = p.B;
  bool here = warp == 0;
  if (tid == 0) tiles = 0;
  if (p.B > 32) {
    const int per = ((p.B + S::THREADS - 1) / S::THREADS) * 32;
    r0 = min(warp * per, p.B);
    r1 = min(r0 + per, p.B);
    int64_t mine = 0;
#pragma unroll 4
    for (int r = r0 + lane; r < r1; r += 32) mine += (int64_t)p.H * load_request<S>(p, r).rt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) wsum[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < S::WARPS; ++w)
      if (w < warp) before += wsum[w];
    here = item >= before && item < before + mine;
  } else {
    __syncthreads();
  }
  if (here) {  // items before each request, 32 requests at a time
    for (int base = r0; base < r1 && before <= item; base += 32) {
      Request q{};
      if (base + lane < r1) q = load_request<S>(p, base + lane);
      const int64_t n = (int64_t)p.H * q.rt;
      int64_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      const int64_t i = item - (before + inc - n);
      if (i >= 0 && i < n) {
        found = Place{base + lane, (int)i / q.rt, (int)i % q.rt, 0};
        tiles = q.tiles;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  const int n = tiles, warps = S::WARPS * p.cluster, each = (n + warps - 1) / warps;  // tiles of a warp
  const int first = min((warp * p.cluster + rank) * each, n), last = min(first + each, n);
  pc = Piece{};
  pc.at = found;
  pc.at.off = S::START + first;
  pc.begin = pc.at.off;
  pc.end = S::START + last;
  pc.chunk = pc.warps = 1;
  pc.cta_end = pc.item_end = pc.total = n == 0 ? 0 : S::START + n;  // (0: no item is left for this CTA)
}

// What follows from the line's length: pieces, and how many of them a CTA has.
template <typename S>
__device__ __forceinline__ void set_piece(const Kv4Params &p, int64_t total, int longest, int warp, Piece &pc) {
  // equal pieces, but none so small that one item would be cut into more than
  // kMostParts CTAs: their merging would cost more than the tiles
  const int64_t chunk = max(max(divide(total + p.pieces - 1, p.pieces), (int64_t)kLeastUnits),
                            (int64_t)((longest + kMostParts * S::WARPS - 1) / (kMostParts * S::WARPS)));
  // where there are few pieces they are spread over the CTAs
  int warps = S::WARPS;
  if (chunk * (p.pieces - (int)gridDim.x) >= total)
    warps = (int)divide(divide(total + chunk - 1, chunk) + gridDim.x - 1, gridDim.x);
  pc.chunk = chunk;
  pc.total = total;
  pc.warps = warps;
  pc.cta_begin = min((int64_t)blockIdx.x * warps * chunk, total);
  pc.cta_end = min(pc.cta_begin + warps * chunk, total);
  pc.begin = min(pc.cta_begin + warp * chunk, pc.cta_end);
  pc.end = min(pc.begin + chunk, pc.cta_end);
}

// The place of unit `at` of the line in request r, whose first unit is `base`.
template <typename S>
__device__ __forceinline__ Place place_of(int64_t at, int64_t base, int r, const Request &q) {
  const int each = q.tiles + S::START;
  const int64_t i = divide(at - base, each);
  Place f;
  f.r = r;
  f.off = (int)(at - base - i * each);
  f.h = (int)divide(i, q.rt);
  f.rt = (int)(i - (int64_t)f.h * q.rt);
  return f;
}

// The warp's piece and where it begins, up to 128 requests: every warp looks
// them all up by itself, four a lane, without waiting for another.
template <typename S>
__device__ __forceinline__ void find_piece_few(const Kv4Params &p, Piece &pc) {
  constexpr int PER = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.B + 31) >> 5, r0 = lane * per;
  Request q[PER];
  int64_t mine = 0;
  int longest = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    q[k] = Request{0, 0, 0, 1, 0};
    if (k < per && r0 + k < p.B) q[k] = load_request<S>(p, r0 + k);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    mine += q[k].units(p.H, S::START);
    longest = max(longest, q[k].tiles);
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  const bool empty = longest >= kDescends;
  set_piece<S>(p, empty ? 0 : __shfl_sync(0xffffffffu, inc, 31), longest, warp, pc);
  Place mine_at{}, cta_at{};
  int64_t a = empty ? pc.cta_end + 1 : inc - mine;
  int each = 0;
  bool has = false, has_cta = false;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int64_t n = q[k].units(p.H, S::START);
    if (pc.begin >= a && pc.begin < a + n) {
      mine_at = place_of<S>(pc.begin, a, r0 + k, q[k]);
      has = true;
    }
    if (pc.cta_begin >= a && pc.cta_begin < a + n) {
      cta_at = place_of<S>(pc.cta_begin, a, r0 + k, q[k]);
      each = q[k].tiles + S::START;
      has_cta = true;
    }
    a += n;
  }
  const unsigned from = __ballot_sync(0xffffffffu, has), cta = __ballot_sync(0xffffffffu, has_cta);
  const int src = from ? __ffs(from) - 1 : 0, src_cta = cta ? __ffs(cta) - 1 : 0;
  pc.at = Place{__shfl_sync(0xffffffffu, mine_at.r, src), __shfl_sync(0xffffffffu, mine_at.h, src),
                __shfl_sync(0xffffffffu, mine_at.rt, src), __shfl_sync(0xffffffffu, mine_at.off, src)};
  pc.item_begin = cta ? pc.cta_begin - __shfl_sync(0xffffffffu, cta_at.off, src_cta) : 0;
  pc.item_end = cta ? pc.item_begin + __shfl_sync(0xffffffffu, each, src_cta) : 0;
}

// The same for any number of requests, by all threads of the CTA together.
template <typename S>
__device__ __forceinline__ void find_piece(const Kv4Params &p, Piece &pc) {
  __shared__ int64_t wsum[S::WARPS], item[2];
  __shared__ int wmax[S::WARPS];
  __shared__ Place found[S::WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + S::THREADS - 1) / S::THREADS;  // consecutive requests of a thread
  const int r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);
  int64_t mine = 0;
  int longest = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const Request q = load_request<S>(p, r);
    mine += q.units(p.H, S::START);
    longest = max(longest, q.tiles);
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    wsum[warp] = inc;
    wmax[warp] = longest;
  }
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < S::WARPS; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
    longest = max(longest, wmax[w]);
  }
  if (longest >= kDescends) total = 0;
  set_piece<S>(p, total, longest, warp, pc);
  int64_t a = before + inc - mine;
  if (mine > 0 && a < pc.cta_end && a + mine > pc.cta_begin) {  // some of the thread's requests are here
    for (int r = r0; r < r1; ++r) {
      const Request q = load_request<S>(p, r);
      const int64_t n = q.units(p.H, S::START);
#pragma unroll 1
      for (int w = 0; w < pc.warps; ++w) {
        const int64_t begin = pc.cta_begin + w * pc.chunk;
        if (begin < a || begin >= a + n) continue;
        found[w] = place_of<S>(begin, a, r, q);
        if (w == 0) {
          item[0] = begin - found[w].off;
          item[1] = item[0] + q.tiles + S::START;
        }
      }
      a += n;
    }
  }
  __syncthreads();
  pc.at = pc.begin < pc.end ? found[warp] : Place{};
  pc.item_begin = pc.cta_begin < total ? item[0] : 0;
  pc.item_end = pc.cta_begin < total ? item[1] : 0;
}

// One (request, kv head, row tile) of a piece: tiles [tile0, tile0 + n).
struct Item {
  Request q;
  int r, h, rt, tile0, n;
  bool whole;     // the piece holds all of the item
  int64_t end;    // the item's last unit + 1, in the line
  // last visible key + 1 of row `row` (rows count query token x group head)
  __device__ __forceinline__ int limit(int row, const Kv4Params &p) const {
    const int i = row < p.group ? 0 : row / p.group;
    return p.causal ? min(q.len, max(0, i + 1 + q.len - q.nq)) : q.len;
  }
};

// The first request from r on that has query tokens (B if none): the first whose
// end in cu, which does not descend here, lies past the end of request r - 1, by a
// search of the warp in 32 parts.
__device__ __noinline__ int next_active(const int *cu, int B, int T, int r) {
  const int lane = threadIdx.x & 31, from = min(max(cu[r], 0), T);
  int lo = r, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, last = min(lo + (lane + 1) * step, hi) - 1;
    const bool past = lo + lane * step < hi && min(max(cu[last + 1], 0), T) > from;
    const unsigned parts = __ballot_sync(0xffffffffu, past);
    if (parts == 0) return B;
    lo += (__ffs(parts) - 1) * step;
    if (step == 1) return lo;
    hi = min(lo + step, hi);
  }
  return B;
}

struct Walk {
  int64_t begin;   // of the place, in the line
  int left;        // units of the piece from there on
  Place at;
  Request q;
  template <typename S>
  __device__ __forceinline__ void start(const Kv4Params &p, const Piece &pc) {
    begin = pc.begin;
    left = (int)(pc.end - pc.begin);
    at = pc.at;
    if (left > 0) q = load_request<S>(p, at.r);
  }
  // Next item of the piece that has a tile in it; false at its end.
  template <typename S>
  __device__ __forceinline__ bool next(const Kv4Params &p, Item &it) {
    while (left > 0) {
      if (at.h == p.H) {
        if (++at.r >= p.B) return false;
        q = load_request<S>(p, at.r);
        if (q.rt == 0) {
          at.r = next_active(p.cu, p.B, p.T, at.r + 1);
          if (at.r >= p.B) return false;
          q = load_request<S>(p, at.r);
        }
        at.h = at.rt = at.off = 0;
      }
      const int each = q.tiles + S::START, n = min(each - at.off, left);
      const int tile0 = max(0, at.off - S::START), tile1 = max(0, at.off + n - S::START);
      it.q = q;
      it.r = at.r;
      it.h = at.h;
      it.rt = at.rt;
      it.tile0 = tile0;
      it.n = tile1 - tile0;
      it.end = begin - at.off + each;
      it.whole = it.n == q.tiles;
      left -= n;
      begin += n;
      at.off += n;
      if (at.off == each) {
        at.off = 0;
        if (++at.rt == q.rt) {
          at.rt = 0;
          ++at.h;
        }
      }
      if (tile1 > tile0) return true;  // (else no tile of the item itself: it begins in the next piece)
    }
    return false;
  }
};

// Output row (token x query head) of row q of an item whose first query token is t0.
__device__ __forceinline__ int64_t out_row(const Kv4Params &p, int t0, int h, int q) {
  const int i = q < p.group ? 0 : q / p.group;
  return (int64_t)(t0 + i) * (p.H * p.group) + h * p.group + (q - i * p.group);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8x8 matrices of 16-bit elements; lanes 8 i .. 8 i + 7 give the rows of
// the i-th.  Register i of lane (g, t): row g, elements 2t and 2t + 1 (or,
// transposed, column g, rows 2t and 2t + 1).
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Waits until all but the warp's last N groups of copies have landed (each lane its own; then __syncwarp).
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int4 as_int4(uint4 v) { return make_int4((int)v.x, (int)v.y, (int)v.z, (int)v.w); }
__device__ __forceinline__ float4 as_float4(uint4 v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t u;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(addr) : "memory");
  return u;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

// A row (or its part) without a visible key.  A row whose scores are all NaN
// keeps the initial reference too, but its l is NaN.
__device__ __forceinline__ bool saw_none(float ref, float l) { return ref == kNoRef && l == 0.f; }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// Exponent e of x = f * 2^e, f in [1, 2), for a positive normal x.
__device__ __forceinline__ int exp_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// The lane's part of the copy of tile `tile` of an item into the stage at
// `dst`: 16 bytes of every 512.  The pages' ids are in the lanes (lane i: page
// first + i; page 0 where the request has no further page, whose rows are
// never used).
template <typename S>
__device__ __forceinline__ void copy_tile(const uint8_t *head, uint32_t page_row, int tile, int ids, int first,
                                          uint32_t dst, int lane) {
  constexpr int CHUNKS = S::STAGE / 16, PAGE = S::PAGE_BYTES / 16;  // of 16 bytes
  const int at = tile * S::PAGES - first;
  const uint32_t id0 = __shfl_sync(0xffffffffu, ids, at);
  const uint8_t *src0 = head + (uint64_t)id0 * page_row + lane * 16, *src1 = src0;
  if (S::PAGES == 2) {
    const uint32_t id1 = __shfl_sync(0xffffffffu, ids, at + 1);
    src1 = head + (uint64_t)id1 * page_row + lane * 16 - S::PAGE_BYTES;
  }
  dst += lane * 16;
#pragma unroll
  for (int k = 0; k * 32 < CHUNKS; ++k) {
    const bool in_first = S::PAGES == 1 || k * 32 + 31 < PAGE || (k * 32 < PAGE && k * 32 + lane < PAGE);
    const uint8_t *src = in_first ? src0 : src1;
    if (k * 32 + 31 < CHUNKS || k * 32 + lane < CHUNKS) cp_async16(dst + k * 512, src + k * 512);
  }
}

// Ids of 32 pages from `first` on, one a lane (what is not a page of the
// cache is reported and read as the first page).
__device__ __forceinline__ int load_ids(const Kv4Params &p, int r, int first, int pages, int lane) {
  int id = 0;
  if (first + lane < pages) {
    id = p.table[(int64_t)r * p.table_stride + first + lane];
    if ((unsigned)id >= (unsigned)p.num_pages) {
      atomicCAS(p.status, 0, kStatusDevice);
      id = 0;
    }
  }
  return id;
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1) attn_kv4_kernel(const Kv4Params p) {
  constexpr int G = S::G, R = S::R, P = S::P, NT = S::NT, D = S::D, TK = S::TK;
  constexpr int STAGES = S::STAGES, WARPS = S::WARPS, THREADS = S::THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *ring = smem + warp * STAGES * S::STAGE;
  __shared__ float2 warp_ml[WARPS][R], cta_ml[R];
  __shared__ int4 warp_held[WARPS], cta_held;
  // What the loop over the tiles does not need waits in shared memory, so that
  // the loop keeps its operands in registers.
  __shared__ Walk walks[WARPS];
  __shared__ Piece pieces[WARPS];
  bool more;
  Item it;
  {
    Piece pc;
    if (p.pieces == 0)
      find_item<S>(p, pc);
    else if (p.B <= 128)
      find_piece_few<S>(p, pc);
    else
      find_piece<S>(p, pc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Walk walk;
    walk.start<S>(p, pc);
    more = walk.next<S>(p, it);
    if (lane == 0) {
      pieces[warp] = pc;
      walks[warp] = walk;
    }
    __syncwarp();
  }
  const int piece = blockIdx.x * WARPS + warp;
  const int g = lane >> 2, t = lane & 3;
  // the lane's row of the ldmatrix loads: matrices (tokens 0-7, 8-15) x (bytes 0-15, 16-31)
  const uint32_t row_off = ((lane & 7) + ((lane >> 3) & 1) * 8) * kKv4RowBytes + (lane >> 4) * 16;
  const uint32_t ring_s = smem_u32(ring);
  const uint32_t page_row = (uint32_t)p.H * (uint32_t)S::PAGE_BYTES;

  int st = 0;  // stage of the next tile
  int4 cut = make_int4(0, 0, 0, 0);  // the item left unfinished (no rows: none) ...
  int cut_last = 0, cut_flags = 0;   // ... the piece that ends it, and whether its first and last CTA share it (1, 2)
  int4 held = make_int4(0, 0, 0, 0);  // the last item this warp worked on (query token, head, first row, rows)
  // what the item's copies need: its tiles [tile0, stop), pages, and their ids
  int stop, pages, first, ids, ids_next, asked;
  const uint8_t *head;  // the kv head's block of the first page
  auto begin_copies = [&]() {
    const int last_row = min(it.q.nq * p.group, (it.rt + 1) * R) - 1;
    stop = min(it.tile0 + it.n, (it.limit(last_row, p) + TK - 1) / TK);
    pages = (it.q.len + P - 1) / P;
    first = it.tile0 * S::PAGES;
    head = p.cache + (int64_t)it.h * S::PAGE_BYTES;
    ids = load_ids(p, it.r, first, pages, lane);
    ids_next = load_ids(p, it.r, first + 32, pages, lane);
    asked = it.tile0;
    int s = st;
    for (int i = 0; i < STAGES; ++i) {  // one group a stage, whether it copies or not; 32 ids cover the first tiles
      if (asked < stop) copy_tile<S>(head, page_row, asked++, ids, first, ring_s + s * S::STAGE, lane);
      cp_async_commit();
      if (++s == STAGES) s = 0;
    }
  };
  if (more) begin_copies();

  while (more) {
    const int rows = it.q.nq * p.group;
    const int row0 = it.rt * R;
    const int full_to = min(it.limit(row0, p), it.q.len);  // tokens before it are visible to every row

    // Q: lane (g, t) holds row g's dims of word t of each half of each group,
    // scaled by a power of two so that the row's largest value is in [2^14, 2^15)
    uint32_t qb[NT][G][4][2];
    float fac[NT][2], qsum[NT][G][2];  // per column pair (rows 2t, 2t + 1): scale of y, sums of the scaled q
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 8 + g;
      uint4 w[G][2];
#pragma unroll
      for (int j = 0; j < G; ++j) w[j][0] = w[j][1] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const int i = row < p.group ? 0 : row / p.group, hg = row - i * p.group;
        const __nv_bfloat16 *src =
            p.q + (int64_t)(it.q.t0 + i) * p.qt + (int64_t)(it.h * p.group + hg) * p.qh + t * 8;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          w[j][0] = *reinterpret_cast<const uint4 *>(src + j * kKv4Group);
          w[j][1] = *reinterpret_cast<const uint4 *>(src + j * kKv4Group + 32);
        }
      }
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t ws[4] = {w[j][k].x, w[j][k].y, w[j][k].z, w[j][k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            big = max3f(big, fabsf(__uint_as_float(ws[e] << 16)), fabsf(__uint_as_float(ws[e] & 0xffff0000u)));
        }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^e scales the row (e in [-114, 126]; zero, subnormal and infinite rows stay in range)
      const int e = min(126, 14 - exp_of(fmaxf(big, 0x1p-112f)));
      const float up = pow2(e), up16 = pow2(e - 4);
      float qs[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        qs[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[8];
          const uint32_t ws[4] = {w[j][k].x, w[j][k].y, w[j][k].z, w[j][k].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // odd dims over 16: their nibbles carry that factor
            v[2 * c] = __uint_as_float(ws[c] << 16) * up;
            v[2 * c + 1] = __uint_as_float(ws[c] & 0xffff0000u) * up16;
            qs[j] = fmaf(v[2 * c + 1], 16.f, qs[j] + v[2 * c]);
          }
          // nibbles (0, 4) and (1, 5), then (2, 6) and (3, 7)
          qb[nt][j][2 * k][0] = half2_bits(v[0], v[4]);
          qb[nt][j][2 * k][1] = half2_bits(v[1], v[5]);
          qb[nt][j][2 * k + 1][0] = half2_bits(v[2], v[6]);
          qb[nt][j][2 * k + 1][1] = half2_bits(v[3], v[7]);
        }
        qs[j] += __shfl_xor_sync(0xffffffffu, qs[j], 1);
        qs[j] += __shfl_xor_sync(0xffffffffu, qs[j], 2);
        // the accumulators hold 2^-24 of q . c
#pragma unroll
        for (int c = 0; c < 2; ++c) qsum[nt][j][c] = __shfl_sync(0xffffffffu, qs[j], (2 * t + c) * 4) * 0x1p-24f;
      }
      const float down = pow2(-e) * p.scale_log2 * 0x1p24f;
#pragma unroll
      for (int c = 0; c < 2; ++c) fac[nt][c] = __shfl_sync(0xffffffffu, down, (2 * t + c) * 4);
    }

    float acc[NT][G][4][4];  // O^T: [row tile][group][dim tile][c]
    float ref[NT][2], l[NT][2], vm[NT][G][2];
    float isig[NT][G][2];  // the power of two by which a row's weighted scales of V are brought to half precision
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = row0 + nt * 8 + 2 * t + c;
        lim[nt][c] = row < rows ? it.limit(row, p) : 0;
      }

    // The item's tiles.  Usually V's scales lie within 2^6 of each other, and one power of two a group serves all rows
    // (EACH false); where they do not, or a score passes 2^20, that ends with false, and the tiles are taken again with
    // one for each row and group.
    auto attend = [&](auto each) -> bool {
      constexpr bool EACH = decltype(each)::value;
      float top_sig[G];  // the rows' largest power of two
      int least[G];      // exponent (biased by 127) of the smallest scale in the units that moved a reference
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          ref[nt][c] = kNoRef;
          l[nt][c] = 0.f;
          // (0: a row that sees nothing here)
#pragma unroll
          for (int j = 0; j < G; ++j) isig[nt][j][c] = lim[nt][c] > it.tile0 * TK ? pow2(kMostSig) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
          vm[nt][j][0] = vm[nt][j][1] = 0.f;
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[nt][j][d][0] = acc[nt][j][d][1] = acc[nt][j][d][2] = acc[nt][j][d][3] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        top_sig[j] = pow2(kMostSig);
        least[j] = 255;
      }

      for (int tile = it.tile0; tile < stop; ++tile) {
        cp_async_wait<STAGES - 1>();
        __syncwarp();
#pragma unroll 1
        for (int u = 0; u < TK / 32; ++u) {
          const int tok0 = tile * TK + u * 32;
          if (u > 0 && tok0 >= it.q.len) break;
          const bool tail = tok0 + 32 > it.q.len;
          bool edge = tok0 + 32 > full_to;
          // the first K row of each 16 tokens; everything else is at a fixed distance
          const uint32_t kc = ring_s + st * S::STAGE + u * (S::code_row(2, 0) - S::code_row(0, 0)) + row_off;
          const uint32_t km = ring_s + st * S::STAGE + u * (S::pair_row(2, 0) - S::pair_row(0, 0)) +
                              kv4_codes_bytes(G, P) + g * kKv4PairBytes;
          // the lane's tokens of S^T: ta, ta + 8 of each 16
          const int ta = tok0 + g;

          // S^T = K Q^T on the codes, joined over the groups with scales and minima
          float x[2][NT][4];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
              uint32_t w[4];  // tokens g and g + 8 of the first 32 dims, then of the others
              ldmatrix4(w, kc + S::code_row(hf, j));
              const uint32_t pa = lds32(km + S::pair_row(hf, j));
              const uint32_t pb = lds32(km + S::pair_row(hf, j) + 8 * kKv4PairBytes);
              float s[NT][4];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t xa = w[2 * k], xb = w[2 * k + 1];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const uint32_t a0 = xa & 0x000f000fu, a1 = xb & 0x000f000fu;
                  const uint32_t a2 = xa & 0x00f000f0u, a3 = xb & 0x00f000f0u;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma_f16(s[nt], a0, a1, a2, a3, qb[nt][j][2 * k + hh][0], qb[nt][j][2 * k + hh][1]);
                  xa >>= 8;
                  xb >>= 8;
                }
              }
              const float sa = __uint_as_float(pa << 16), ma = __uint_as_float(pa & 0xffff0000u);
              const float sb = __uint_as_float(pb << 16), mb = __uint_as_float(pb & 0xffff0000u);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float &xa = x[hf][nt][c], &xb = x[hf][nt][2 + c];
                  xa = fmaf(sa, s[nt][c], j ? fmaf(ma, qsum[nt][j][c], xa) : ma * qsum[nt][j][c]);
                  xb = fmaf(sb, s[nt][2 + c], j ? fmaf(mb, qsum[nt][j][c], xb) : mb * qsum[nt][j][c]);
                }
            }
          }
          // V's scales and minima of the lane's tokens (of those past the request's end none, whatever they are)
          uint32_t pv[2][G][2];
          float big_v = 0.f;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int j = 0; j < G; ++j) {
              const uint32_t vp = km + kv4_side_bytes(G, P) + S::pair_row(hf, j);
              pv[hf][j][0] = lds32(vp);
              pv[hf][j][1] = lds32(vp + 8 * kKv4PairBytes);
              if (tail) {
                if (ta + hf * 16 >= it.q.len) pv[hf][j][0] = 0u;
                if (ta + hf * 16 + 8 >= it.q.len) pv[hf][j][1] = 0u;
              }
              big_v = max3f(big_v, __uint_as_float(pv[hf][j][0] << 16) * top_sig[j],
                            __uint_as_float(pv[hf][j][1] << 16) * top_sig[j]);
            }
          // e = y - ref in log2 units; hidden tokens -inf (selected, so that nothing they hold is used)
          float e[2][NT][4];
          float top = -INFINITY;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float &ea = e[hf][nt][c], &eb = e[hf][nt][2 + c];
                ea = fmaf(x[hf][nt][c], fac[nt][c], -ref[nt][c]);
                eb = fmaf(x[hf][nt][2 + c], fac[nt][c], -ref[nt][c]);
                if (edge) {
                  if (ta + hf * 16 >= lim[nt][c]) ea = -INFINITY;
                  if (ta + hf * 16 + 8 >= lim[nt][c]) eb = -INFINITY;
                }
                top = max3f(top, ea, eb);
              }
          if (__any_sync(0xffffffffu, top > 15.f || big_v > 1.9f)) {  // move the references up
            if constexpr (!EACH) {
              // The largest scale becomes [0.5, 1), so that no weight up to 2^15 overflows.  A row's largest product
              // is then at least 2^(kLeastTop - 1), if the smallest scale of the units that moved references is not
              // below 2^-6 of the largest: the row's heaviest token (weight 2^10 then) was in one of them.
              bool plain = true;
              float fs[G];
#pragma unroll
              for (int j = 0; j < G; ++j) {
                int big = 0;  // of the scales that are numbers
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const uint32_t s = pv[hf][j][u] << 16;
                    const int ex = s < 0x7f800000u ? s >> 23 : 0;
                    big = max(big, ex);
                    if (!tail || ta + hf * 16 + u * 8 < it.q.len) least[j] = min(least[j], ex);
                  }
                big = __reduce_max_sync(0xffffffffu, big);
                least[j] = __reduce_min_sync(0xffffffffu, least[j]);
                const int old = exp_of(top_sig[j]), now = max(-126, min(old, 126 - big));
                plain = plain && least[j] + now >= 127 - 11 + kLeastTop;
                top_sig[j] = pow2(now);
                fs[j] = pow2(max(now - old, -126));  // (from its first value there is nothing to take along)
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float m = -INFINITY;
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = c; u < 4; u += 2)
                      if (e[hf][nt][u] != -INFINITY) m = fmaxf(m, x[hf][nt][u] * fac[nt][c]);
#pragma unroll
                  for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                  const float now = fmaxf(ref[nt][c], m - 10.f);
                  const float f = ex2_approx(ref[nt][c] - now);
                  plain = plain && (now <= kNoRef || fabsf(now) < 0x1p20f);
                  ref[nt][c] = now;
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = c; u < 4; u += 2)
                      if (e[hf][nt][u] != -INFINITY) e[hf][nt][u] = fmaf(x[hf][nt][u], fac[nt][c], -now);
                  l[nt][c] *= f;
#pragma unroll
                  for (int j = 0; j < G; ++j) {
                    vm[nt][j][c] *= f;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                      acc[nt][j][d][c] *= f * fs[j];
                      acc[nt][j][d][2 + c] *= f * fs[j];
                    }
                  }
                }
              if (!__all_sync(0xffffffffu, plain)) return false;
            } else {
              // Exponents (biased by 127) of the scales that are numbers, in both halves of a word, and of the largest
              // of a group; those of the rows' new powers of two
              uint32_t es[G][2][2];
              int big[G], most[G];
              bool far_off = false;  // a scale times the power of two may pass float32, at a token of next to no weight
#pragma unroll
              for (int j = 0; j < G; ++j) {
                big[j] = 0;
                most[j] = -127;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const uint32_t s = pv[hf][j][u] << 16;
                    const int ex = s < 0x7f800000u ? s >> 23 : 0;
                    es[j][hf][u] = ex * 0x10001u;
                    big[j] = max(big[j], ex);
                  }
                big[j] = __reduce_max_sync(0xffffffffu, big[j]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float down[2], f[2];
                uint32_t ey[2][2][2];  // [half][token][row]: the weight's exponent, far down where the token is hidden
                int up[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float m = -INFINITY;
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = c; u < 4; u += 2)
                      if (e[hf][nt][u] != -INFINITY) m = fmaxf(m, __fmul_rn(x[hf][nt][u], fac[nt][c]));
#pragma unroll
                  for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                  const float now = fmaxf(ref[nt][c], m - 10.f);
                  down[c] = ref[nt][c] - now;
                  f[c] = ex2_approx(down[c]);
                  up[c] = (int)ceilf(fminf(-down[c], 300.f));  // whole powers of two that the weights have shrunk by
                  ref[nt][c] = now;
                  l[nt][c] *= f[c];
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = c; u < 4; u += 2)
                      if (e[hf][nt][u] != -INFINITY) e[hf][nt][u] = fmaf(x[hf][nt][u], fac[nt][c], -now);
                  if (__any_sync(0xffffffffu, now > kNoRef && fabsf(now) >= 0x1p20f)) {
                    // The rounding of the product that gave the reference counts here: without it the largest score's
                    // y may be anything instead of 10, and its weight none or infinite.
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                      for (int u = c; u < 4; u += 2) {
                        const float y = __fsub_rn(__fmul_rn(x[hf][nt][u], fac[nt][c]), now);
                        if (e[hf][nt][u] != -INFINITY) e[hf][nt][u] = y > 15.f ? 15.f : y;
                      }
                  }
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                      const float y = e[hf][nt][2 * u + c];
                      const bool seen = y != -INFINITY;
                      // (the bits of 1.5 * 2^23 + y are those of 1.5 * 2^23, plus y's nearest whole number)
                      const float near = fminf(fmaxf(y, -1000.f), 100.f);
                      ey[hf][u][c] = seen ? __float_as_uint(near + 12582912.f) - 0x4b400000u + kBias : kBias - 2000u;
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                  // The exponent of the largest weighted scale that each row sees here (row c in half c), or of what it
                  // has summed so far over the largest code.
                  uint32_t key = 0;
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    float held = 0.f;
#pragma unroll
                    for (int d = 0; d < 4; ++d) held = max3f(held, acc[nt][j][d][c], acc[nt][j][d][2 + c]);
                    const int sum = exp_of(held) + 20 - exp_of(isig[nt][j][c]) - up[c];
                    key |= (uint32_t)(sum + 127 + (int)kBias) << (16 * c);
                  }
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = 0; u < 2; ++u) key = __vmaxu2(key, es[j][hf][u] + ey[hf][u][0] + (ey[hf][u][1] << 16));
#pragma unroll
                  for (int o = 4; o < 32; o <<= 1) key = __vmaxu2(key, __shfl_xor_sync(0xffffffffu, key, o));
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    vm[nt][j][c] *= f[c];
                    // The largest scale becomes [0.5, 1), so that no weight up to 2^15 overflows, unless that took the
                    // row's largest product too low; what the row has summed keeps its place where that falls.
                    const int old = exp_of(isig[nt][j][c]);
                    const int low = min(old, 126 - big[j]);
                    const int need = kLeastTop + 127 + (int)kBias - (int)(c ? key >> 16 : key & 0xffffu);
                    const int next = old == -127 ? old : max(-126, min(min(old + up[c], kMostSig), max(low, need)));
                    const float by =
                        next <= old ? f[c] * pow2(max(next - old, -126)) : ex2_approx(down[c] + (float)(next - old));
                    isig[nt][j][c] = pow2(next);
                    most[j] = max(most[j], next);
                    far_off = far_off || next > 252 - big[j];
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                      acc[nt][j][d][c] *= by;
                      acc[nt][j][d][2 + c] *= by;
                    }
                  }
                }
              }
#pragma unroll
              for (int j = 0; j < G; ++j) top_sig[j] = pow2(__reduce_max_sync(0xffffffffu, most[j]));
              if (__any_sync(0xffffffffu, far_off)) edge = true;
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float pr[NT][4], pm[NT][4];  // weights, and what multiplies the minima
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                pr[nt][c] = ex2_approx(e[hf][nt][c]);
                pr[nt][2 + c] = ex2_approx(e[hf][nt][2 + c]);
                l[nt][c] += pr[nt][c] + pr[nt][2 + c];
                pm[nt][c] = pr[nt][c] * kDown;
                pm[nt][2 + c] = pr[nt][2 + c] * kDown;
              }
            // O^T += V^T P^T
#pragma unroll
            for (int j = 0; j < G; ++j) {
              const uint32_t pa = pv[hf][j][0], pb = pv[hf][j][1];
              const float sa = __uint_as_float(pa << 16), sb = __uint_as_float(pb << 16);
              const float ma = __uint_as_float(pa & 0xffff0000u), mb = __uint_as_float(pb & 0xffff0000u);
              uint32_t b0[NT], b1[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float w[4];
                if constexpr (EACH) {
                  const uint64_t up = f2_pack(isig[nt][j][0], isig[nt][j][1]);
                  f2_unpack(f2_mul(f2_pack(pr[nt][0], pr[nt][1]), f2_mul(f2_pack(sa, sa), up)), w[0], w[1]);
                  f2_unpack(f2_mul(f2_pack(pr[nt][2], pr[nt][3]), f2_mul(f2_pack(sb, sb), up)), w[2], w[3]);
                } else {
                  const float ua = sa * top_sig[j], ub = sb * top_sig[j];
                  w[0] = pr[nt][0] * ua;
                  w[1] = pr[nt][1] * ua;
                  w[2] = pr[nt][2] * ub;
                  w[3] = pr[nt][3] * ub;
                }
                if (!edge) {
#pragma unroll
                  for (int c = 0; c < 2; ++c) vm[nt][j][c] = fmaf(pm[nt][2 + c], mb, fmaf(pm[nt][c], ma, vm[nt][j][c]));
                } else {
                  // A hidden token's scale and minimum may be anything; a scale of next to no weight may have passed
                  // float32 (of a weight above 2^-120 it has not: the row's products are below 2^6).
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const bool no_a = e[hf][nt][c] == -INFINITY, no_b = e[hf][nt][2 + c] == -INFINITY;
                    if (no_a || (EACH && e[hf][nt][c] < -120.f && sa < INFINITY)) w[c] = 0.f;
                    if (no_b || (EACH && e[hf][nt][2 + c] < -120.f && sb < INFINITY)) w[2 + c] = 0.f;
                    vm[nt][j][c] = fmaf(pm[nt][2 + c], no_b ? 0.f : mb, fmaf(pm[nt][c], no_a ? 0.f : ma, vm[nt][j][c]));
                  }
                }
                b0[nt] = transpose8x8(half2_bits(w[0], w[1]));
                b1[nt] = transpose8x8(half2_bits(w[2], w[3]));
              }
              // dims 4g .. 4g + 3 of tokens (2t, 2t + 1) and (8 + 2t, 9 + 2t), then those of the other 32 dims
              uint32_t z[4];
              ldmatrix4_trans(z, kc + kv4_side_bytes(G, P) + S::code_row(hf, j));
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t z0 = z[2 * k], z1 = z[2 * k + 1];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const uint32_t a0 = z0 & 0x000f000fu, a1 = z0 & 0x00f000f0u;
                  const uint32_t a2 = z1 & 0x000f000fu, a3 = z1 & 0x00f000f0u;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][j][2 * k + hh], a0, a1, a2, a3, b0[nt], b1[nt]);
                  z0 >>= 8;
                  z1 >>= 8;
                }
              }
            }
          }
        }
        __syncwarp();  // every lane has read the stage
        if (asked < stop) {
          if (asked * S::PAGES - first >= 32) {
            first += 32;
            ids = ids_next;
            ids_next = load_ids(p, it.r, first + 32, pages, lane);
          }
          copy_tile<S>(head, page_row, asked++, ids, first, ring_s + st * S::STAGE, lane);
        }
        cp_async_commit();
        if (++st == STAGES) st = 0;
      }
      if constexpr (!EACH) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < G; ++j) isig[nt][j][0] = isig[nt][j][1] = top_sig[j];
      }
      return true;
    };
    if (!attend(std::false_type{})) {
      cp_async_wait<0>();  // the copies that are on their way land before their stages are filled again
      __syncwarp();
      begin_copies();
      attend(std::true_type{});
    }

    // ---- the item's end: the next item's first tiles are asked for, then the lanes are summed and the rows written
    const Item done = it;
    const Piece &pc = pieces[warp];
    {
      Walk walk = walks[warp];
      more = walk.next<S>(p, it);
      __syncwarp();
      if (lane == 0) walks[warp] = walk;
      __syncwarp();
    }
    const bool part_s = pc.shared();  // a part of the item that the whole CTA shares
    const bool whole = done.whole && !part_s;
    if (more) begin_copies();
    if (done.tile0 == 0 && !whole && !(part_s && pc.complete(S::START))) {
      cut = make_int4(done.q.t0, done.h, row0, min(rows - row0, R));
      cut_last = (int)((done.end - 1) / pc.chunk);
      const int64_t last_begin = (int64_t)(cut_last / pc.warps) * pc.warps * pc.chunk;
      const int64_t last_end = min(last_begin + pc.warps * pc.chunk, pc.total);
      const bool last_s =
          cut_last / pc.warps != (int)blockIdx.x && done.end >= last_end && last_begin + pc.chunk < last_end;
      cut_flags = (part_s ? 1 : 0) | (last_s ? 2 : 0);
    }
    // a shared item's part goes to shared memory (this warp's ring, empty by now)
    const int64_t part = ((int64_t)piece * 2 + (done.tile0 > 0 ? 0 : 1)) * R;
    float *const part_o = part_s ? reinterpret_cast<float *>(ring) : p.ws_o + part * D;
    float2 *const part_ml = part_s ? warp_ml[warp] : p.ws_ml + part;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
#pragma unroll
          for (int j = 0; j < G; ++j) vm[nt][j][c] += __shfl_xor_sync(0xffffffffu, vm[nt][j][c], o);
        }
        const int row = nt * 8 + 2 * t + c, q = row0 + row;
        if (q >= rows) continue;
        const bool none = saw_none(ref[nt][c], l[nt][c]);
        const float inv = whole ? (none ? 0.f : __frcp_rn(l[nt][c]) / kDown) : 1.f;
        const int64_t at = out_row(p, done.q.t0, done.h, q);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          // 1 / isig, a power of two as isig is
          const float sig = __uint_as_float((254u << 23) - __float_as_uint(isig[nt][j][c])), m = vm[nt][j][c];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float o[4];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              o[2 * d] = fmaf(acc[nt][j][2 * k + d][c] * (0x1p24f * kDown), sig, m) * inv;
              o[2 * d + 1] = fmaf(acc[nt][j][2 * k + d][2 + c] * (0x1p20f * kDown), sig, m) * inv;
            }
            const int dim = j * kKv4Group + k * 32 + g * 4;
            if (whole)
              *reinterpret_cast<uint2 *>(p.o + at * D + dim) =
                  make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            else
              *reinterpret_cast<float4 *>(part_o + row * D + dim) = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
        if (g == 0) {
          if (whole)
            p.lse[at] = none ? -INFINITY : (ref[nt][c] + log2f(l[nt][c])) * kLn2;
          else
            part_ml[row] = make_float2(ref[nt][c], l[nt][c]);
        }
      }
    held = make_int4(done.q.t0, done.h, row0, min(rows - row0, R));
  }
  const Piece &pc = pieces[warp];
  if (pc.shared()) {
    // The warps' parts of the one item, merged: to the output if that is all of it, else to the CTA's partial.
    if (lane == 0) warp_held[warp] = held;
    __syncthreads();
    int4 d = warp_held[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w)
      if (d.w == 0) d = warp_held[w];  // (a warp may have had none of its tiles)
    const bool all = pc.complete(S::START), clustered = p.cluster > 1;
    // the CTA's partial: its own shared memory (behind warp 0's part), or the workspace
    const int64_t part = (int64_t)blockIdx.x * WARPS * 2 * R;
    float *const cta_o = clustered ? reinterpret_cast<float *>(smem) + R * D : p.ws_o + part * D;
    float2 *const to_ml = clustered ? cta_ml : p.ws_ml + part;
    for (int i = tid; i < d.w * (D / 4); i += THREADS) {
      const int row = i / (D / 4), dim = (i % (D / 4)) * 4;
      float m = kNoRef, l = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        if (warp_held[w].w) m = fmaxf(m, warp_ml[w][row].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        if (warp_held[w].w == 0) continue;
        const float2 ml = warp_ml[w][row];
        if (saw_none(ml.x, ml.y)) continue;
        const float f = ex2_approx(ml.x - m);
        const float *theirs = reinterpret_cast<const float *>(smem + w * STAGES * S::STAGE);
        const float4 v = *reinterpret_cast<const float4 *>(theirs + row * D + dim);
        l = fmaf(f, ml.y, l);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      if (all && !clustered) {
        const bool none = saw_none(m, l);
        const float inv = none ? 0.f : 1.f / kDown / l;
        const int64_t at = out_row(p, d.x, d.y, d.z + row);
        *reinterpret_cast<uint2 *>(p.o + at * D + dim) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (dim == 0) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(cta_o + row * D + dim) = o;
        if (dim == 0) to_ml[row] = make_float2(m, l);
      }
    }
    if (clustered) {
      // The CTAs' partials, merged by all of them.  Every CTA of the cluster is here: they share one item.  The first
      // one's first warp has the item's first tile, so it knows the rows.
      if (tid == 0) cta_held = d;
      __syncwarp();
      cluster_sync_all();
      const uint32_t o_s = smem_u32(cta_o), ml_s = smem_u32(cta_ml), held_s = smem_u32(&cta_held);
      d = as_int4(ld_cluster_v4(mapa_shared(held_s, 0)));
      const int rank = (int)cluster_ctarank();
      for (int i = rank * THREADS + tid; i < d.w * (D / 4); i += p.cluster * THREADS) {
        const int row = i / (D / 4), dim = (i % (D / 4)) * 4;
        float2 ml[kMostCluster];
        float4 v[kMostCluster];
        float m = kNoRef, l = 0.f;
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          ml[c] = make_float2(kNoRef, 0.f);
          v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          // (.w: a CTA without a tile)
          if (c >= p.cluster || ld_cluster_u32(mapa_shared(held_s + 12, c)) == 0) continue;
          ml[c] = ld_cluster_f2(mapa_shared(ml_s + row * 8, c));
          v[c] = as_float4(ld_cluster_v4(mapa_shared(o_s + (row * D + dim) * 4, c)));
          m = fmaxf(m, ml[c].x);
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          if (saw_none(ml[c].x, ml[c].y)) continue;
          const float f = ex2_approx(ml[c].x - m);
          l = fmaf(f, ml[c].y, l);
          o.x = fmaf(f, v[c].x, o.x);
          o.y = fmaf(f, v[c].y, o.y);
          o.z = fmaf(f, v[c].z, o.z);
          o.w = fmaf(f, v[c].w, o.w);
        }
        const bool none = saw_none(m, l);
        const float inv = none ? 0.f : 1.f / kDown / l;
        const int64_t at = out_row(p, d.x, d.y, d.z + row);
        *reinterpret_cast<uint2 *>(p.o + at * D + dim) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (dim == 0) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      __syncwarp();
      cluster_sync_all();  // no CTA leaves while another reads its shared memory
    }
  }
  if (lane == 0 && p.pieces > 0) {
    p.ws_cut[piece * 2] = cut;
    p.ws_cut[piece * 2 + 1] = make_int4(cut_last, cut_flags, pc.warps, 0);
  }
}

// Merges the items that the pieces of CTA blockIdx.x of the first kernel began
// and left unfinished.  Their parts, in order: the beginning piece's second
// partial and the first partials of the pieces after it in that CTA, one
// partial for each CTA that shares the item, the first partials of the last
// CTA's pieces.  With M = max ref_i:
//     O = sum 2^(ref_i - M) O_i / sum 2^(ref_i - M) l_i.
// The rows of all these items are the CTA's tasks; a warp sums every per-th
// part of one of them with a running reference, several loads in flight, and
// the warps of a row are joined through shared memory: a fixed order.
constexpr int kMergeWarps = 32;
constexpr int kMergeThreads = kMergeWarps * 32;

template <typename S>
__global__ void __launch_bounds__(kMergeThreads) attn_kv4_merge_kernel(const Kv4Params p) {
  constexpr int D = S::D, R = S::R, WARPS = S::WARPS, V = (D / 4 + 31) / 32;  // float4s of a lane
  constexpr int U = V == 1 ? 4 : 2;                        // parts in flight
  __shared__ __align__(16) float part[kMergeWarps][D];
  __shared__ float2 part_ml[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * WARPS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // lane k: the item that piece k left unfinished, and its rows summed up to it
  int4 cut = make_int4(0, 0, 0, 0), end = cut;
  if (lane < WARPS) {
    cut = p.ws_cut[2 * (c0 + lane)];
    end = p.ws_cut[2 * (c0 + lane) + 1];
  }
  int sum = cut.w;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, x);
    if (lane >= x) sum += u;
  }
  const int tasks = __shfl_sync(0xffffffffu, sum, 31);
  // warps of a task: the most that leaves every task some
  int per = kMergeWarps;
  while (per > 1 && tasks * per > kMergeWarps) per >>= 1;
  for (int task0 = 0; task0 < tasks; task0 += kMergeWarps / per) {
    const int task = task0 + warp / per, sub = warp % per;
    const bool mine = task < tasks;
    const int k = __popc(__ballot_sync(0xffffffffu, sum <= task)) & 31;
    const int4 d = make_int4(__shfl_sync(0xffffffffu, cut.x, k), __shfl_sync(0xffffffffu, cut.y, k),
                             __shfl_sync(0xffffffffu, cut.z, k), __shfl_sync(0xffffffffu, cut.w, k));
    const int3 e = make_int3(__shfl_sync(0xffffffffu, end.x, k), __shfl_sync(0xffffffffu, end.y, k),
                             __shfl_sync(0xffffffffu, end.z, k));
    const int row = task - (__shfl_sync(0xffffffffu, sum, k) - d.w);
    float m = kNoRef, l = 0.f;
    float4 o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) {
      // pieces in order: piece i is warp i % e.z of CTA i / e.z
      const int first = blockIdx.x * e.z + k, last = e.x, lc = last / e.z;
      const int n1 = e.y & 1 ? 1 : min(last, (int)(blockIdx.x + 1) * e.z - 1) - first + 1;
      const int nm = max(0, lc - (int)blockIdx.x - 1);
      const int n = n1 + nm + (lc == (int)blockIdx.x ? 0 : e.y & 2 ? 1 : last - lc * e.z + 1);
      for (int i0 = sub; i0 < n; i0 += per * U) {
        float2 ml[U];
        float4 w[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * per;
          ml[u] = make_float2(kNoRef, 0.f);
          if (i >= n) continue;
          const int slot = i < n1        ? (e.y & 1 ? 2 * c0 : 2 * (c0 + k + i) + (i == 0 ? 1 : 0))
                           : i < n1 + nm ? 2 * WARPS * ((int)blockIdx.x + 1 + i - n1)
                                         : 2 * (lc * WARPS + i - n1 - nm);
          const int64_t at = (int64_t)slot * R + row;
          ml[u] = p.ws_ml[at];
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v * 128 + lane * 4 < D)
              w[u][v] = *reinterpret_cast<const float4 *>(p.ws_o + at * D + v * 128 + lane * 4);
        }
        float now = m;
#pragma unroll
        for (int u = 0; u < U; ++u) now = fmaxf(now, ml[u].x);
        const float f0 = ex2_approx(m - now);
        m = now;
        l *= f0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v].x *= f0;
          o[v].y *= f0;
          o[v].z *= f0;
          o[v].w *= f0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u * per >= n || saw_none(ml[u].x, ml[u].y)) continue;
          const float f = ex2_approx(ml[u].x - m);
          l = fmaf(f, ml[u].y, l);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            o[v].x = fmaf(f, w[u][v].x, o[v].x);
            o[v].y = fmaf(f, w[u][v].y, o[v].y);
            o[v].z = fmaf(f, w[u][v].z, o[v].z);
            o[v].w = fmaf(f, w[u][v].w, o[v].w);
          }
        }
      }
    }
    if (per > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 128 + lane * 4 < D) *reinterpret_cast<float4 *>(&part[warp][v * 128 + lane * 4]) = o[v];
      if (lane == 0) part_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (mine && sub == 0) {
        float now = m;
        for (int w = 1; w < per; ++w) now = fmaxf(now, part_ml[warp + w].x);
        const float f0 = saw_none(m, l) ? 0.f : ex2_approx(m - now);
        m = now;
        l *= f0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v].x *= f0;
          o[v].y *= f0;
          o[v].z *= f0;
          o[v].w *= f0;
        }
        for (int w = 1; w < per; ++w) {
          const float2 ml = part_ml[warp + w];
          if (saw_none(ml.x, ml.y)) continue;
          const float f = ex2_approx(ml.x - m);
          l = fmaf(f, ml.y, l);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (v * 128 + lane * 4 >= D) break;
            const float4 u = *reinterpret_cast<const float4 *>(&part[warp + w][v * 128 + lane * 4]);
            o[v].x = fmaf(f, u.x, o[v].x);
            o[v].y = fmaf(f, u.y, o[v].y);
            o[v].z = fmaf(f, u.z, o[v].z);
            o[v].w = fmaf(f, u.w, o[v].w);
          }
        }
      }
    }
    if (mine && sub == 0) {
      const bool none = saw_none(m, l);
      const float inv = none ? 0.f : 1.f / kDown / l;
      const int64_t at = out_row(p, d.x, d.y, d.z + row);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 128 + lane * 4 < D)
          *reinterpret_cast<uint2 *>(p.o + at * D + v * 128 + lane * 4) =
              make_uint2(pack_bf16x2(o[v].x * inv, o[v].y * inv), pack_bf16x2(o[v].z * inv, o[v].w * inv));
      if (lane == 0) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    if (per > 1) __syncthreads();  // the shared sums are free again
  }
}

// Sets a variant's shared-memory limit on its first call on a device.
constexpr int kMaxDevices = 64;
std::mutex g_mu;

// A launch of `ctas` CTAs in clusters of `cluster`.
template <typename S>
struct ClusterLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  ClusterLaunch(int64_t ctas, int cluster, cudaStream_t st) {
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};

// Once a device: the kernel's shared memory, and how many clusters of 2, 4 and 8
// CTAs the device holds at once (fewer than its SMs would give: a cluster does
// not reach over the device's groups of SMs).
template <typename S>
cudaError_t prepare(int device, const int **held) {
  static bool done[kMaxDevices];
  static int most[kMaxDevices][kClusterSizes];
  std::lock_guard<std::mutex> lock(g_mu);
  if (!done[device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_kv4_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < kClusterSizes; ++i) {
      ClusterLaunch<S> launch(2 << i, 2 << i, nullptr);
      if (cudaOccupancyMaxActiveClusters(&most[device][i], attn_kv4_kernel<S>, &launch.cfg) != cudaSuccess) {
        cudaGetLastError();
        most[device][i] = 0;
      }
    }
    done[device] = true;
  }
  *held = most[device];
  return cudaSuccess;
}

template <typename S>
int launch_kv4(Kv4Params &p, int device, int sms, cudaStream_t st) {
  const int *held = nullptr;  // clusters of 2, 4, 8 that the device holds at once
  cudaError_t e = prepare<S>(device, &held);
  if (e != cudaSuccess) return record_cuda_error(e);
  // What the lengths can be at most.  A request's query tokens fill no more row
  // tiles than each of them alone would, and one more than its rows / R.
  const int64_t by_rows = (int64_t)p.T * p.group / S::R + p.B, by_token = (int64_t)p.T * ((p.group + S::R - 1) / S::R);
  const int64_t tiles = ((int64_t)p.max_pages * S::P + S::TK - 1) / S::TK + 1;
  const int64_t items = (by_rows < by_token ? by_rows : by_token) * p.H;
  if (items > ((int64_t)1 << 40) / (tiles + S::START)) return ATTN_ERR_ARG;  // a piece's units are 32-bit
  // Few and short items have a cluster of CTAs each: the most (a power of two up
  // to 8) that leaves each warp a tile and all clusters resident at once (a second
  // wave costs more than it gives: 32 items of 2000 tokens 10.4 us in clusters of
  // 4, 28.0 of 8), and no second kernel.  Pieces would have each warp's tiles done
  // by all SMs, but cost about two tiles' time more.  Against pieces (D 128, 8 kv
  // heads): 1 request of 2000 tokens 10.1 us against 13.4, of 8000 13.4 against
  // 14.2, of 16000 (5 tiles a warp, 64 of 152 SMs) 16.9 against 16.7, 4 of 4000 12.9
  // against 16.4, 8 of 2000 12.6 against 16.4, 16 of 2000 15.4 against 19.5.  Above 8
  // tiles a warp, shorter requests' warps wait for the longest: 16 of 4000 and
  // less 20.9 against 18.0.
  p.cluster = 1;
  for (int i = 0; i < kClusterSizes && tiles > S::WARPS * p.cluster && items <= held[i]; ++i) p.cluster *= 2;
  const int64_t ctas = items * p.cluster, warps = S::WARPS * p.cluster;  // of all items, of one item
  if (items <= sms && tiles <= 8 * warps && tiles * (sms - ctas) <= 2 * sms * warps) {
    p.pieces = 0;
    const ClusterLaunch<S> launch(ctas, p.cluster, st);
    e = cudaLaunchKernelEx(&launch.cfg, attn_kv4_kernel<S>, (const Kv4Params)p);
    return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
  }
  p.cluster = 1;
  const int64_t most = (items * (tiles + S::START) + S::WARPS - 1) / S::WARPS;
  const int grid = (int)(most < sms ? most : sms);
  p.pieces = grid * S::WARPS;
  const size_t o_bytes = (size_t)p.pieces * 2 * S::R * S::D * 4, ml_bytes = (size_t)p.pieces * 2 * S::R * 8;
  uint8_t *ws = nullptr;
  if (scratch_alloc(reinterpret_cast<void **>(&ws), o_bytes + ml_bytes + (size_t)p.pieces * 32, st) != cudaSuccess ||
      !ws) {
    cudaGetLastError();
    return ATTN_ERR_NOMEM;
  }
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float2 *>(ws + o_bytes);
  p.ws_cut = reinterpret_cast<int4 *>(ws + o_bytes + ml_bytes);
  attn_kv4_kernel<S><<<(unsigned)grid, S::THREADS, S::SMEM, st>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_kv4_merge_kernel<S>, (const Kv4Params)p);
  }
  const cudaError_t f = cudaFreeAsync(ws, st);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

template <int P>
int launch_page_size(Kv4Params &p, int G, bool wide, int device, int sms, cudaStream_t st) {
  switch (G) {
    case 1:
      return wide ? launch_kv4<Shape<1, 16, P>>(p, device, sms, st) : launch_kv4<Shape<1, 8, P>>(p, device, sms, st);
    case 2:
      return wide ? launch_kv4<Shape<2, 16, P>>(p, device, sms, st) : launch_kv4<Shape<2, 8, P>>(p, device, sms, st);
    case 3:
      return launch_kv4<Shape<3, 8, P>>(p, device, sms, st);
    default:
      return launch_kv4<Shape<4, 8, P>>(p, device, sms, st);
  }
}

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace
}  // namespace attn

extern "C" {

int attn_fwd_kv4(const void *q, long long q_stride_t, long long q_stride_h, const int *cu, const int *lens,
                 const int *block_table, long long table_stride, int max_pages, const void *cache, int num_pages,
                 void *o, float *lse, int B, int T, int Hq, int Hkv, int D, int page_size, float scale, int causal,
                 attn_stream_t stream) {
  using namespace attn;
  if (B < 0 || B > kMaxRequests || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65535) return ATTN_ERR_ARG;
  if (D < 64 || D > ATTN_KV4_MAX_HEAD_DIM || D % 64 != 0) return ATTN_ERR_ARG;
  const int shift = kv4_page_shift(page_size);
  if (shift < 0 || num_pages < 0 || max_pages < 0 || (causal != 0 && causal != 1) || !isfinite(scale))
    return ATTN_ERR_ARG;
  if (max_pages > (0x7fffffff >> shift) - 4 || table_stride < max_pages) return ATTN_ERR_ARG;
  if ((int64_t)T * (Hq / Hkv) > 0x3fffffff || (int64_t)num_pages * page_size > 0x7fffffffLL) return ATTN_ERR_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!q || !o || !lse || !cu || !lens) return ATTN_ERR_ARG;
  if ((max_pages > 0 && !block_table) || (num_pages > 0 && !cache)) return ATTN_ERR_ARG;
  if (q_stride_t < 0 || q_stride_h < 0) return ATTN_ERR_ARG;
  if (off16(q) || off16(o) || off16(lse) || off16(cache) || q_stride_t % 8 || q_stride_h % 8) return ATTN_ERR_ALIGN;
  for (const int *a : {cu, lens, block_table})
    if (reinterpret_cast<uintptr_t>(a) & 3u) return ATTN_ERR_ALIGN;
  int device = 0, sms = 0;
  Kv4Params p{};
  const int rc = current_device(&device, &sms, &p.status);
  if (rc != ATTN_OK) return rc;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.qt = q_stride_t; p.qh = q_stride_h;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.cu = cu; p.lens = lens; p.table = block_table; p.table_stride = table_stride;
  p.cache = static_cast<const uint8_t *>(cache);
  p.num_pages = num_pages;
  p.max_pages = num_pages > 0 ? max_pages : 0;  // without pages no request holds a token
  p.B = B; p.T = T; p.H = Hkv; p.group = Hq / Hkv; p.shift = shift; p.causal = causal;
  p.scale_log2 = scale * kLog2e;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // 16 rows a tile where the requests have more than 64 on average: K and V are
  // then unpacked once for 16 rows.  With 16 heads on each of 4 kv heads: 112 rows
  // (7 tokens, D 64, 4 requests up to 16384) 35.7 us against 39.0 in tiles of 8,
  // 256 rows (D 64, 2 requests of 8192) 37.9 against 40.2, 112 rows at D 128 (51
  // requests of 4096) 240 against 274; 64 rows (D 128, 4 requests of 8192) 37.3
  // against 38.5, 16 rows (32 requests up to 4096) 24.1 against 23.4 (fewer warps
  // an SM).  At D > 128 the accumulators of 16 rows do not fit the registers.
  const bool wide = (int64_t)p.group * ((T + B - 1) / B) > 64;
  switch (page_size) {
    case 16: return launch_page_size<16>(p, D / 64, wide, device, sms, st);
    case 32: return launch_page_size<32>(p, D / 64, wide, device, sms, st);
    default: return launch_page_size<64>(p, D / 64, wide, device, sms, st);
  }
}

}  // extern "C"
