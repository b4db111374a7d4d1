// Attention over the 8-bit paged cache: O = softmax(scale Q K^T) V and its LSE for
// requests of any length with a few query tokens each.
//
// Both products run on the tensor cores' 8-bit form (tcgen05 kind::f8f6f4) on the codes
// as the cache holds them:
//     S^T[token, row] = K Q^T,      O^T[dim, row] = V^T P^T,
// K and V^T being the 128-row operand and the query rows (query token x head of the kv
// head's group) the columns, so that a decode step's few rows cost few columns.  Q and
// P are not e4m3 numbers; each is a sum of four (Q of three from 16 rows on, where the
// fourth is no longer free),
//     x = x0 + 2^-5 x1 + 2^-10 x2 + 2^-15 x3,   x0 = e4m3(x), x1 = e4m3(2^5 (x - x0)), ...
// (the remainder of a rounding to 4 bits is at most 2^-4 of the value, and exact in
// float32), in columns side by side whose products are added in float32.  With the
// largest value brought to 2^7 .. 2^8 three parts hold 12 bits and more of each value,
// four 16, down to 2^-19 and 2^-24: bfloat16's 8 bits of q exactly from 2^-12 of a
// row's largest value on, P to 2^-16 relative.  The columns are nearly free: a product
// of 128 rows and 32 of the sum takes 50 clocks with up to 64 columns, 56 with 96, 64
// with 128.
//
// Scales.  A token's score takes the block's scale of K as a factor, y = s c sk.  A row
// has two references, Y of its scores and E of V's scales: l = sum 2^(y - Y), and the
// block's scale of V is joined to the weight in the exponent, P = 2^((y - Y) + (log2 sv
// - E)), so that O = 2^E / l times the accumulators and a token's product with V counts
// by its size, whatever other tokens' scales are.  The first difference is exact where
// it matters and the second is one of small numbers, so scores of any size leave V's
// scale its place.  (With one reference of y + log2 sv, scores past 2^24 rounded the scale
// away: O was off by its power of two.)  Y is the largest score when it was set, and set
// again when one exceeds it by 60; E lets the largest exponent be 4 when it is set, and is set
// again when one exceeds 8 (then the accumulators are multiplied).  Exponents,
// references, l and accumulators are float32; what is rounded to fewer bits are the
// parts of Q and P above and O, once, to bfloat16.
//
// Hidden tokens have weight 0 in P; V's codes of tokens past the length are zeroed in
// shared memory first, so that nothing which a page holds there (0 times NaN) reaches a
// sum.
//
// Roles of a CTA (one per SM): two groups of four softmax warps, thread = token of the
// tile = dim of the output; one warp that finds the work and copies pages into a ring
// of stages of 128 tokens (pages are laid out as the products read them: plain bulk
// copies); one that issues the products; two or four that split Q.  The next tile's
// scores are computed while the softmax works on this one's.  Products and copies are
// issued by warps that stay together, one elected lane of them: a group of four
// products and a commit takes 156 clocks so, 306 issued by a lane in a branch (64
// requests of 1 to 8192 tokens 82 -> 69 us).  P is stored with the columns of a token
// together, so that a softmax thread writes 16 bytes at a time.
//
// Groups.  Up to 4 rows the groups have the tiles in turn, each with accumulators and
// references of its own, joined at the item's end; else they share the rows.  In turn
// against one group: 64 requests of 2730 tokens, D 64 49 -> 45 us, D 128 62.6 -> 62.4.
// Of 8 rows in turn D 64 58 -> 53 but ragged lengths, D 128, 71 -> 83; of 16 rows 80 ->
// 95 (a thread's 16 rows leave no registers): shared.
//
// Rows of a tile: the fewest of 4, 8, 16 and (up to 128 dims) 32 that hold a request's
// rows, or the most there are.  64 requests of 2730 tokens, 8 kv heads of 128, us for
// tiles of 4 / 8 / 16 / 32 rows:
//     4 rows 63 / 63 / 69 / 101;  8 rows 100 / 66 / 70 / 103;  12 rows 134 / 106 / 73 / 105;
//     28 rows 270 / 195 / 130 / 114;  64 rows 596 / 378 / 244 / 205.
// The rule goes by T / B, so requests of one call should have about as many query tokens:
// one of 64 among 63 idle slots takes 46 us (by itself 22), a chunk of 512 beside 63
// single tokens 192 (apart 107 and 61).
//
// Work split.  The tiles of all (request, kv head, row tile) items form one line, an
// item counting START more for its beginning and end, cut into equal pieces, one a CTA;
// lengths are read on the device.  START 1 / 2 / 3 / 4: 4 rows, 64 requests of 1 to
// 8192 tokens 83 / 66 / 67 / 68 us; START 2 / 3 / 4 / 6: 16 rows, 64 of 1 to 4096 55 /
// 53 / 54 / 57, of D 256 (16 requests) 19.6 / 19.5 / 18.6 / 18.4, 28 rows 94 / 85 / 78
// / 80.  A cut item's parts go to a workspace and are merged by a second kernel in the
// order of the tokens.  Few and short items have a cluster of CTAs each instead, merged
// through distributed shared memory (the rule and its figures: launch_kv8).
//
// Measured (graph, one GB300; HBM's time for the cache at 6.80 TB/s in brackets), 8 kv
// heads of 128, 32 heads: 256 requests of 8192 tokens 606 us (634; 7.1 TB/s), 64 of
// 2730 62 (53), 64 of 1 to 8192 in pages of 16 66 (54), one of 131072 46 (40).  What
// they are over is an item's beginning and end, the search for the piece (2.5 us), the
// first tile and the merge (4 us).  D 256 63 (53); 16 requests of up to 4096 with 4
// query tokens 18.6 (7): that latency alone.  D 64 45 (27): a tile's 16 KB arrive
// faster than one warp issues its copies and one its products (about 800 clocks a tile
// each). 64 of 2730 with 16 rows 74, with 28 115 (53): the softmax's chain (every weight
// split in four), of which an SM holds two warps a scheduler: they issue in 0.39 of the
// clocks.  One request of 129 tokens 6.2.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include <mutex>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv8.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int TK = 128;           // tokens of a tile: rows of the first product
constexpr int kItems = 4;         // items published ahead
constexpr int kMostParts = 64;    // pieces that one item is cut into, at most
constexpr int kMergeTiles = 4;    // what cutting items costs more than not doing so, in tiles' time
constexpr int kMaxStages = 12;
constexpr int kClusterSizes = 3;  // clusters of 2, 4 and 8 CTAs
constexpr int kMostCluster = 1 << kClusterSizes;
constexpr int kFew = 128;         // requests that one warp looks through
constexpr int kMaxRows = 32;
constexpr int kMaxRequests = ATTN_KV8_MAX_REQUESTS;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// References of a row that has seen no token: Y is no larger than any score, and E so low that any score sets both.
constexpr float kNoRef = -FLT_MAX, kNoExp = -1e30f;
constexpr float kBelow = 4.f;     // a new E lets the largest exponent of P be this much ...
constexpr float kAbove = 8.f;     // ... and holds until one exceeds this: weights stay below e4m3's 448
constexpr float kSumAbove = 60.f; // the same for Y, which is the largest score when it is set
constexpr float kStep = 32.f;     // 2^5, between the parts of Q and P
constexpr int kSmemMax = 232448;
// What a CTA waits at its end for its own copies and products, whatever the limit of the other waits is.
constexpr uint64_t kDrainNs = 2000000000ull;

struct Kv8Params {
  const __nv_bfloat16 *q;
  int64_t qt, qh;  // element strides of token and head
  __nv_bfloat16 *o;
  float *lse;
  const int *cu, *lens, *table;
  int64_t table_stride;
  const uint8_t *cache;
  int num_pages, max_pages, B, T, H, group, shift, causal;
  int cluster;       // CTAs that share an item, one item each; 0: pieces of the line
  float scale_log2;  // scale * log2 e
  float *ws_o;       // partial O of cut items: [CTAs][2][R][D]
  float4 *ws_ml;     // their references E and Y, and l: [CTAs][2][R]
  int4 *ws_cut;      // [CTAs][2]: the item that each CTA leaves unfinished
  int *status;
  uint64_t wait_limit_ns;
  int drop;          // test support: each CTA's second tile waits for bytes that do not come
};

// A variant: head dim and query rows of a tile.
template <int D_, int R_>
struct Shape {
  static constexpr int D = D_, R = R_;
  // Two groups of four softmax warps. With few rows they have the tiles in turn, with accumulators and references of
  // their own, else they share the rows.
  static constexpr bool TURNS = R <= 4;
  static constexpr int GROUPS = 2, RW = TURNS ? R : R / GROUPS;
  static constexpr int START = R >= 16 ? 4 : 2;  // an item's beginning and end cost about as much as this many tiles
  // Parts of Q and P.  Q's fourth is free where 16 columns are the least there can be.
  static constexpr int QP = R >= 16 ? 3 : 4, PP = 4;
  static constexpr int NQ = QP * R, NP = PP * R;  // columns: row r's part a is column (r / RW) parts RW + a RW + r % RW
  static constexpr int NH = (D + 127) / 128;      // 128-dim halves of the output
  static constexpr int K_BYTES = TK * D;
  static constexpr int V_STEP = kv8_block_bytes(D);  // a block of 16 tokens
  static constexpr int STAGE = K_BYTES + TK / kKv8Block * V_STEP;
  static constexpr int Q_BYTES = NQ * D, P_BYTES = NP * TK;
  // Q's buffers: one where it gives K and V a stage (16 requests of up to 4096, 4 query tokens, D 256: 18.6 us, two
  // buffers 20.4; 64 of 2000, 16 rows 38 and 46).
  static constexpr int QBUF = D >= 192 && R >= 16 ? 1 : 2;
  // Of 64 dims (and the second half of 192) the second product multiplies 128 rows
  // all the same: it reads up to 1 KB behind a block, whose results no one reads.
  // Q's and P's buffers lie there.
  static constexpr int FIXED = QBUF * Q_BYTES + 2 * P_BYTES;
  static constexpr int FIT = (kSmemMax - FIXED - 5120) / STAGE;
  static constexpr int STAGES = FIT > kMaxStages ? kMaxStages : FIT;
  static constexpr int OFF_Q = STAGES * STAGE, OFF_P = OFF_Q + QBUF * Q_BYTES;
  static constexpr int SMEM = OFF_P + 2 * P_BYTES;
  static constexpr int COLS = 2 * NQ + (TURNS ? 2 : 1) * NH * NP;   // of tensor memory: two tiles' scores, the output
  static constexpr uint32_t TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  // Warps: softmax, then one that loads, one that multiplies, and those that split Q: two, which leave 168 registers a
  // thread, but four for 16 rows of many dims. 2 / 4, us: 16 requests of 4 query tokens, D 256, up to 4096 20.2 / 18.6,
  // of 1365 16.0 / 15.5; 64 of 2730 with 16 rows, D 128 74.4 / 78.5, of 1 to 4096 54.1 / 55.9, 32 of 1000, D 64 24.9 /
  // 25.5; 28 rows 115 / 174 (spills).
  static constexpr int WARP_LOAD = GROUPS * 4, WARP_MMA = WARP_LOAD + 1, WARP_Q = WARP_LOAD + 2;
  static constexpr int Q_WARPS = R == 16 && D >= 192 ? 4 : 2;
  static constexpr int SOFTMAX = GROUPS * 128, AT_TILE = TURNS ? 128 : SOFTMAX, THREADS = (WARP_Q + Q_WARPS) * 32;
  static constexpr int LPR = D == 64 ? 4 : D == 128 ? 8 : 16;  // lanes that split a row, 16 dims each
  static_assert(STAGES >= 2 && COLS <= 512 && STAGE % 16 == 0 && OFF_Q % 128 == 0 && Q_BYTES + P_BYTES >= 1024, "");
  static_assert(NQ % 16 == 0 && NP % 16 == 0 && R <= kMaxRows, "");
};

// Shared-memory descriptor of an operand in core matrices of 8 x 16 bytes (no
// swizzle): `lbo` bytes from one to the next along the product, `sbo` from one to the
// next across it.  K, V and Q have 16 bytes of the product's axis together
// (K-major); P has 16 columns of a token together, as a softmax thread writes them.
__device__ __forceinline__ uint64_t core_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return (a | b) >> 31 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The tiles of a request whose cu descends (requests could then share query tokens
// and the line be longer than the host took it to be): no request has any work then.
constexpr int kDescends = 1 << 30;

// What a request's tiles look like, from the device arrays, with whatever they hold
// brought into range (reported once through the status word).
struct Request {
  int t0, nq, len;  // first query token, query tokens, cached tokens
  int tiles, rt;    // tiles of tokens (at least one), row tiles
  template <typename S>
  __device__ __forceinline__ int64_t units(int H) const {
    return (int64_t)H * rt * (tiles + S::START);
  }
};

template <typename S>
__device__ __forceinline__ Request load_request(const Kv8Params &p, int r) {
  Request q;
  const int a = p.cu[r], b = p.cu[r + 1], l = p.lens[r];
  const int room = p.max_pages << p.shift;
  q.t0 = min(max(a, 0), p.T);
  const int t1 = min(max(b, q.t0), p.T);
  q.nq = t1 - q.t0;
  q.len = min(max(l, 0), room);
  if (q.t0 != a || t1 != b || q.len != l) atomicCAS(p.status, 0, kStatusDevice);
  q.tiles = b < a ? kDescends : max(1, (q.len + TK - 1) / TK);
  q.rt = (int)(((int64_t)q.nq * p.group + S::R - 1) / S::R);
  return q;
}

// The part of an item that a CTA works on.
struct Item {
  int t0, nq, len;       // the request
  int h, row0, rows;     // kv head, query rows
  int tile0, tile1;      // tiles (none for a request without tokens)
  int slot;              // where the part goes: -1 the output, 0 or 1 the CTA's partials
  int more;              // 0: no item, the line is at its end
};

struct Shared {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], item_full[kItems],
      item_empty[kItems], drain;
  Item item[kItems];
  int64_t wsum[16];
  int wmax[16];
  int start[4];  // the piece's first unit: request (-1: none), head, row tile, offset in the item
  Request first;  // and that request
  uint32_t tmem;
  volatile int abort;
  // per buffer of Q and row: what turns its sums into log2 scores, the last token it sees, its place in the output
  float row_factor[2][kMaxRows];
  int row_limit[2][kMaxRows];
  int64_t row_out[2][kMaxRows];
  // [row][warp of the group]: the largest y, and the largest (y - that) + log2 sv
  __align__(16) float warp_y[kMaxRows][4], warp_z[kMaxRows][4];
  // [softmax warp][row of the group]: references E and Y, negated, what their last change takes the accumulators by, and
  // l by (at an item's end the warp's sum of l)
  __align__(16) float ref_e[8][kMaxRows / 2], ref_y[8][kMaxRows / 2], by_o[8][kMaxRows / 2], warp_l[8][kMaxRows / 2];
  float row_weight[kMaxRows];       // [group][row], or [row]: what turns accumulators into the output
  float4 group_ml[2][4];            // [group][row]: the references E and Y of groups that have the tiles in turn
  float4 part_ml[kMaxRows];                // a cluster's CTA: the references E and Y, and l, of its part's rows
};

__device__ __forceinline__ void raise_abort(Shared *sh, int *status) {
  sh->abort = 1;
  atomicCAS(status, 0, kStatusTimeout);
}

// A barrier of a group's softmax threads that tells whether any of them says yes.
template <int N = 128>
__device__ __forceinline__ bool any_softmax(int group, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"((uint32_t)yes), "n"(N)
      : "memory");
  return r != 0;
}

// The largest of the warp's values; NaN counts as none (all NaN: NaN).
__device__ __forceinline__ float warp_largest(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Two e4m3 codes as a pair of floats.
__device__ __forceinline__ uint64_t f2_of_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float lo, hi;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return f2_pack(lo, hi);
}
__device__ __forceinline__ uint64_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_low(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo;
}
__device__ __forceinline__ float f2_high(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return hi;
}

// The parts of a pair of values: part a of the lower one in the low byte of out[a], of the other in the next.
template <int PARTS>
__device__ __forceinline__ void split2(uint64_t x, uint32_t (&out)[PARTS]) {
#pragma unroll
  for (int a = 0; a < PARTS; ++a) {
    out[a] = pack_e4m3x2(f2_low(x), f2_high(x));
    if (a == PARTS - 1) break;
    x = f2_fma(f2_of_e4m3x2(out[a]), f2_both(-kStep), f2_mul(x, f2_both(kStep)));  // (exact)
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// PARTS columns RW apart, put together, of two rows.
template <int PARTS, int RW>
__device__ __forceinline__ uint64_t join(const uint32_t *s) {
  auto pair = [&](int a) { return f2_pack(__uint_as_float(s[a * RW]), __uint_as_float(s[a * RW + 1])); };
  uint64_t x = pair(PARTS - 1);
#pragma unroll
  for (int a = PARTS - 2; a >= 0; --a) x = f2_fma(x, f2_both(1.f / kStep), pair(a));
  return x;
}

// N columns of tensor memory from `addr` on.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N % 8 == 0, "");
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[8 * i]), "=r"(r[8 * i + 1]), "=r"(r[8 * i + 2]), "=r"(r[8 * i + 3]), "=r"(r[8 * i + 4]),
                   "=r"(r[8 * i + 5]), "=r"(r[8 * i + 6]), "=r"(r[8 * i + 7])
                 : "r"(addr + 8 * i));
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");  // no use of them may move before the wait
}

// References (E, Y) of a part of a row's tokens, as E beside another Y: what counts of
// it there.  Parts of a row are joined by their largest Y and, beside that, their largest E.
__device__ __forceinline__ float beside(float e, float y, float all_y) { return (y - all_y) + e; }
// What brings the part's accumulators to references (all_e, all_y).  (The scores' difference comes first: it is exact
// where it matters.)
__device__ __forceinline__ float part_factor(float e, float y, float all_e, float all_y) {
  return ex2_approx((y - all_y) + (e - all_e));
}

// Row q of a request's rows (query token x head of the group) in the output.
__device__ __forceinline__ int64_t out_row(const Kv8Params &p, int t0, int h, int q) {
  return (int64_t)(t0 + q / p.group) * ((int64_t)p.H * p.group) + (int64_t)h * p.group + q % p.group;
}

__device__ __forceinline__ void sync_finders(bool alone) {
  if (alone)
    __syncwarp();
  else
    __syncthreads();
}

// The CTA's piece [begin, end) of the line and where it begins (sh->start, sh->first), by one
// warp alone or by all threads: each has `per` consecutive requests, the first of them looked up by the caller.
template <typename S>
__device__ __forceinline__ void find_piece(const Kv8Params &p, Shared *sh, const Request &mine0, bool alone, int finder, int per,
                                           int64_t &begin, int64_t &end, int64_t &chunk) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = min(finder * per, p.B), r1 = min(r0 + per, p.B);
  int64_t mine = 0;
  int longest = 0;
  if (r0 < r1) {
    mine = mine0.units<S>(p.H);
    longest = mine0.tiles;
  }
#pragma unroll 4
  for (int r = r0 + 1; r < r1; ++r) {
    const Request q = load_request<S>(p, r);
    mine += q.units<S>(p.H);
    longest = max(longest, q.tiles);
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  int64_t before = 0, total = 0;
  if (alone) {
    total = __shfl_sync(0xffffffffu, sum, 31);
  } else {
    if (lane == 31) {
      sh->wsum[warp] = sum;
      sh->wmax[warp] = longest;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < S::THREADS / 32; ++w) {
      if (w < warp) before += sh->wsum[w];
      total += sh->wsum[w];
      longest = max(longest, sh->wmax[w]);
    }
  }
  if (longest >= kDescends) total = 0;
  // equal pieces, but none so small that an item would be cut into more than kMostParts
  chunk = max(max(divide(total + gridDim.x - 1, gridDim.x), (int64_t)(S::START + 1)),
              (int64_t)((longest + kMostParts - 1) / kMostParts));
  begin = min((int64_t)blockIdx.x * chunk, total);
  end = min(begin + chunk, total);
  int64_t a = before + sum - mine;
  if (begin < end && begin >= a && begin < a + mine) {
    for (int r = r0; r < r1; ++r) {
      const Request q = r == r0 ? mine0 : load_request<S>(p, r);
      const int64_t n = q.units<S>(p.H);
      if (begin < a + n) {
        const int each = q.tiles + S::START;
        const int64_t i = divide(begin - a, each);
        sh->start[0] = r;
        sh->start[1] = (int)divide(i, q.rt);
        sh->start[2] = (int)(i - (int64_t)sh->start[1] * q.rt);
        sh->start[3] = (int)(begin - a - i * each);
        sh->first = q;
        break;
      }
      a += n;
    }
  }
  sync_finders(alone);
}

// One cluster of CTAs for each item: the CTA's item and its share of the item's tiles (p.cluster of them), as a piece
// of one item.
template <typename S>
__device__ __forceinline__ void find_item(const Kv8Params &p, Shared *sh, const Request &mine0, bool alone, int finder, int per,
                                          int64_t &begin, int64_t &end, int64_t &chunk) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = min(finder * per, p.B), r1 = min(r0 + per, p.B);
  const int item = (int)blockIdx.x / p.cluster, rank = (int)blockIdx.x - item * p.cluster;
  int64_t mine = r0 < r1 ? (int64_t)p.H * mine0.rt : 0;
  bool descends = r0 < r1 && mine0.tiles >= kDescends;
#pragma unroll 4
  for (int r = r0 + 1; r < r1; ++r) {
    const Request q = load_request<S>(p, r);
    mine += (int64_t)p.H * q.rt;
    descends |= q.tiles >= kDescends;
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  int64_t a = sum - mine;
  if (finder == 0) sh->start[0] = -1;
  if (!alone && lane == 31) sh->wsum[warp] = sum;
  const bool none = alone ? __any_sync(0xffffffffu, descends) : __syncthreads_or(descends);
  if (alone) {
    __syncwarp();
  } else {
#pragma unroll
    for (int w = 0; w < S::THREADS / 32; ++w)
      if (w < warp) a += sh->wsum[w];
  }
  if (!none && item >= a && item < a + mine) {
    for (int r = r0; r < r1; ++r) {
      const Request q = r == r0 ? mine0 : load_request<S>(p, r);
      const int64_t n = (int64_t)p.H * q.rt;
      if (item < a + n) {
        const int i = (int)(item - a);
        sh->start[0] = r;
        sh->start[1] = i / q.rt;
        sh->start[2] = i % q.rt;
        sh->first = q;
        break;
      }
      a += n;
    }
  }
  sync_finders(alone);
  const int n = sh->first.tiles, each = (n + p.cluster - 1) / p.cluster;
  begin = min(rank * each, n);
  end = sh->start[0] < 0 ? begin : min((int)begin + each, n);
  chunk = 1;
}

// The first request from r on that has query tokens, or B: a look at 32, then a
// search, which holds as cu ascends.  Whole warp.
__device__ __forceinline__ int next_active(const Kv8Params &p, int r) {
  const int lane = threadIdx.x & 31;
  bool has = r + lane < p.B && p.cu[r + lane + 1] > p.cu[r + lane];
  uint32_t who = __ballot_sync(0xffffffffu, has);
  if (who) return r + __ffs(who) - 1;
  int lo = r + 32, hi = p.B;  // the answer is in [lo, hi]
  if (lo >= hi) return p.B;
  const int from = p.cu[lo];
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    who = __ballot_sync(0xffffffffu, at < hi && p.cu[at + 1] > from);
    if (who) {  // the first lane that says yes: the answer is behind the lane before it
      const int f = __ffs(who) - 1;
      hi = min(lo + f * step, hi);
      lo = f ? lo + (f - 1) * step + 1 : lo;
    } else {
      lo = min(lo + ((hi - lo - 1) / step) * step + 1, hi);
    }
  }
  return lo;
}

// V's codes past the length, up to the end of the last 32 tokens, cleared by the softmax threads.
template <typename S>
__device__ __forceinline__ void clear_tail(uint8_t *v, int n, int tid) {
#pragma unroll 1
  for (int i = tid; i < 2 * S::D; i += S::AT_TILE) {
    const int block = (n >> 5) * 2 + i / S::D, keep = n - block * kKv8Block;  // tokens of it that count
    if (keep >= kKv8Block) continue;
    uint4 *c = reinterpret_cast<uint4 *>(v + block * S::V_STEP) + i % S::D;
    uint32_t w[4] = {0, 0, 0, 0};
    if (keep > 0) {
      const uint4 x = *c;
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = min(max(keep - 4 * j, 0), 4);
        w[j] = k == 4 ? w[j] : w[j] & ((1u << (8 * k)) - 1);
      }
    }
    *c = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1) attn_kv8_kernel(const Kv8Params p) {
  static_assert(S::SMEM + sizeof(Shared) <= kSmemMax, "");
  constexpr int D = S::D, RW = S::RW, NQ = S::NQ, NP = S::NP, QP = S::QP, PP = S::PP, NH = S::NH, STAGES = S::STAGES;
  constexpr bool TURNS = S::TURNS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared shared;
  Shared *const sh = &shared;
  volatile int *const abortf = &sh->abort;
  const uint64_t limit = p.wait_limit_ns;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The thread's first request, asked for before anything else.  Up to kFew requests the loading warp finds its work by
  // itself, else all threads do.
  const bool few = p.B <= kFew;
  const int finders = few ? 32 : S::THREADS, finder = few ? (warp == S::WARP_LOAD ? lane : 32) : tid;
  const int per_finder = (p.B + finders - 1) / finders, first_request = finder * per_finder;
  Request mine{0, 0, 0, 1, 0};
  if (finder < finders && first_request < p.B) mine = load_request<S>(p, first_request);
  if (warp == 0) {
    if (lane < STAGES) {
      mbar_init(&sh->kv_full[lane], 1);
      mbar_init(&sh->kv_empty[lane], 1);
    } else if (lane >= 16 && lane < 18) {
      const int i = lane - 16;
      mbar_init(&sh->q_full[i], 32 * S::Q_WARPS);
      mbar_init(&sh->q_empty[i], 1 + 4 * S::GROUPS);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], S::AT_TILE);
      mbar_init(&sh->pv_done[i], 1);
    } else if (lane >= 20 && lane < 20 + kItems) {
      mbar_init(&sh->item_full[lane - 20], 1);
      mbar_init(&sh->item_empty[lane - 20], 1 + S::Q_WARPS + 4 * S::GROUPS);
    } else if (lane == 31) {
      mbar_init(&sh->drain, 1);
      sh->abort = 0;
    }
    fence_mbar_init();
  }
  if (warp == S::WARP_MMA) {
    tmem_alloc(&sh->tmem, S::TMEM);
    tmem_relinquish();
  }
  int64_t begin = 0, end = 0, chunk = 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!few || warp == S::WARP_LOAD) {
    if (p.cluster > 0)
      find_item<S>(p, sh, mine, few, finder, per_finder, begin, end, chunk);
    else
      find_piece<S>(p, sh, mine, few, finder, per_finder, begin, end, chunk);
  }
  const uint32_t tmem = sh->tmem, t_o = tmem + 2 * NQ;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // a wait of a whole warp, whose lanes go on together also where it gives up
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity) || mbar_wait(bar, parity, abortf, limit)) != 0;
  };
  if (warp == S::WARP_LOAD) {
    // ---------------- finds the items and copies their pages
    const uint32_t lead = elect_lead();
    int stage = 0, sphase = 0, slot = 0, iphase = 0;
    int4 cut = make_int4(0, 0, 0, 0);
    int cut_last = 0;
    bool ok = true;
    int64_t left = end - begin;
    int r = sh->start[0], h = sh->start[1], rt = sh->start[2], off = sh->start[3];
    const int per_tile = TK >> p.shift, P = 1 << p.shift;
    int64_t at = begin;
    Request q = sh->first;
    const int *row = p.table + (int64_t)max(r, 0) * p.table_stride;
    // A page a lane, from tile t's first on, 0 behind the last: a tile's time is less than the table's answer takes, so
    // 32 pages are asked for at once, the next 32 while these are copied.
    auto look_up = [&](int t) {
      int page = (int64_t)t * per_tile + lane < (q.len + P - 1) >> p.shift ? row[t * per_tile + lane] : 0;
      return page;
    };
    const int ahead = 32 / per_tile;  // tiles
    int copied = 0;                  // tiles
    int first = 0, first_tile = -1;  // the heads of a request begin with the same pages
    // Publishes an item and copies its tiles.
    auto take_item = [&](int tile0, int tile1, int to_slot) {
      if (tile0 != first_tile) {
        first = look_up(tile0);
        first_tile = tile0;
      }
      if (!wait_warp(&sh->item_empty[slot], iphase ^ 1)) return false;
      Item it;
      it.t0 = q.t0; it.nq = q.nq; it.len = q.len;
      it.h = h; it.row0 = rt * S::R; it.rows = (int)min((int64_t)q.nq * p.group - rt * S::R, (int64_t)S::R);
      it.tile0 = q.len > 0 ? tile0 : 0;
      it.tile1 = q.len > 0 ? tile1 : 0;
      it.slot = to_slot;
      it.more = 1;
      if (lane == 0) {
        sh->item[slot] = it;
        mbar_arrive(&sh->item_full[slot]);
      }
      if (++slot == kItems) slot = 0, iphase ^= 1;
      if (to_slot == 1) cut = make_int4(it.t0, h, it.row0, it.rows);
      int next = first, page = 0, from_lane = 32;
      for (int t = it.tile0; t < it.tile1; ++t, from_lane += per_tile) {
        if (from_lane == 32) {
          from_lane = 0;
          page = next;
          if (t + ahead < it.tile1) next = look_up(t + ahead);
          if ((unsigned)page >= (unsigned)p.num_pages) {
            atomicCAS(p.status, 0, kStatusDevice);
            page = 0;
          }
        }
        const int n = min(q.len - t * TK, TK);
        if (!wait_warp(&sh->kv_empty[stage], sphase ^ 1)) return false;
        const uint32_t to = smem_u32(smem) + stage * S::STAGE, bar = smem_u32(&sh->kv_full[stage]);
        // (`drop` waits for bytes that do not come. To skip a copy instead would make the copies conditional, which
        // took 20 of 70 us from pages of 16 tokens)
        mbar_expect_lead(lead, bar, (uint32_t)((n + 7) / 8 * 8 * D + (n + 15) / 16 * S::V_STEP + (p.drop && copied == 1 ? 16 : 0)));
        ++copied;
        // page by page, the warp together
        const int pages = (n + P - 1) >> p.shift;
        for (int i = 0; i < pages; ++i) {
          const int here = min(n - i * P, P);  // tokens of the page
          const uint8_t *from = p.cache + ((int64_t)__shfl_sync(0xffffffffu, page, from_lane + i) * p.H + h) * kv8_page_bytes(D, P);
          bulk_load_lead(lead, to + i * P * D, from, (uint32_t)((here + 7) / 8 * 8 * D), bar);
          bulk_load_lead(lead, to + S::K_BYTES + i * (P / kKv8Block) * S::V_STEP, from + P * D,
                         (uint32_t)((here + 15) / 16 * S::V_STEP), bar);
        }
        if (++stage == STAGES) stage = 0, sphase ^= 1;
      }
      return true;
    };
    if (p.cluster > 0) {
      // one item; its parts are merged in shared memory where several CTAs have it
      if (r >= 0) ok = take_item((int)begin, (int)end, p.cluster > 1 ? 2 : -1);
    } else {
      while (ok && left > 0 && r < p.B) {
        for (; ok && left > 0 && h < p.H; ++h, rt = 0)
          for (; ok && left > 0 && rt < q.rt; ++rt, off = 0) {
            const int each = q.tiles + S::START, take = (int)min((int64_t)(each - off), left);
            const int tile0 = max(off - S::START, 0), tile1 = max(off + take - S::START, 0);
            const int64_t item_end = at + each - off;
            left -= take;
            at += take;
            if (tile0 == tile1) continue;  // only the beginning's units: the next CTA has the tiles
            const bool whole = tile0 == 0 && tile1 == q.tiles;
            if (!whole && tile0 == 0) cut_last = (int)divide(item_end - 1, chunk);
            ok = take_item(tile0, tile1, whole ? -1 : tile0 == 0 ? 1 : 0);
          }
        if (left > 0 && h >= p.H) {
          h = 0;
          r = next_active(p, r + 1);
          if (r >= p.B) break;
          q = load_request<S>(p, r);
          row = p.table + (int64_t)r * p.table_stride;
          first_tile = -1;
        }
      }
    }
    // the end of the line
    if (ok && wait_warp(&sh->item_empty[slot], iphase ^ 1)) {
      if (lane == 0) {
        sh->item[slot].more = 0;
        mbar_arrive(&sh->item_full[slot]);
      }
    } else {
      ok = false;
    }
    if (!ok) raise_abort(sh, p.status);
    if (lane == 0 && p.cluster == 0) {
      p.ws_cut[blockIdx.x * 2] = cut;
      p.ws_cut[blockIdx.x * 2 + 1] = make_int4(cut_last, 0, 0, 0);
    }
    __syncwarp();
    // No copy may be in flight when the CTA leaves, whatever the other roles did: the phase that the last copy into
    // each stage completes (stages behind `stage` were last filled a turn ago, or never).
    for (int i = 0; i < STAGES; ++i) mbar_wait_drain(&sh->kv_full[i], i < stage ? sphase : sphase ^ 1, kDrainNs);
  } else if (warp == S::WARP_MMA) {
    // ---------------- products (the warp stays together; one lane issues)
    const uint32_t lead = elect_lead(), base = smem_u32(smem);
    constexpr uint32_t idesc_q = idesc_e4m3(128, NQ), idesc_p = idesc_e4m3(128, NP) | 1u << 16;  // P: columns contiguous
    int stage = 0, sphase = 0, slot = 0, iphase = 0, qb = 0, qphase = 0;
    uint32_t n_tile = 0;  // tiles so far: buffer n & 1, its phase n >> 1
    bool ok = true;
    auto all = [](bool yes) { return __all_sync(0xffffffffu, yes) != 0; };  // (of a test that does not wait)
    // the second product of a tile: `tokens` of it count
    auto second = [&](uint32_t tile, int st, int tokens, uint32_t more) {
      const uint32_t b = tile & 1;
      if (!wait_warp(&sh->p_full[b], (tile >> 1) & 1)) return false;
      tc_fence_after();
      const uint64_t v = core_desc(base + st * S::STAGE + S::K_BYTES, S::V_STEP, 128);
      const uint64_t pt = core_desc(base + S::OFF_P + b * S::P_BYTES, 128, TK * 16);
      const uint32_t acc = t_o + (TURNS ? b * (NH * NP) : 0);
      auto step = [&](int ks) {
#pragma unroll
        for (int hf = 0; hf < NH; ++hf)
          mma_f8_ss_lead(lead, acc + hf * NP, v + (ks * 2 * S::V_STEP + hf * 2048) / 16, pt + ks * 32, idesc_p, ks > 0 ? 1 : more);
      };
      if (tokens > TK - 32) {  // (no branch between them)
#pragma unroll
        for (int ks = 0; ks < TK / 32; ++ks) step(ks);
      } else {
#pragma unroll 1
        for (int ks = 0; ks * 32 < tokens; ++ks) step(ks);
      }
      mma_commit_lead(lead, &sh->kv_empty[st]);
      mma_commit_lead(lead, &sh->pv_done[b]);
      return true;
    };
    // The tile whose second product is still to come.  A tile's first product goes ahead of it, so that the next scores
    // are there when the softmax asks for them; across items only where the next one's operands are there already.
    bool pending = false;
    int p_stage = 0, p_tokens = 0;
    uint32_t p_more = 0;
    auto flush = [&]() {
      if (pending) ok = second(n_tile - 1, p_stage, p_tokens, p_more);
      pending = false;
    };
    while (ok) {
      if (pending && !(all(mbar_test_wait(&sh->item_full[slot], iphase)) && all(mbar_test_wait(&sh->q_full[qb], qphase)) &&
                       all(mbar_test_wait(&sh->kv_full[stage], sphase))))
        flush();
      if (!ok || !wait_warp(&sh->item_full[slot], iphase)) {
        ok = false;
        break;
      }
      auto told = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // (uniform to the compiler)
      const int tile0 = told(sh->item[slot].tile0), tile1 = told(sh->item[slot].tile1);
      const int len = told(sh->item[slot].len), more = told(sh->item[slot].more);
      if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
      if (++slot == kItems) slot = 0, iphase ^= 1;
      if (!more || tile0 == tile1) flush();
      if (!more) break;
      if (!ok || !wait_warp(&sh->q_full[qb], qphase)) {
        ok = false;
        break;
      }
      const uint64_t q = core_desc(base + S::OFF_Q + qb * S::Q_BYTES, NQ * 16, 128);
      for (int t = tile0; ok && t < tile1; ++t) {
        if (!wait_warp(&sh->kv_full[stage], sphase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t b = n_tile & 1;
        const uint64_t k = core_desc(base + stage * S::STAGE, 128, 8 * D);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
          mma_f8_ss_lead(lead, tmem + b * NQ, k + ks * 16, q + ks * 2 * NQ, idesc_q, ks > 0);
        mma_commit_lead(lead, &sh->s_full[b]);
        if (t == tile1 - 1) mma_commit_lead(lead, &sh->q_empty[qb]);
        flush();
        ++n_tile;
        pending = ok;
        p_stage = stage;
        p_tokens = min(len - t * TK, TK);
        p_more = t - tile0 >= (TURNS ? 2 : 1);
        if (++stage == STAGES) stage = 0, sphase ^= 1;
      }
      if (tile0 == tile1) mma_commit_lead(lead, &sh->q_empty[qb]);
      if (++qb == S::QBUF) qb = 0, qphase ^= 1;
    }
    if (!ok) raise_abort(sh, p.status);
    mma_commit_lead(lead, &sh->drain);  // no product may be in flight when the CTA leaves
    mbar_wait_drain(&sh->drain, 0, kDrainNs);
    __syncwarp();
  } else if (warp >= S::WARP_Q) {
    // ---------------- Q's rows, split: 16 dims of a row a lane
    constexpr int LPR = S::LPR, ROWS = 32 / LPR;  // lanes of a row, rows of a warp
    const int chunk16 = lane % LPR;
    int slot = 0, iphase = 0, qb = 0, qphase = 0;
    bool ok = true;
    while (ok) {
      if (!wait_warp(&sh->item_full[slot], iphase)) {
        ok = false;
        break;
      }
      const Item it = sh->item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
      if (++slot == kItems) slot = 0, iphase ^= 1;
      if (!it.more) break;
      const uint32_t to = smem_u32(smem) + S::OFF_Q + qb * S::Q_BYTES;
      // all of the warp's rows are asked for before the first is split
      constexpr int ROUNDS = (S::R + S::Q_WARPS * ROWS - 1) / (S::Q_WARPS * ROWS);
      uint32_t w[ROUNDS][8];
#pragma unroll
      for (int k = 0; k < ROUNDS; ++k) {
        const int row = (warp - S::WARP_Q + k * S::Q_WARPS) * ROWS + lane / LPR;
#pragma unroll
        for (int x = 0; x < 8; ++x) w[k][x] = 0;
        if (row < it.rows && chunk16 < D / 16) {
          const int qr = it.row0 + row, i = qr / p.group, j = it.h * p.group + qr - i * p.group;
          const uint4 *from = reinterpret_cast<const uint4 *>(p.q + (int64_t)(it.t0 + i) * p.qt + (int64_t)j * p.qh) + chunk16 * 2;
          const uint4 x = from[0], y = from[1];
          w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
          w[k][4] = y.x; w[k][5] = y.y; w[k][6] = y.z; w[k][7] = y.w;
        }
      }
      if (!wait_warp(&sh->q_empty[qb], qphase ^ 1)) {
        ok = false;
        break;
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < ROUNDS; ++k) {
        const int row = (warp - S::WARP_Q + k * S::Q_WARPS) * ROWS + lane / LPR;
        const bool is_row = row < S::R, in = row < it.rows;
        uint32_t m = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x) m = __vmaxu2(m, w[k][x] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool bad = m >= 0x7f80u;  // an infinity or a NaN: the row's scores are NaN
        // the row's largest value to 2^7 .. 2^8, by two factors that float32 holds
        const int e = 134 - max((int)(m >> 7), 1), e1 = e / 2, e2 = e - e1;
        const uint64_t f1 = f2_both(__uint_as_float((uint32_t)(e1 + 127) << 23));
        const uint64_t f2 = f2_both(__uint_as_float((uint32_t)(e2 + 127) << 23));
        auto scaled = [&](uint32_t x) {
          return f2_mul(f2_mul(f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), f1), f2);
        };
        uint32_t part[QP][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t lo[QP], hi[QP];
          const uint32_t u = bad ? 0 : w[k][2 * x], v = bad ? 0 : w[k][2 * x + 1];
          split2<QP>(scaled(u), lo);
          split2<QP>(scaled(v), hi);
#pragma unroll
          for (int a = 0; a < QP; ++a) part[a][x] = lo[a] | hi[a] << 16;
        }
        if (is_row && chunk16 < D / 16) {
#pragma unroll
          for (int a = 0; a < QP; ++a) {
            const int n = row / RW * (QP * RW) + a * RW + row % RW;  // the part's column
            st_shared_v4(to + chunk16 * (NQ * 16) + n * 16, part[a][0], part[a][1], part[a][2], part[a][3]);
          }
        }
        if (is_row && chunk16 == 0) {
          const int qr = it.row0 + (in ? row : 0), i = qr / p.group, j = it.h * p.group + qr - i * p.group;
          sh->row_factor[qb][row] = bad ? NAN : ldexpf(p.scale_log2, -e);
          sh->row_limit[qb][row] = p.causal && in ? it.len - it.nq + i : it.len - 1;
          sh->row_out[qb][row] = (int64_t)(it.t0 + i) * ((int64_t)p.H * p.group) + j;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh->q_full[qb]);
      if (++qb == S::QBUF) qb = 0, qphase ^= 1;
    }
    if (!ok) raise_abort(sh, p.status);
  } else {
    // ---------------- softmax, and the items' ends
    const int group = warp >> 2, key = tid & 127, wq = warp & 3;  // key: the token of the tile, and the dim of the output
    int stage = 0, sphase = 0, slot = 0, iphase = 0, qb = 0, qphase = 0;
    uint32_t n_tile = 0;
    bool fail = false;
    const uint32_t t_lanes = (uint32_t)(wq * 32) << 16;
    // the group's first row, and its columns of scores and accumulators
    const int row0 = TURNS ? 0 : group * RW;
    const uint32_t t_s = tmem + t_lanes + row0 * QP, t_acc = t_o + t_lanes + (TURNS ? group * (NH * NP) : row0 * PP);
    // groups that have the tiles in turn begin and end an item together
    auto any_at_end = [&](bool yes) { return TURNS ? any_softmax<256>(2, yes) : any_softmax(group, yes); };
    while (true) {
      fail = !mbar_wait(&sh->item_full[slot], iphase, abortf, limit);
      const Item it = sh->item[slot];
      // (an item that did not come has no work; the next vote ends the loop)
      if (!fail && it.more) fail = !mbar_wait(&sh->q_full[qb], qphase, abortf, limit);
      if (any_at_end(fail || !it.more)) break;
      if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
      if (++slot == kItems) slot = 0, iphase ^= 1;
      // pairs of rows: references E and Y (negated), l, and what turns sums into scores
      constexpr int RP = RW / 2;
      uint64_t eref[RP], yref[RP], l[RP], factor[RP];
      if (lane < RW) {
        sh->ref_e[warp][lane] = -kNoExp;
        sh->ref_y[warp][lane] = -kNoRef;
      }
#pragma unroll
      for (int i = 0; i < RP; ++i) {
        eref[i] = f2_both(-kNoExp);
        yref[i] = f2_both(-kNoRef);
        l[i] = f2_both(0.f);
        factor[i] = f2_pack(sh->row_factor[qb][row0 + 2 * i], sh->row_factor[qb][row0 + 2 * i + 1]);
      }
      const int *const limits = sh->row_limit[qb] + row0;
      const int first_limit = sh->row_limit[qb][0];  // the first row sees the fewest tokens
      bool some = false;  // the group has a tile of the item
      for (int t = it.tile0; t < it.tile1; ++t, ++n_tile) {
        const uint32_t b = n_tile & 1;
        if (TURNS && (int)b != group) {
          if (++stage == STAGES) stage = 0, sphase ^= 1;
          continue;
        }
        fail = fail || !mbar_wait(&sh->kv_full[stage], sphase, abortf, limit) ||
               !mbar_wait(&sh->s_full[b], (n_tile >> 1) & 1, abortf, limit);
        tc_fence_after();
        const uint8_t *const vs = smem + stage * S::STAGE + S::K_BYTES;
        const int n = min(it.len - t * TK, TK);
        const Kv8Tail tail = *reinterpret_cast<const Kv8Tail *>(vs + (key >> 4) * S::V_STEP + D * kKv8Block);
        const float sk = tail.kbad >> (key & 15) & 1 ? NAN : __uint_as_float(tail.sk);
        // (what a page holds past the length is neither a scale nor a mark)
        const float lv = key < n ? (float)((int)(tail.sv >> 23) - 127) : 0.f;
        const bool nan_v = key < n && tail.vbad >> (key & 15) & 1, some_nan = __any_sync(0xffffffffu, nan_v);
        uint64_t y[RP];
        {
          uint32_t s[QP * RW];
          tmem_ld<QP * RW>(t_s + b * NQ, s);
#pragma unroll
          for (int i = 0; i < RP; ++i)  // (factor sk by itself may pass float32 where the scores do not)
            y[i] = f2_mul(f2_mul(join<QP, RW>(s + 2 * i), factor[i]), f2_both(sk));
        }
        if (first_limit - t * TK < TK - 1) {  // some row does not see all of the tile
#pragma unroll
          for (int i = 0; i < RP; ++i)
            y[i] = f2_pack(key > limits[2 * i] - t * TK ? -INFINITY : f2_low(y[i]),
                           key > limits[2 * i + 1] - t * TK ? -INFINITY : f2_high(y[i]));
        }
        // y - Y and (y - Y) + (lv - E): exponents of the weights in l and in P
        uint64_t tz[RP], ty[RP];
        auto exponents = [&]() {
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            ty[i] = f2_add(y[i], yref[i]);
            tz[i] = f2_add(ty[i], f2_add(f2_both(lv), eref[i]));
          }
        };
        exponents();
        float most_z = -INFINITY, most_y = -INFINITY;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          most_z = max3f(most_z, f2_low(tz[i]), f2_high(tz[i]));
          most_y = max3f(most_y, f2_low(ty[i]), f2_high(ty[i]));
        }
        if (any_softmax(group, fail || most_z > kAbove || most_y > kSumAbove)) {
          // New references, from the tile's scores: a row a lane, each warp for itself (unrolled over the rows it is long
          // code that is run a few times an item: 16 requests of 4 query tokens, D 256, 500 tokens 10.8 -> 11.5 us)
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            const float w0 = warp_largest(f2_low(y[i])), w1 = warp_largest(f2_high(y[i]));
            const uint64_t z = f2_add(f2_add(y[i], f2_pack(-w0, -w1)), f2_both(lv));
            const float z0 = warp_largest(f2_low(z)), z1 = warp_largest(f2_high(z));
            if (lane == 0) {
              sh->warp_y[group * RW + 2 * i][wq] = w0;
              sh->warp_y[group * RW + 2 * i + 1][wq] = w1;
              sh->warp_z[group * RW + 2 * i][wq] = z0;
              sh->warp_z[group * RW + 2 * i + 1][wq] = z1;
            }
          }
          if (any_softmax(group, fail)) {
            fail = true;
            break;
          }
          if (lane < RW) {  // (fmaxf leaves out the NaN of a warp that has no score)
            const float4 w = *reinterpret_cast<const float4 *>(sh->warp_y[group * RW + lane]);
            const float4 z = *reinterpret_cast<const float4 *>(sh->warp_z[group * RW + lane]);
            const float e = -sh->ref_e[warp][lane], s = -sh->ref_y[warp][lane];
            const float y_now = fmaxf(s, fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)));
            const float z_now = fmaxf(fmaxf(beside(z.x, w.x, y_now), beside(z.y, w.y, y_now)),
                                      fmaxf(beside(z.z, w.z, y_now), beside(z.w, w.w, y_now)));
            const float e_now = fmaxf(beside(e, s, y_now), z_now - kBelow);
            sh->ref_e[warp][lane] = -e_now;
            sh->ref_y[warp][lane] = -y_now;
            sh->by_o[warp][lane] = part_factor(e, s, e_now, y_now);
            sh->warp_l[warp][lane] = ex2_approx(s - y_now);
          }
          __syncwarp();
          auto rows2 = [&](const float(&x)[8][kMaxRows / 2], int i) { return *reinterpret_cast<const uint64_t *>(&x[warp][2 * i]); };
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            eref[i] = rows2(sh->ref_e, i);
            yref[i] = rows2(sh->ref_y, i);
            l[i] = f2_mul(l[i], rows2(sh->warp_l, i));
          }
          exponents();
          if (some) {
            const uint32_t last = n_tile - (TURNS ? 2 : 1);  // its last tile
            fail = !mbar_wait(&sh->pv_done[last & 1], (last >> 1) & 1, abortf, limit);  // (told at the next vote)
            tc_fence_after();
#pragma unroll 1
            for (int hf = 0; hf < NH; ++hf)
#pragma unroll
              for (int c0 = 0; c0 < PP * RW; c0 += 16) {
                uint32_t o[16];
                tmem_ld<16>(t_acc + hf * NP + c0, o);
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * sh->by_o[warp][(c0 + c) % RW]);
                tmem_st16(t_acc + hf * NP + c0, o);
              }
            tmem_wait_st();
          }
        }
        // the thread's columns, 16 bytes at a time
        uint4 *const pt = reinterpret_cast<uint4 *>(smem + S::OFF_P + b * S::P_BYTES) + row0 * PP / 16 * TK + key;
        uint32_t cols[PP * RW / 4];
#pragma unroll
        for (int i = 0; i < RP; i += 2) {
          uint32_t part[2][PP];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x0 = ex2_approx(f2_low(tz[i + k])), x1 = ex2_approx(f2_high(tz[i + k]));
            if (some_nan) {  // a marked token's V is NaN to the rows that see it
              if (nan_v && f2_low(y[i + k]) != -INFINITY) x0 = NAN;
              if (nan_v && f2_high(y[i + k]) != -INFINITY) x1 = NAN;
            }
            split2<PP>(f2_pack(x0, x1), part[k]);
          }
#pragma unroll
          for (int a = 0; a < PP; ++a) cols[(a * RW + 2 * i) / 4] = part[0][a] | part[1][a] << 16;
        }
#pragma unroll
        for (int i = 0; i < PP * RW / 16; ++i)
          pt[i * TK] = make_uint4(cols[4 * i], cols[4 * i + 1], cols[4 * i + 2], cols[4 * i + 3]);
#pragma unroll
        for (int i = 0; i < RP; ++i) l[i] = f2_add(l[i], f2_pack(ex2_approx(f2_low(ty[i])), ex2_approx(f2_high(ty[i]))));
        if (n & 31) clear_tail<S>(smem + stage * S::STAGE + S::K_BYTES, n, TURNS ? key : tid);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sh->p_full[b]);
        some = true;
        if (++stage == STAGES) stage = 0, sphase ^= 1;
      }
      // The item's end: l over the threads, then a dim a thread.  A warp's sums by halving: lanes that differ in bit 4
      // take a half of the rows each, and so on; then lanes of one row are summed.
      int row = 0;
      float ls[RW];
#pragma unroll
      for (int i = 0; i < RP; ++i) f2_unpack(l[i], ls[2 * i], ls[2 * i + 1]);
#pragma unroll
      for (int half = RW / 2, o = 16; half >= 1; half >>= 1, o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int r = 0; r < half; ++r) {
          const float mine = upper ? ls[r + half] : ls[r], theirs = upper ? ls[r] : ls[r + half];
          ls[r] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
        }
        row += upper ? half : 0;
      }
#pragma unroll
      for (int o = 16 / RW; o >= 1; o >>= 1) ls[0] += __shfl_xor_sync(0xffffffffu, ls[0], o);
      if (lane % (32 / RW) == 0) sh->warp_l[warp][row] = ls[0];
      if (TURNS && key < RW)
        sh->group_ml[group][key] = make_float4(-sh->ref_e[warp][lane], -sh->ref_y[warp][lane], some ? 1.f : 0.f, 0.f);
      if (some && !fail) {
        // (one barrier for each of two tiles in turn: when the last tile's scores were there, the product of the tile
        // three before it was done, that of the one before it perhaps not, so a single barrier could be two phases
        // back)
        const uint32_t last = n_tile - 1 - (TURNS && ((n_tile - 1) & 1) != (uint32_t)group ? 1 : 0);
        fail = !mbar_wait(&sh->pv_done[last & 1], (last >> 1) & 1, abortf, limit);
        tc_fence_after();
      }
      if (any_at_end(fail)) {
        fail = true;
        break;
      }
      auto sum_of = [&](int g, int row) {
        const float(*const x)[kMaxRows / 2] = sh->warp_l + 4 * g;
        return (x[0][row] + x[1][row]) + (x[2][row] + x[3][row]);
      };
      if (TURNS && tid < RW) {
        // both groups' parts of a row, brought to the larger references
        const float4 u = sh->group_ml[0][tid], w = sh->group_ml[1][tid];
        const float c = fmaxf(u.y, w.y), a = fmaxf(beside(u.x, u.y, c), beside(w.x, w.y, c));
        const float x = sum_of(0, tid) * ex2_approx(u.y - c) + sum_of(1, tid) * ex2_approx(w.y - c);
        const bool none = x == 0.f;
        const float lg = log2f(x), f = it.slot >= 0 ? 1.f : none ? 0.f : ex2_approx(a - lg);
        sh->row_weight[tid] = part_factor(u.x, u.y, a, c) * f;
        sh->row_weight[RW + tid] = part_factor(w.x, w.y, a, c) * f;
        if (tid < it.rows) {
          if (it.slot < 0)
            p.lse[sh->row_out[qb][tid]] = none ? -INFINITY : (c + lg) * kLn2;
          else if (it.slot == 2)
            sh->part_ml[tid] = make_float4(a, c, x, 0.f);
          else
            p.ws_ml[((int64_t)blockIdx.x * 2 + it.slot) * S::R + tid] = make_float4(a, c, x, 0.f);
        }
      }
      if (!TURNS && key < RW) {
        const int all = row0 + key;
        const float x = sum_of(group, key), a = -sh->ref_e[warp][lane], c = -sh->ref_y[warp][lane];
        const bool none = x == 0.f;
        const float lg = log2f(x);
        sh->row_weight[all] = it.slot >= 0 ? 1.f : none ? 0.f : ex2_approx(a - lg);
        if (all < it.rows) {
          if (it.slot < 0)
            p.lse[sh->row_out[qb][all]] = none ? -INFINITY : (c + lg) * kLn2;
          else if (it.slot == 2)
            sh->part_ml[all] = make_float4(a, c, x, 0.f);
          else
            p.ws_ml[((int64_t)blockIdx.x * 2 + it.slot) * S::R + all] = make_float4(a, c, x, 0.f);
        }
      }
      any_at_end(false);
      auto put = [&](int row, int dim, float x) {
        if (it.slot < 0)
          p.o[sh->row_out[qb][row] * D + dim] = __float2bfloat16_rn(x);
        else if (it.slot == 2)  // (the first stage: no tile comes any more)
          reinterpret_cast<float *>(smem)[row * D + dim] = x;
        else
          p.ws_o[(((int64_t)blockIdx.x * 2 + it.slot) * S::R + row) * D + dim] = x;
      };
      if constexpr (TURNS) {
        // half of the rows a group, from both groups' accumulators
        tc_fence_after();
        static_assert(RW == 4, "");
        const bool some0 = sh->group_ml[0][0].z != 0.f, some1 = sh->group_ml[1][0].z != 0.f;
#pragma unroll 1
        for (int hf = 0; hf < NH; ++hf) {
          uint32_t u[PP * RW], w[PP * RW];
#pragma unroll
          for (int c = 0; c < PP * RW; ++c) u[c] = w[c] = 0;
          if (some0) tmem_ld<PP * RW>(t_o + t_lanes + hf * NP, u);
          if (some1) tmem_ld<PP * RW>(t_o + t_lanes + (NH + hf) * NP, w);
          const int dim = hf * 128 + key;
          if (D % 128 != 0 && dim >= D) continue;
#pragma unroll
          for (int i = 0; i < RP; ++i) {
            if (i != group) continue;
            const uint64_t x = join<PP, RW>(u + 2 * i), y = join<PP, RW>(w + 2 * i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = 2 * i + k;
              if (r >= it.rows) break;
              const float from0 = k ? f2_high(x) : f2_low(x), from1 = k ? f2_high(y) : f2_low(y);
              put(r, dim, from0 * sh->row_weight[r] + from1 * sh->row_weight[RW + r]);
            }
          }
        }
      } else
#pragma unroll 1
      for (int hf = 0; hf < NH; ++hf) {
        uint32_t o[PP * RW];
        if (some) {
          tmem_ld<PP * RW>(t_acc + hf * NP, o);
        } else {
#pragma unroll
          for (int c = 0; c < PP * RW; ++c) o[c] = 0;
        }
        const int dim = hf * 128 + key;
        if (D % 128 != 0 && dim >= D) continue;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          const uint64_t both = join<PP, RW>(o + 2 * i);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = row0 + 2 * i + k;
            if (r >= it.rows) break;
            put(r, dim, (k ? f2_high(both) : f2_low(both)) * sh->row_weight[r]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_empty[qb]);
      if (++qb == S::QBUF) qb = 0, qphase ^= 1;
    }
    if (fail) raise_abort(sh, p.status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM);
  }
  if (p.cluster > 1) {
    // The parts of the cluster's CTAs, merged by all of them; every CTA of a cluster has the same item, or none.
    cluster_sync_all();
    if (sh->start[0] >= 0 && !*abortf) {  // (a CTA that gave up may have no item)
      const Item &it = sh->item[0];
      const uint32_t o_s = smem_u32(smem), ml_s = smem_u32(sh->part_ml);
      const int rank = (int)cluster_ctarank();
      for (int i = rank * S::THREADS + tid; i < it.rows * (D / 4); i += p.cluster * S::THREADS) {
        const int row = i / (D / 4), dim = (i % (D / 4)) * 4;
        float4 ml[kMostCluster], v[kMostCluster];
        float e = kNoExp, m = kNoRef, l = 0.f;
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          ml[c] = make_float4(kNoExp, kNoRef, 0.f, 0.f);
          v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c >= p.cluster) continue;
          ml[c] = ld_cluster_f4(mapa_shared(ml_s + row * 16, c));
          v[c] = ld_cluster_f4(mapa_shared(o_s + (row * D + dim) * 4, c));
          m = fmaxf(m, ml[c].y);
        }
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) e = fmaxf(e, beside(ml[c].x, ml[c].y, m));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          const float f = part_factor(ml[c].x, ml[c].y, e, m);
          l = fmaf(ml[c].z, ex2_approx(ml[c].y - m), l);
          o.x = fmaf(f, v[c].x, o.x);
          o.y = fmaf(f, v[c].y, o.y);
          o.z = fmaf(f, v[c].z, o.z);
          o.w = fmaf(f, v[c].w, o.w);
        }
        const bool none = l == 0.f;
        const float lg = log2f(l), w = none ? 0.f : ex2_approx(e - lg);
        const int64_t at = out_row(p, it.t0, it.h, it.row0 + row);
        *reinterpret_cast<uint2 *>(p.o + at * D + dim) =
            make_uint2(pack_bf16x2(o.x * w, o.y * w), pack_bf16x2(o.z * w, o.w * w));
        if (dim == 0) p.lse[at] = none ? -INFINITY : (m + lg) * kLn2;
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
  }
}

// Merges the item that CTA blockIdx.x of the first kernel began and left unfinished:
// row blockIdx.y, its parts in the order of the tokens.  With Y = max Y_i and
// E = max (Y_i - Y) + E_i:  l = sum 2^(Y_i - Y) l_i,  O = 2^E sum 2^((Y_i - Y) + (E_i - E)) O_i / l.
// Two dependent passes through L2, launched ahead of the first kernel's end: about 4 us.
constexpr int kMergeWarps = 8;

template <typename S>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_kv8_merge_kernel(const Kv8Params p) {
  constexpr int D = S::D, R = S::R, V = (D / 4 + 31) / 32;  // float4s of a lane
  constexpr int U = V == 1 ? 4 : 2;                        // parts in flight
  __shared__ __align__(16) float part[kMergeWarps][D];
  __shared__ float4 part_ml[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y, cta = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 d = p.ws_cut[2 * cta];
  const int n = p.ws_cut[2 * cta + 1].x - cta + 1;  // parts: this CTA's second partial, then the first ones of those behind it
  if (row >= d.w) return;
  auto at = [&](int i) { return ((int64_t)(cta + i) * 2 + (i == 0 ? 1 : 0)) * R + row; };
  // a warp sums every eighth part, several in flight, with references of its own
  float e = kNoExp, m = kNoRef, l = 0.f;
  float4 o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < n; i0 += kMergeWarps * U) {
    float4 ml[U], x[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMergeWarps;
      ml[u] = make_float4(kNoExp, kNoRef, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) x[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i >= n) continue;
      ml[u] = p.ws_ml[at(i)];
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 128 + lane * 4 < D) x[u][v] = *reinterpret_cast<const float4 *>(p.ws_o + at(i) * D + v * 128 + lane * 4);
    }
    float mnow = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mnow = fmaxf(mnow, ml[u].y);
    float enow = beside(e, m, mnow);
#pragma unroll
    for (int u = 0; u < U; ++u) enow = fmaxf(enow, beside(ml[u].x, ml[u].y, mnow));
    const float f0 = part_factor(e, m, enow, mnow);
    l *= ex2_approx(m - mnow);
    e = enow;
    m = mnow;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(o[v].x * f0, o[v].y * f0, o[v].z * f0, o[v].w * f0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f = part_factor(ml[u].x, ml[u].y, e, m);
      l = fmaf(ml[u].z, ex2_approx(ml[u].y - m), l);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v].x = fmaf(f, x[u][v].x, o[v].x);
        o[v].y = fmaf(f, x[u][v].y, o[v].y);
        o[v].z = fmaf(f, x[u][v].z, o[v].z);
        o[v].w = fmaf(f, x[u][v].w, o[v].w);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * 128 + lane * 4 < D) *reinterpret_cast<float4 *>(&part[warp][v * 128 + lane * 4]) = o[v];
  if (lane == 0) part_ml[warp] = make_float4(e, m, l, 0.f);
  __syncthreads();
  l = 0.f;
  e = kNoExp;
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) m = fmaxf(m, part_ml[i].y);
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) e = fmaxf(e, beside(part_ml[i].x, part_ml[i].y, m));
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) l = fmaf(part_ml[i].z, ex2_approx(part_ml[i].y - m), l);
  const bool none = l == 0.f;
  const float lg = log2f(l), w = none ? 0.f : ex2_approx(e - lg);
  const int64_t to = out_row(p, d.x, d.y, d.z + row);
  for (int dim = threadIdx.x; dim < D; dim += kMergeWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) x = fmaf(part[i][dim], part_factor(part_ml[i].x, part_ml[i].y, e, m), x);
    p.o[to * D + dim] = __float2bfloat16_rn(x * w);
  }
  if (threadIdx.x == 0) p.lse[to] = none ? -INFINITY : (m + lg) * kLn2;
}

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
// CTAs the device holds at once.
template <typename S>
cudaError_t prepare(int device, const int **held) {
  static bool done[kMaxDevices];
  static int most[kMaxDevices][kClusterSizes];
  std::lock_guard<std::mutex> lock(g_mu);
  if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!done[device]) {
    const cudaError_t e = cudaFuncSetAttribute(attn_kv8_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < kClusterSizes; ++i) {
      ClusterLaunch<S> launch(2 << i, 2 << i, nullptr);
      if (cudaOccupancyMaxActiveClusters(&most[device][i], attn_kv8_kernel<S>, &launch.cfg) != cudaSuccess) {
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
int launch_kv8(Kv8Params &p, int device, int sms, cudaStream_t st) {
  const int *held = nullptr;  // clusters of 2, 4, 8 that the device holds at once
  cudaError_t e = prepare<S>(device, &held);
  if (e != cudaSuccess) return record_cuda_error(e);
  // What the lengths can be at most.  A request's query tokens fill no more row
  // tiles than each of them alone would, and one more than its rows / R.
  const int64_t by_rows = (int64_t)p.T * p.group / S::R + p.B, by_token = (int64_t)p.T * ((p.group + S::R - 1) / S::R);
  const int64_t tiles = (((int64_t)p.max_pages << p.shift) + TK - 1) / TK;
  const int64_t items = (by_rows < by_token ? by_rows : by_token) * p.H;
  if (items > ((int64_t)1 << 40) / (tiles + 1 + S::START)) return ATTN_ERR_ARG;  // the line's units: far inside 64 bits
  // Few and short items have a cluster of CTAs each (a power of two up to 8, doubled while a CTA has more than two
  // tiles and all clusters are resident at once), and no second kernel; pieces spread the tiles over all SMs, but
  // cost the merge's launch and about kMergeTiles tiles' time more.  The lengths are taken to be half of what the
  // table allows on average: a cluster waits for the longest.  Requests x tokens (D 128, 8 kv heads), pieces ->
  // clusters, us: 1 x 500 9.3 -> 7.5, 1 x 4000 10.5 -> 9.1, 1 x 8000 10.9 -> 11.5, 1 x 16000 12.9 -> 16.6, 8 x 2000
  // 13.8 -> 12.0 (ragged, up to 2000: 12.0 both), 16 x 1000 15.0 -> 10.8; 4 x 4000 13.7 -> 12.1 and 16 x 2000 18.8 ->
  // 15.6 have pieces all the same, as ragged ones take 11.1 -> 12.1 and 14.0 -> 15.6 (16 of up to 4000: 16.5 -> 25.2).
  // Doubled down to one tile a CTA, one request of 129 tokens 6.4 -> 6.9 us; three or four left, 1 x 1000 7.9 -> 9.1.
  p.cluster = 1;
  for (int i = 0; i < kClusterSizes && tiles > 2 * p.cluster && items <= held[i]; ++i) p.cluster *= 2;
  if (items <= sms && (tiles + p.cluster - 1) / p.cluster <= items * (tiles / 2 + S::START) / sms + kMergeTiles) {
    const ClusterLaunch<S> launch(items * p.cluster, p.cluster, st);
    e = cudaLaunchKernelEx(&launch.cfg, attn_kv8_kernel<S>, (const Kv8Params)p);
    return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
  }
  p.cluster = 0;
  const int64_t most = items * (tiles > 0 ? tiles : 1);
  const int grid = (int)(most < sms ? most : sms);
  const size_t o_bytes = (size_t)grid * 2 * S::R * S::D * 4, ml_bytes = (size_t)grid * 2 * S::R * 16;
  uint8_t *ws = nullptr;
  if (scratch_alloc(reinterpret_cast<void **>(&ws), o_bytes + ml_bytes + (size_t)grid * 32, st) != cudaSuccess || !ws) {
    cudaGetLastError();
    return ATTN_ERR_NOMEM;
  }
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float4 *>(ws + o_bytes);
  p.ws_cut = reinterpret_cast<int4 *>(ws + o_bytes + ml_bytes);
  attn_kv8_kernel<S><<<(unsigned)grid, S::THREADS, S::SMEM, st>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, S::R);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_kv8_merge_kernel<S>, (const Kv8Params)p);
  }
  const cudaError_t f = cudaFreeAsync(ws, st);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

template <int D>
int launch_rows(Kv8Params &p, int64_t rows, int device, int sms, cudaStream_t st) {
  if (rows <= 4) return launch_kv8<Shape<D, 4>>(p, device, sms, st);
  if (rows <= 8) return launch_kv8<Shape<D, 8>>(p, device, sms, st);
  // (of 192 and 256 dims the parts of 32 rows would leave K and V two stages)
  if (rows <= 16 || D > 128) return launch_kv8<Shape<D, 16>>(p, device, sms, st);
  return launch_kv8<Shape<D, D <= 128 ? 32 : 16>>(p, device, sms, st);
}

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace
}  // namespace attn

extern "C" {

int attn_fwd_kv8(const void *q, long long q_stride_t, long long q_stride_h, const int *cu, const int *lens,
                 const int *block_table, long long table_stride, int max_pages, const void *cache, int num_pages,
                 void *o, float *lse, int B, int T, int Hq, int Hkv, int D, int page_size, float scale, int causal,
                 attn_stream_t stream) {
  using namespace attn;
  if (B < 0 || B > kMaxRequests || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65535) return ATTN_ERR_ARG;
  if (D < 64 || D > ATTN_KV8_MAX_HEAD_DIM || D % 64 != 0) return ATTN_ERR_ARG;
  const int shift = kv4_page_shift(page_size);
  if (shift < 0 || num_pages < 0 || max_pages < 0 || (causal != 0 && causal != 1) || !isfinite(scale))
    return ATTN_ERR_ARG;
  if (max_pages > (0x7fffffff >> shift) - 16 || table_stride < max_pages) return ATTN_ERR_ARG;
  if ((int64_t)T * (Hq / Hkv) > 0x3fffffff || (int64_t)num_pages * page_size > 0x7fffffffLL) return ATTN_ERR_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!q || !o || !lse || !cu || !lens) return ATTN_ERR_ARG;
  if ((max_pages > 0 && !block_table) || (num_pages > 0 && !cache)) return ATTN_ERR_ARG;
  if (q_stride_t < 0 || q_stride_h < 0) return ATTN_ERR_ARG;
  if (off16(q) || off16(o) || off16(lse) || off16(cache) || q_stride_t % 8 || q_stride_h % 8) return ATTN_ERR_ALIGN;
  for (const int *a : {cu, lens, block_table})
    if (reinterpret_cast<uintptr_t>(a) & 3u) return ATTN_ERR_ALIGN;
  int device = 0, sms = 0;
  Kv8Params p{};
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
  p.wait_limit_ns = wait_limit_ns();
  p.drop = debug_flags() & ATTN_DEBUG_DROP_V_COPY;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Rows of a tile, by the rows that a request has on average: the fewest that hold them, or the most there are.
  const int64_t rows = (int64_t)p.group * ((T + B - 1) / B);
  switch (D / 64) {
    case 1: return launch_rows<64>(p, rows, device, sms, st);
    case 2: return launch_rows<128>(p, rows, device, sms, st);
    case 3: return launch_rows<192>(p, rows, device, sms, st);
    default: return launch_rows<256>(p, rows, device, sms, st);
  }
}

}  // extern "C"
