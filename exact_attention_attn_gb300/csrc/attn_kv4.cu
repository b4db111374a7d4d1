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
// accumulator transposed through movmatrix.  The order of the dims inside the
// first product and of the tokens inside the second is free, and is chosen so
// that every operand register comes from an aligned word of the page.
//
// Softmax.  p = 2^(y - ref), ref a per-row reference 10 above which the warp
// rescales only when some y exceeds ref + 15; P s' is rounded to half
// precision (2^-11 relative; bfloat16's 2^-8 would be as large as the output's own
// rounding) after dividing by a power of two that tracks the group's
// largest scale, so that its products keep 11 bits down to 2^-24 of the
// largest.  l and the sums of p m' are in float32.
//
// Work split.  The tiles of 64 tokens of all (request, kv head, row tile)
// items form one line, cut into equal pieces, one per resident CTA: lengths
// are read on the device, and no CTA is longer than another by more than a
// tile.  An item cut by a piece's border leaves partial (ref, l, O) in a
// workspace, at most two per CTA, which a second kernel -- launched early, its
// wait overlapping the first's end -- merges in the order of the tokens.
//
// Memory.  A producer warp copies each tile's pages (one contiguous bulk copy
// per page: 36 bytes x D/32 per token) into a ring of stages; four consumer
// warps take 16 tokens each.  Bound: HBM for up to 8 rows per kv head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <mutex>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

#ifndef KV4_CW
#define KV4_CW 4
#endif
#ifndef KV4_E
#define KV4_E 4
#endif
#ifndef KV4_MIN
#define KV4_MIN 1
#endif
#ifndef KV4_CTAS
#define KV4_CTAS 0
#endif
constexpr int CW = KV4_CW;     // consumer warps, 16 tokens of a tile each
constexpr int TK = CW * 16;    // tokens per tile (a stage of the ring)
constexpr int CT = CW * 32;
constexpr int THREADS = CT + 32;
constexpr int START = KV4_E;   // an item's beginning and end cost about as much as this many tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -1e37f;  // reference of a row that has seen no key
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
  int chunk_min;     // least tiles of a CTA
  float *ws_o;       // partial O of cut items: [grid][2][R][D]
  float2 *ws_ml;     // their reference and l: [grid][2][R]
  int4 *ws_cut;      // [grid][2]: the item that each CTA leaves unfinished
  int *status;
  uint64_t wait_limit;
};

// What a request's tiles look like, from the device arrays, with whatever
// they hold brought into range (reported once through the status word).
struct Request {
  int t0, nq, len;   // first query token, query tokens, cached tokens
  int tiles, rt;     // tiles of 64 tokens (at least one), row tiles
  __device__ __forceinline__ int64_t units(int H) const { return (int64_t)H * rt * (tiles + START); }
};

template <int R>
__device__ __forceinline__ Request load_request(const Kv4Params &p, int r) {
  Request q;
  const int a = p.cu[r], b = p.cu[r + 1], l = p.lens[r];
  const int room = p.max_pages << p.shift;
  q.t0 = min(max(a, 0), p.T);
  const int t1 = min(max(b, q.t0), p.T);
  q.nq = t1 - q.t0;
  q.len = min(max(l, 0), room);
  if (q.t0 != a || t1 != b || q.len != l) atomicCAS(p.status, 0, kStatusDevice);
  q.tiles = max(1, (q.len + TK - 1) / TK);
  q.rt = (int)(((int64_t)q.nq * p.group + R - 1) / R);
  return q;
}

// Position of a CTA's piece in the line of tiles.
struct Piece {
  int64_t begin, end, chunk, total;
  int r;            // request that holds tile `begin`
  int64_t base;     // its first tile
};

// All threads: total tiles, this CTA's piece, and the request it begins in.
template <int R>
__device__ __forceinline__ void find_piece(const Kv4Params &p, Piece &pc) {
  __shared__ int64_t wsum[THREADS / 32];
  __shared__ int64_t found_base;
  __shared__ int found_r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + THREADS - 1) / THREADS;  // consecutive requests of a thread
  const int r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += load_request<R>(p, r).units(p.H);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
  if (chunk < p.chunk_min) chunk = p.chunk_min;
  pc.chunk = chunk;
  pc.total = total;
  pc.begin = min((int64_t)blockIdx.x * chunk, total);
  pc.end = min(pc.begin + chunk, total);
  int64_t at = before + inc - mine;
  if (pc.begin >= at && pc.begin < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t n = load_request<R>(p, r).units(p.H);
      if (pc.begin < at + n) {
        found_r = r;
        found_base = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  pc.r = pc.begin < total ? found_r : 0;
  pc.base = pc.begin < total ? found_base : 0;
}

// One (request, kv head, row tile) of a piece: tiles [tile0, tile0 + n).
struct Item {
  Request q;
  int r, h, rt, tile0, n;
  bool whole;     // the piece holds all of the item
  int64_t end;    // the item's last unit + 1, in the line
  // last visible key + 1 of row `row` (rows count query token x group head)
  __device__ __forceinline__ int limit(int row, const Kv4Params &p) const {
    const int i = row / p.group;
    return p.causal ? min(q.len, max(0, i + 1 + q.len - q.nq)) : q.len;
  }
};

struct Walk {
  int64_t at, end, base;
  int r;
  Request q;
  template <int R>
  __device__ __forceinline__ void start(const Kv4Params &p, const Piece &pc) {
    at = pc.begin;
    end = pc.end;
    base = pc.base;
    r = pc.r;
    if (at < end) q = load_request<R>(p, r);
  }
  // Next item of the piece; false at its end.
  template <int R>
  __device__ __forceinline__ bool next(const Kv4Params &p, Item &it) {
    while (at < end) {
      while (at >= base + q.units(p.H)) {  // also steps over requests without query tokens
        base += q.units(p.H);
        if (++r >= p.B) return false;
        q = load_request<R>(p, r);
      }
      const int64_t local = at - base;
      const int per = q.tiles + START;
      const int64_t item = local / per;
      const int off = (int)(local - item * per), n = (int)min((int64_t)(per - off), end - at);
      const int tile0 = max(0, off - START), tile1 = max(0, off + n - START);
      at += n;
      if (tile0 == tile1) continue;  // no tile of the item itself: it begins in the next piece
      it.q = q;
      it.r = r;
      it.tile0 = tile0;
      it.h = (int)(item / q.rt);
      it.rt = (int)(item - (int64_t)it.h * q.rt);
      it.n = tile1 - tile0;
      it.end = at - n - off + per;
      it.whole = it.n == q.tiles;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

template <int G, int R>
struct Kv4Shape {
  static constexpr int D = G * kKv4Group;
  static constexpr int NT = R / 8;                       // n8 tiles of rows
  static constexpr int STAGE = TK * G * 2 * (kKv4RowBytes + kKv4PairBytes);
  static constexpr int STAGES = G <= 2 ? 4 : 3;
  static constexpr int MERGE_PITCH = D + 4;              // floats per row of the warps' merge buffer
  static constexpr int MERGE = CW * R * MERGE_PITCH * 4;
  static constexpr int SMEM = STAGES * STAGE + MERGE + 2 * CW * R * 4 + 2 * STAGES * 8 + 16;
};

template <int G, int R>
__global__ void __launch_bounds__(THREADS) attn_kv4_kernel(const Kv4Params p) {
  using Sh = Kv4Shape<G, R>;
  constexpr int NT = Sh::NT, D = Sh::D, STAGES = Sh::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  float *merge_o = reinterpret_cast<float *>(smem + STAGES * Sh::STAGE);     // [CW][R][MERGE_PITCH]
  float *merge_ref = merge_o + CW * R * Sh::MERGE_PITCH;                     // [CW][R]
  float *merge_l = merge_ref + CW * R;                                       // [CW][R]
  uint64_t *full = reinterpret_cast<uint64_t *>(merge_l + CW * R);
  uint64_t *empty = full + STAGES;
  volatile int *abort = reinterpret_cast<volatile int *>(empty + STAGES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], CW);
    }
    *abort = 0;
    fence_mbar_init();
  }
  Piece pc;
  find_piece<R>(p, pc);  // its barriers also publish the mbarriers
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int P = 1 << p.shift;
  const int page_bytes = kv4_page_bytes(G, P);
  Walk walk;
  walk.start<R>(p, pc);
  Item it;

  if (warp == CW) {  // ---------------------------------------------------------------- producer
    int n = 0, st = 0, ph = 1;  // tiles issued; stage, and the parity of its last release
    const int ppt = TK >> p.shift;  // pages of a tile
    bool ok = true;
    while (ok && walk.next<R>(p, it)) {
      const int last_row = min(it.q.nq * p.group, (it.rt + 1) * R) - 1;
      const int stop = min(it.tile0 + it.n, (it.limit(last_row, p) + TK - 1) / TK);
      const int *row = p.table + (int64_t)it.r * p.table_stride;
      const int pages = (it.q.len + P - 1) >> p.shift;
      for (int tile = it.tile0; ok && tile < stop; ++tile, ++n) {
        const int pg = tile * ppt + lane;
        const bool have = lane < ppt && pg < pages;
        int id = have ? row[pg] : 0;
        if ((unsigned)id >= (unsigned)p.num_pages) {  // not a page: report it and read the first one instead
          atomicCAS(p.status, 0, kStatusDevice);
          id = 0;
        }
        if (n >= STAGES) ok = mbar_wait(&empty[st], ph, abort, p.wait_limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          atomicCAS(p.status, 0, kStatusTimeout);
          *abort = 1;
          break;
        }
        const int cnt = min(ppt, pages - tile * ppt);
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(cnt * page_bytes));
        __syncwarp();
        if (have)
          bulk_load(smem + st * Sh::STAGE + lane * page_bytes, p.cache + ((int64_t)id * p.H + it.h) * page_bytes,
                    (uint32_t)page_bytes, &full[st]);
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // Every copy of this CTA lands before its shared memory is given back.
    // (The consumers have waited for all of them unless a wait ran out.)
    if (*abort)
      for (int i = max(0, n - STAGES); i < n; ++i) mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1, p.wait_limit);
    return;
  }

  // ------------------------------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  // token of row m of the K operand: 0 6 1 7 2 4 3 5 (+ 8 for the upper rows),
  // which makes both the K rows a half warp reads and the V rows of one k
  // index fall into different 32-byte quarters of the banks
  const int perm = (g >> 1) + ((g & 1) ? ((g >> 1) < 2 ? 6 : 2) : 0);
  const int vtok = ((t + 2) & 3) + 4;  // V token of k index 2t + 1 (that of 2t is t)
  int st = 0, ph = 0;  // stage of the next tile, and its parity
  it.tile0 = -1;       // (a piece may hold no tile at all)
  while (walk.next<R>(p, it)) {
    const int rows = it.q.nq * p.group;
    const int row0 = it.rt * R;
    const int last_row = min(rows, row0 + R) - 1;
    const int stop = min(it.tile0 + it.n, (it.limit(last_row, p) + TK - 1) / TK);
    const int full_to = min(it.limit(row0, p), it.q.len);  // tokens before it are visible to every row

    // Q: lane (g, t) holds row g's dims of the words 2t, 2t + 1 of each group,
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
        const int i = row / p.group, hg = row - i * p.group;
        const __nv_bfloat16 *src =
            p.q + (int64_t)(it.q.t0 + i) * p.qt + (int64_t)(it.h * p.group + hg) * p.qh + t * 16;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          w[j][0] = *reinterpret_cast<const uint4 *>(src + j * kKv4Group);
          w[j][1] = *reinterpret_cast<const uint4 *>(src + j * kKv4Group + 8);
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
      const float up = pow2(e);
      float qs[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        qs[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[8];
          const uint32_t ws[4] = {w[j][k].x, w[j][k].y, w[j][k].z, w[j][k].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v[2 * c] = __uint_as_float(ws[c] << 16) * up;
            v[2 * c + 1] = __uint_as_float(ws[c] & 0xffff0000u) * up;
            qs[j] += v[2 * c] + v[2 * c + 1];
          }
          // nibbles (0, 4) and (1, 5), then (2, 6) and (3, 7); odd nibbles carry a factor 16
          qb[nt][j][2 * k][0] = half2_bits(v[0], v[4]);
          qb[nt][j][2 * k][1] = half2_bits(v[1] * 0.0625f, v[5] * 0.0625f);
          qb[nt][j][2 * k + 1][0] = half2_bits(v[2], v[6]);
          qb[nt][j][2 * k + 1][1] = half2_bits(v[3] * 0.0625f, v[7] * 0.0625f);
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
    float ref[NT][2], l[NT][2], vm[NT][G][2], isig[G];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ref[nt][c] = kNoRef;
        l[nt][c] = 0.f;
        const int row = row0 + nt * 8 + 2 * t + c;
        lim[nt][c] = row < rows ? it.limit(row, p) : 0;
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        vm[nt][j][0] = vm[nt][j][1] = 0.f;
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[nt][j][d][0] = acc[nt][j][d][1] = acc[nt][j][d][2] = acc[nt][j][d][3] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < G; ++j) isig[j] = 0x1p100f;

    for (int tile = it.tile0; tile < stop; ++tile) {
      const bool got = mbar_wait(&full[st], ph, abort, p.wait_limit);
      if (!__all_sync(0xffffffffu, got)) {
        atomicCAS(p.status, 0, kStatusTimeout);
        *abort = 1;  // every role stops; the loops run out without waiting
        continue;
      }
      const int tok0 = tile * TK + warp * 16;
      if (tok0 < it.q.len) {
        const int in = warp * 16, pgi = in >> p.shift, off = in & (P - 1);
        const uint8_t *kc = smem + st * Sh::STAGE + pgi * page_bytes + off * kKv4RowBytes;
        const uint8_t *km = smem + st * Sh::STAGE + pgi * page_bytes + kv4_codes_bytes(G, P) + off * kKv4PairBytes;
        const uint8_t *vc = kc + kv4_side_bytes(G, P), *vp = km + kv4_side_bytes(G, P);
        const int ta = tok0 + perm, tb = ta + 8;  // the lane's two tokens of S^T
        const bool edge = tok0 + 16 > full_to;
const bool tail = tok0 + 16 > it.q.len;

        // S^T = K Q^T on the codes, joined over the groups with scales and minima
        float x[NT][4];
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint2 wa = *reinterpret_cast<const uint2 *>(kc + (j * P + perm) * kKv4RowBytes + t * 8);
          const uint2 wb = *reinterpret_cast<const uint2 *>(kc + (j * P + perm + 8) * kKv4RowBytes + t * 8);
          const uint32_t pa = *reinterpret_cast<const uint32_t *>(km + (j * P + perm) * kKv4PairBytes);
          const uint32_t pb = *reinterpret_cast<const uint32_t *>(km + (j * P + perm + 8) * kKv4PairBytes);
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t xa = k ? wa.y : wa.x, xb = k ? wb.y : wb.x;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t a0 = xa & 0x000f000fu, a1 = xb & 0x000f000fu, a2 = xa & 0x00f000f0u, a3 = xb & 0x00f000f0u;
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
              x[nt][c] = fmaf(sa, s[nt][c], j ? fmaf(ma, qsum[nt][j][c], x[nt][c]) : ma * qsum[nt][j][c]);
              x[nt][2 + c] = fmaf(sb, s[nt][2 + c], j ? fmaf(mb, qsum[nt][j][c], x[nt][2 + c]) : mb * qsum[nt][j][c]);
            }
        }
        // V's scales (over the warp's power of two) and minima of the lane's two tokens
        float ua[G], ub[G], ma[G], mb[G];
        float big_v = 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          uint32_t pa = *reinterpret_cast<const uint32_t *>(vp + (j * P + perm) * kKv4PairBytes);
          uint32_t pb = *reinterpret_cast<const uint32_t *>(vp + (j * P + perm + 8) * kKv4PairBytes);
          if (tail) {  // nothing past the request's end is used, whatever it is
            pa = ta < it.q.len ? pa : 0u;
            pb = tb < it.q.len ? pb : 0u;
          }
          ua[j] = __uint_as_float(pa << 16) * isig[j];
          ub[j] = __uint_as_float(pb << 16) * isig[j];
          ma[j] = __uint_as_float(pa & 0xffff0000u);
          mb[j] = __uint_as_float(pb & 0xffff0000u);
          big_v = max3f(big_v, ua[j], ub[j]);
        }
        // e = y - ref in log2 units; hidden tokens -inf (selected, so that nothing they hold is used)
        float e[NT][4];
        float top = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            e[nt][c] = fmaf(x[nt][c], fac[nt][c], -ref[nt][c]);
            e[nt][2 + c] = fmaf(x[nt][2 + c], fac[nt][c], -ref[nt][c]);
            if (edge) {
              if (ta >= lim[nt][c]) e[nt][c] = -INFINITY;
              if (tb >= lim[nt][c]) e[nt][2 + c] = -INFINITY;
            }
            top = max3f(top, e[nt][c], e[nt][2 + c]);
          }
        if (__any_sync(0xffffffffu, top > 15.f || big_v > 1.9f)) {  // move the references up
          float fs[G];
#pragma unroll
          for (int j = 0; j < G; ++j) {
            // from the scales themselves: over the old power of two they may have overflowed
            const uint32_t pa = *reinterpret_cast<const uint32_t *>(vp + (j * P + perm) * kKv4PairBytes);
            const uint32_t pb = *reinterpret_cast<const uint32_t *>(vp + (j * P + perm + 8) * kKv4PairBytes);
            const float sa = ta < it.q.len ? __uint_as_float(pa << 16) : 0.f;
            const float sb = tb < it.q.len ? __uint_as_float(pb << 16) : 0.f;
            float big = fmaxf(sa < INFINITY ? sa : 0.f, sb < INFINITY ? sb : 0.f);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            fs[j] = 1.f;
            if (big * isig[j] > 1.f) {  // the largest scale becomes [0.5, 1)
              const float now = pow2(max(-126, -1 - exp_of(big)));
              fs[j] = now / isig[j];
              isig[j] = now;
              ua[j] = sa * now;
              ub[j] = sb * now;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float ya = e[nt][c] == -INFINITY ? -INFINITY : x[nt][c] * fac[nt][c];
              const float yb = e[nt][2 + c] == -INFINITY ? -INFINITY : x[nt][2 + c] * fac[nt][c];
              float m = fmaxf(ya, yb);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
              const float now = fmaxf(ref[nt][c], m - 10.f);
              const float f = ex2_approx(ref[nt][c] - now);
              ref[nt][c] = now;
              e[nt][c] = ya - now;
              e[nt][2 + c] = yb - now;
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
        }
        float pr[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            pr[nt][c] = ex2_approx(e[nt][c]);
            pr[nt][2 + c] = ex2_approx(e[nt][2 + c]);
            l[nt][c] += pr[nt][c] + pr[nt][2 + c];
          }
        // O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < G; ++j) {
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4] = {pr[nt][0] * ua[j], pr[nt][1] * ua[j], pr[nt][2] * ub[j], pr[nt][3] * ub[j]};
            if (!edge) {
#pragma unroll
              for (int c = 0; c < 2; ++c) vm[nt][j][c] = fmaf(pr[nt][2 + c], mb[j], fmaf(pr[nt][c], ma[j], vm[nt][j][c]));
            } else {  // a hidden token's scale and minimum may be anything
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const bool no_a = e[nt][c] == -INFINITY, no_b = e[nt][2 + c] == -INFINITY;
                if (no_a) w[c] = 0.f;
                if (no_b) w[2 + c] = 0.f;
                vm[nt][j][c] = fmaf(pr[nt][2 + c], no_b ? 0.f : mb[j], fmaf(pr[nt][c], no_a ? 0.f : ma[j], vm[nt][j][c]));
              }
            }
            b0[nt] = transpose8x8(half2_bits(w[0], w[1]));
            b1[nt] = transpose8x8(half2_bits(w[2], w[3]));
          }
          const uint8_t *v0 = vc + (j * P + t) * kKv4RowBytes + g * 4, *v1 = vc + (j * P + vtok) * kKv4RowBytes + g * 4;
          const uint32_t x0 = *reinterpret_cast<const uint32_t *>(v0), x1 = *reinterpret_cast<const uint32_t *>(v1);
          const uint32_t x2 = *reinterpret_cast<const uint32_t *>(v0 + 8 * kKv4RowBytes);
          const uint32_t x3 = *reinterpret_cast<const uint32_t *>(v1 + 8 * kKv4RowBytes);
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // dims 0-3, then 4-7 of the lane's 8
            uint32_t z0 = __byte_perm(x0, x1, k ? 0x7632 : 0x5410), z1 = __byte_perm(x2, x3, k ? 0x7632 : 0x5410);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t a0 = z0 & 0x000f000fu, a1 = z0 & 0x00f000f0u, a2 = z1 & 0x000f000fu, a3 = z1 & 0x00f000f0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][j][2 * k + hh], a0, a1, a2, a3, b0[nt], b1[nt]);
              z0 >>= 8;
              z1 >>= 8;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (++st == STAGES) {
        st = 0;
        ph ^= 1;
      }
    }

    // ---- the item's end: sum over the lanes, then merge the warps
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
        const int row = nt * 8 + 2 * t + c;
        if (g == 0) {
          merge_ref[warp * R + row] = ref[nt][c];
          merge_l[warp * R + row] = l[nt][c];
        }
        float *dst = merge_o + (warp * R + row) * Sh::MERGE_PITCH + g * 8;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float sig = 0x1p24f / isig[j], m = vm[nt][j][c];
          float4 lo, hi;
          lo.x = fmaf(acc[nt][j][0][c], sig, m);
          lo.y = fmaf(acc[nt][j][0][2 + c], sig * 0.0625f, m);
          lo.z = fmaf(acc[nt][j][1][c], sig, m);
          lo.w = fmaf(acc[nt][j][1][2 + c], sig * 0.0625f, m);
          hi.x = fmaf(acc[nt][j][2][c], sig, m);
          hi.y = fmaf(acc[nt][j][2][2 + c], sig * 0.0625f, m);
          hi.z = fmaf(acc[nt][j][3][c], sig, m);
          hi.w = fmaf(acc[nt][j][3][2 + c], sig * 0.0625f, m);
          *reinterpret_cast<float4 *>(dst + j * kKv4Group) = lo;
          *reinterpret_cast<float4 *>(dst + j * kKv4Group + 4) = hi;
        }
      }
    asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
    const int slot = it.tile0 > 0 ? 0 : 1;
    const int64_t part = ((int64_t)blockIdx.x * 2 + slot) * R;
    for (int i = tid; i < R * (D / 4); i += CT) {
      const int row = i / (D / 4), d = (i % (D / 4)) * 4, q = row0 + row;
      if (q >= rows) break;
      float m = merge_ref[row];
#pragma unroll
      for (int w = 1; w < CW; ++w) m = fmaxf(m, merge_ref[w * R + row]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const float f = ex2_approx(merge_ref[w * R + row] - m);
        const float4 v = *reinterpret_cast<const float4 *>(merge_o + (w * R + row) * Sh::MERGE_PITCH + d);
        if (saw_none(merge_ref[w * R + row], merge_l[w * R + row])) continue;
        sum = fmaf(merge_l[w * R + row], f, sum);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      }
      if (it.whole) {
        const bool none = saw_none(m, sum);
        const float inv = none ? 0.f : 1.f / sum;
        const int64_t at = (int64_t)(it.q.t0 + q / p.group) * (p.H * p.group) + it.h * p.group + q % p.group;
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        uint2 u;
        memcpy(&u.x, &h0, 4);
        memcpy(&u.y, &h1, 4);
        *reinterpret_cast<uint2 *>(p.o + at * D + d) = u;
        if (d == 0) p.lse[at] = none ? -INFINITY : (m + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(p.ws_o + (part + row) * D + d) = o;
        if (d == 0) p.ws_ml[part + row] = make_float2(m, sum);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");  // the merge buffer is free again
  }
  // What the second kernel has to merge: the item that began here and goes on
  // in later CTAs, or nothing (no rows).
  if (tid == 0) {
    int4 d = make_int4(0, 0, 0, 0);
    int last = 0;
    if (it.tile0 == 0 && !it.whole) {
      d = make_int4(it.q.t0, it.h, it.rt * R, min(it.q.nq * p.group - it.rt * R, R));
      last = (int)((it.end - 1) / pc.chunk);  // the CTA that ends it
    }
    p.ws_cut[blockIdx.x * 2] = d;
    p.ws_cut[blockIdx.x * 2 + 1] = make_int4(last, 0, 0, 0);
  }
}

// Merges the partials of one row of the item that CTA blockIdx.x of the first
// kernel began and left unfinished: that CTA's second partial and the first
// partials of the CTAs after it, up to the one that ends the item.  With
// M = max ref_i:  O = sum 2^(ref_i - M) O_i / sum 2^(ref_i - M) l_i.  The
// weights go through shared memory first, so that every load of a partial is
// independent; the partials are summed in a fixed order.
constexpr int kMergeThreads = 256;
constexpr int kMaxGrid = 2048;

template <int G>
__global__ void __launch_bounds__(kMergeThreads) attn_kv4_merge_kernel(const Kv4Params p, int R) {
  constexpr int D = G * kKv4Group, COLS = D / 4, NG = kMergeThreads / COLS;
  __shared__ float weight[kMaxGrid];
  __shared__ float red[kMergeThreads / 32];
  __shared__ __align__(16) float part[NG][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  const int4 d = p.ws_cut[2 * c];
  if (row >= d.w) return;
  const int n = p.ws_cut[2 * c + 1].x - c + 1;
  auto index = [&](int i) { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * R + row; };
  auto reduce = [&](float v, bool sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = sum ? v + u : fmaxf(v, u);
    }
    if ((tid & 31) == 0) red[tid >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kMergeThreads / 32; ++w) v = sum ? v + red[w] : fmaxf(v, red[w]);
    __syncthreads();
    return v;
  };
  float m = kNoRef;
  for (int i = tid; i < n; i += kMergeThreads) m = fmaxf(m, p.ws_ml[index(i)].x);
  m = reduce(m, false);
  float l = 0.f;
  for (int i = tid; i < n; i += kMergeThreads) {
    const float2 ml = p.ws_ml[index(i)];
    const float f = saw_none(ml.x, ml.y) ? 0.f : ex2_approx(ml.x - m);
    weight[i] = f;
    l = fmaf(f, ml.y, l);
  }
  l = reduce(l, true);
  const int grp = tid / COLS, col = (tid % COLS) * 4;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < NG) {
#pragma unroll 4
    for (int i = grp; i < n; i += NG) {
      const float f = weight[i];
      const float4 v = *reinterpret_cast<const float4 *>(p.ws_o + index(i) * D + col);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    *reinterpret_cast<float4 *>(&part[grp][col]) = o;
  }
  __syncthreads();
  const bool none = saw_none(m, l);
  const float inv = none ? 0.f : 1.f / l;
  const int q = d.z + row;
  const int64_t at = (int64_t)(d.x + q / p.group) * (p.H * p.group) + d.y * p.group + q % p.group;
  if (tid < COLS) {
#pragma unroll
    for (int w = 1; w < NG; ++w) {
      const float4 v = *reinterpret_cast<const float4 *>(&part[w][col]);
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
    }
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    uint2 u;
    memcpy(&u.x, &h0, 4);
    memcpy(&u.y, &h1, 4);
    *reinterpret_cast<uint2 *>(p.o + at * D + col) = u;
  }
  if (tid == 0) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// CTAs of a variant that one SM holds, on each device; sets the kernel's
// shared-memory limit on the first call there.
constexpr int kMaxDevices = 64;
std::mutex g_mu;

template <int G, int R>
cudaError_t resident(int device, int *out) {
  static int known[kMaxDevices];
  std::lock_guard<std::mutex> lock(g_mu);
  if (known[device] == 0) {
    constexpr int smem = Kv4Shape<G, R>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(attn_kv4_kernel<G, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kv4_kernel<G, R>, THREADS, smem)) != cudaSuccess)
      return e;
    known[device] = n < 1 ? 1 : n;
  }
  *out = known[device];
  return cudaSuccess;
}

template <int G, int R>
int launch_kv4(Kv4Params &p, int device, int sms, cudaStream_t st) {
  constexpr int D = G * kKv4Group;
  int per_sm = 0;
  cudaError_t e = resident<G, R>(device, &per_sm);
  if (e != cudaSuccess) return record_cuda_error(e);
  // no more CTAs than there can be tiles
  const int64_t rows = (int64_t)p.T * p.group, row_tiles = rows / R + p.B;
  const int64_t tiles = (((int64_t)p.max_pages << p.shift) + TK - 1) / TK + START;
  const int64_t most = row_tiles * p.H * (tiles < 1 ? 1 : tiles);
  int grid = sms * (KV4_CTAS ? KV4_CTAS : per_sm);
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (grid > most) grid = (int)most;
  const size_t o_bytes = (size_t)grid * 2 * R * D * 4, ml_bytes = (size_t)grid * 2 * R * 8;
  uint8_t *ws = nullptr;
  if (scratch_alloc(reinterpret_cast<void **>(&ws), o_bytes + ml_bytes + (size_t)grid * 32, st) != cudaSuccess || !ws) {
    cudaGetLastError();
    return ATTN_ERR_NOMEM;
  }
  p.ws_o = reinterpret_cast<float *>(ws);
  p.ws_ml = reinterpret_cast<float2 *>(ws + o_bytes);
  p.ws_cut = reinterpret_cast<int4 *>(ws + o_bytes + ml_bytes);
  attn_kv4_kernel<G, R><<<grid, THREADS, Kv4Shape<G, R>::SMEM, st>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, R);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_kv4_merge_kernel<G>, (const Kv4Params)p, (int)R);
  }
  const cudaError_t f = cudaFreeAsync(ws, st);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
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
  if ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(block_table)) & 3u)
    return ATTN_ERR_ALIGN;
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
  p.chunk_min = KV4_MIN;
  p.wait_limit = wait_limit_ns();
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // 16 rows a tile where the requests have more than 8 on average: K and V
  // are then read and unpacked once for 16 rows; at D > 128 the accumulators
  // of 16 rows would not leave registers for a second CTA on the SM
  const bool wide = (int64_t)p.group * ((T + B - 1) / B) > 8;
  switch (D / 64) {
    case 1: return wide ? launch_kv4<1, 16>(p, device, sms, st) : launch_kv4<1, 8>(p, device, sms, st);
    case 2: return wide ? launch_kv4<2, 16>(p, device, sms, st) : launch_kv4<2, 8>(p, device, sms, st);
    case 3: return launch_kv4<3, 8>(p, device, sms, st);
    default: return launch_kv4<4, 8>(p, device, sms, st);
  }
}

}  // extern "C"
