// The 8-bit KV cache: quantising tokens into their slots, and reading slots back as
// bfloat16.
//
// Per block of 16 tokens and kv head, for K and for V: the scale is 2^k, k the smallest
// integer from -100 on with max |x| <= 448 2^k over the block's tokens, and a value is
// held as e4m3(x / 2^k), rounded to nearest, ties to even.  Where a later token needs a
// larger scale, the codes held are rounded again (a shift of their exponents: exact but
// for e4m3's subnormals).  A token whose K (V) holds an infinity or a NaN counts for no
// scale, has codes 0 and a bit that makes it stand for NaN.  Writing a block's first
// slot starts the block anew.
//
// A warp has K or V of one block of one head: 16 tokens x D dims, D / 32 dims a lane,
// so that the maximum is one warp reduction and V's rows of 16 tokens are a lane's own
// values (a CTA for a block, its maxima joined in shared memory: 30.6 us for 16384
// tokens of 8 heads of 128).  It works alone: it looks for the first tokens of blocks
// among a few tokens (`window`), and for a block's tokens among the 15 behind that.  A
// block of which the call has one token (a decode step) is taken with work for one
// token only, the K and V of two heads in flight.
//
// Measured: append of 16384 tokens of 8 heads of 128 (101 MB) 20.0 us, 5.0 TB/s, bound
// by the latency of its loads (a lane has 32 registers of the block's words under way, 116
// of the 128 that two CTAs an SM leave, so 16 warps; 3 or 4 CTAs spill: 26 .. 44 us).  Read of them 16.5 us, 6.1 TB/s:
// HBM. Append of 64 single tokens 3.2 us, three dependent loads; of 1024 17.5 us (20 as
// blocks): a token's V is a byte in each of D rows of 16, so what is written are
// partial sectors.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv8.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kAtOnce = 4;       // heads' K or V of a single token
constexpr int kMostWindow = 16;  // tokens whose blocks a warp looks for

struct AppendParams {
  const __nv_bfloat16 *k, *v;
  int64_t kt, kh, vt, vh;  // element strides of token and head
  const int *slots;
  uint8_t *cache;
  int64_t nslots;
  int T, H, shift;
  int window;  // tokens of a warp
  int share;   // (head, side) pairs of a warp: 2 h for K, 2 h + 1 for V
  int *status;
};

// Dims of a lane: of 192 dims 24 lanes have 8 each (6 in 32 lanes cannot be loaded
// or stored at once: append of 8192 tokens of 8 heads 31.7 us).
constexpr __host__ __device__ int lane_dims(int G) { return G == 3 ? 8 : 2 * G; }

// The lane's dims of one token: W words of two bfloat16.
template <int W>
__device__ __forceinline__ void load_words(const __nv_bfloat16 *from, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(from);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(from);
    w[0] = x.x; w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t *>(from)[i];
  }
}

__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Exponent of the scale for a largest magnitude given as bfloat16 bits: 448 =
// 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(uint32_t most) {
  const int k = (int)(most >> 7) - 127 - 8 + ((most & 0x7fu) > 0x60u ? 1 : 0);
  return max(k, kKv8Least);
}

__device__ __forceinline__ uint32_t float_bits_of(int k) { return (uint32_t)(k + 127) << 23; }

// The exponent of a held scale; below every other where there is none.
__device__ __forceinline__ int held_exponent(uint32_t bits) {
  const int k = (int)(bits >> 23) - 127;
  return bits >> 31 || k < kKv8Least || k > 127 ? -1000 : k;
}

__device__ __forceinline__ uint32_t halves_of_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_of_halves(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}

// Four codes times 2^-d, rounded again.  Half precision holds the products: what
// it rounds is below e4m3's smallest number by far.
__device__ __forceinline__ uint32_t shift_codes(uint32_t codes, __half2 factor) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h = halves_of_e4m3x2(codes >> (16 * i));
    __half2 x;
    memcpy(&x, &h, 4);
    x = __hmul2(x, factor);
    memcpy(&h, &x, 4);
    out |= e4m3x2_of_halves(h) << (16 * i);
  }
  return out;
}

__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The largest magnitude (bfloat16 bits) in the warp's words.
template <int N, int W>
__device__ __forceinline__ uint32_t largest(const uint32_t (&x)[N][W]) {
  uint32_t m = 0;
#pragma unroll
  for (int o = 0; o < N; ++o)
#pragma unroll
    for (int i = 0; i < W; ++i) m = __vmaxu2(m, x[o][i] & 0x7fff7fffu);
  return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
}

// The tokens with an infinity or a NaN, whose words are zeroed.
template <int N, int W>
__device__ __forceinline__ uint32_t mark_tokens(uint32_t (&x)[N][W]) {
  uint32_t bad = 0;
#pragma unroll
  for (int o = 0; o < N; ++o)
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (not_finite(x[o][i])) bad |= 1u << o;
  bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
  for (int o = 0; o < N; ++o)
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (bad >> o & 1) x[o][i] = 0;
  return bad;
}

// The words' values over the scale: a power of two, so bfloat16 holds the quotients.
template <int N, int W>
__device__ __forceinline__ void divide_words(uint32_t (&x)[N][W], int e) {
  const uint32_t inv = (uint32_t)(127 - e) << 7, bits = inv | inv << 16;
  __nv_bfloat162 f;
  memcpy(&f, &bits, 4);
#pragma unroll
  for (int o = 0; o < N; ++o)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      __nv_bfloat162 v;
      memcpy(&v, &x[o][i], 4);
      v = __hmul2(v, f);
      memcpy(&x[o][i], &v, 4);
    }
}

// Takes the marked tokens and what the largest scale cannot hold out of the words; returns the largest magnitude.
template <int N, int W>
__device__ __forceinline__ uint32_t clean(uint32_t (&w)[N][W], uint32_t &bad) {
  uint32_t most = largest(w);
  bad = 0;
  if (most >= 0x7f80u) {
    bad = mark_tokens(w);
    most = largest(w);
  }
  constexpr uint32_t kMost = 0x7f70u;  // 240 * 2^120, the largest code below 2^128 at the largest scale
  if (most > kMost) {                  // (what would be rounded up to 2^128)
#pragma unroll
    for (int o = 0; o < N; ++o)
#pragma unroll
      for (int i = 0; i < W; ++i)
        w[o][i] = (w[o][i] & 0x80008000u) | __vminu2(w[o][i] & 0x7fff7fffu, kMost | kMost << 16);
    most = kMost;
  }
  return most;
}

// The lane's codes of a token's K, two in each of c, into the token's row.
template <int W>
__device__ __forceinline__ void store_codes(uint8_t *row, int d, const uint32_t (&c)[W]) {
  if constexpr (W == 4)
    *reinterpret_cast<uint2 *>(row + (d / 16) * 128 + d % 16) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  else if constexpr (W == 2)
    *reinterpret_cast<uint32_t *>(row + (d / 16) * 128 + d % 16) = c[0] | c[1] << 16;
  else
#pragma unroll
    for (int i = 0; i < W; ++i) *reinterpret_cast<uint16_t *>(row + ((d + 2 * i) / 16) * 128 + (d + 2 * i) % 16) = (uint16_t)c[i];
}

template <int G>
__global__ void __launch_bounds__(kThreads, G >= 3 ? 1 : 2) attn_kv8_append_kernel(const AppendParams p) {
  constexpr int D = G * 64, DL = lane_dims(G), W = DL / 2;
  __shared__ int slots[kWarps][48];
  __shared__ __align__(16) int8_t place[kWarps][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool active = D % (32 * DL) == 0 || lane < D / DL;  // the lane has dims
  const int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * p.window;
  if (base >= p.T) return;
  // slots of the 15 tokens before the window (lanes 0 to 14), of the window and of the 15 behind it
  int slot[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = base - 15 + lane + 32 * i;
    slot[i] = t >= 0 && t < p.T && lane + 32 * i < p.window + 30 ? p.slots[t] : -1;
    if (slot[i] < -1 || slot[i] >= p.nslots) {  // no such slot: not written
      atomicCAS(p.status, 0, kStatusDevice);
      slot[i] = -1;
    }
    if (lane + 32 * i < 48) slots[warp][lane + 32 * i] = slot[i];
  }
  // lanes whose block none of the 15 tokens before names
  const uint32_t same = __match_any_sync(0xffffffffu, slot[0] >> 4);
  const bool mine = lane >= 15 && lane < 15 + p.window && slot[0] >= 0;
  uint32_t leads = __ballot_sync(0xffffffffu, mine && !(same & (0x7fffu << (lane - 15 & 31))));
  const int P = 1 << p.shift, u0 = blockIdx.y * p.share, u1 = min(u0 + p.share, 2 * p.H);
  for (; leads; leads &= leads - 1) {
    const int lead = __ffs(leads) - 1, head_slot = __shfl_sync(0xffffffffu, slot[0], lead);
    // which of the block's slots the call writes, and from which token
    __syncwarp();
    const int other = lane < 16 ? slots[warp][lead + lane] : -1;
    const bool member = other >= 0 && other >> 4 == head_slot >> 4;
    if (member) place[warp][other & 15] = (int8_t)lane;
    __syncwarp();
    const uint32_t writes = __reduce_or_sync(0xffffffffu, member ? 1u << (other & 15) : 0u);
    const uint4 where = *reinterpret_cast<const uint4 *>(place[warp]);
    const uint32_t at[4] = {where.x, where.y, where.z, where.w};
    const bool fresh = writes & 1;
    const int alone = __popc(writes) == 1 ? __ffs(writes) - 1 : -1;  // the block's one token
    // the usual case of a prompt: all of the block's tokens, one after the other
    const bool in_order = writes == 0xffffu && at[0] == 0x03020100u && at[1] == 0x07060504u && at[2] == 0x0b0a0908u &&
                          at[3] == 0x0f0e0d0cu;
    const int64_t t0 = base + lead - 15;
    const int block = (head_slot & (P - 1)) >> 4;
    // K's or V's words of the block's first token, and their place in the cache
    auto words_of = [&](int u) {
      return u & 1 ? p.v + (int64_t)(u >> 1) * p.vh + t0 * p.vt + lane * DL : p.k + (int64_t)(u >> 1) * p.kh + t0 * p.kt + lane * DL;
    };
    auto page_of = [&](int u) {
      return p.cache + ((int64_t)(head_slot >> p.shift) * p.H + (u >> 1)) * kv8_page_bytes(D, P);
    };
    for (int ub = u0; ub < u1; ub += kAtOnce) {
      uint32_t todo = (1u << min(u1 - ub, kAtOnce)) - 1;  // of u = ub, ub + 1, ...
      if (alone >= 0) {
        // one token, as in a decode step: several heads' loads in flight, and work for one token only
        uint32_t w[kAtOnce][1][W], was_bits[kAtOnce], was_bad[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          was_bits[k] = was_bad[k] = 0;
#pragma unroll
          for (int i = 0; i < W; ++i) w[k][0][i] = 0;
          const int u = ub + k;
          if (u >= u1) continue;
          if (active) load_words<W>(words_of(u) + (int64_t)place[warp][alone] * (u & 1 ? p.vt : p.kt), w[k][0]);
          const Kv8Tail *tail = reinterpret_cast<const Kv8Tail *>(page_of(u) + P * D + block * kv8_block_bytes(D) + D * 16);
          if (!fresh) {
            was_bits[k] = u & 1 ? tail->sv : tail->sk;
            was_bad[k] = u & 1 ? tail->vbad : tail->kbad;
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int u = ub + k;
          if (u >= u1) continue;
          uint32_t bad, c[W];
          const int k_was = fresh ? -1000 : held_exponent(was_bits[k]), e = max(scale_exponent(clean(w[k], bad)), k_was);
          if (!fresh && e > k_was) continue;  // the block's other codes are rounded again, below
          todo &= ~(1u << k);
          divide_words(w[k], e);
#pragma unroll
          for (int i = 0; i < W; ++i) c[i] = ptx::pack_e4m3x2(low_of(w[k][0][i]), high_of(w[k][0][i]));
          uint8_t *kc = page_of(u) + block * 16 * D, *vc = page_of(u) + P * D + block * kv8_block_bytes(D);
          if (active && !(u & 1)) {
            store_codes<W>(kc + (alone / 8) * 8 * D + (alone % 8) * 16, lane * DL, c);
            if (fresh) {
              const uint32_t zero[W] = {};
#pragma unroll
              for (int o = 1; o < 16; ++o) store_codes<W>(kc + (o / 8) * 8 * D + (o % 8) * 16, lane * DL, zero);
            }
          } else if (active) {
#pragma unroll
            for (int d = 0; d < DL; ++d) {
              const uint32_t code = c[d / 2] >> (8 * (d & 1)) & 0xff;
              uint8_t *to = vc + (lane * DL + d) * 16;
              if (fresh)
                *reinterpret_cast<uint4 *>(to) = make_uint4(code, 0, 0, 0);
              else
                to[alone] = (uint8_t)code;
            }
          }
          if (lane == 0) {
            Kv8Tail *tail = reinterpret_cast<Kv8Tail *>(vc + D * 16);
            (u & 1 ? tail->sv : tail->sk) = float_bits_of(e);
            (u & 1 ? tail->vbad : tail->kbad) = (uint16_t)((was_bad[k] & ~writes) | bad << alone);
            if (u & 1) tail->zero = 0;
          }
        }
      }
      for (; todo; todo &= todo - 1) {
        const int u = ub + __ffs(todo) - 1;
        const bool is_v = u & 1;
        const __nv_bfloat16 *x = words_of(u);
        const int64_t stride = is_v ? p.vt : p.kt;
        uint8_t *page = page_of(u);
        uint8_t *kc = page + block * 16 * D, *vc = page + P * D + block * kv8_block_bytes(D);
        Kv8Tail *tail = reinterpret_cast<Kv8Tail *>(vc + D * 16);
        uint32_t was_bits = 0, was_bad = 0;
        if (!fresh) {
          was_bits = is_v ? tail->sv : tail->sk;
          was_bad = is_v ? tail->vbad : tail->kbad;
        }
        const int k_was = fresh ? -1000 : held_exponent(was_bits);
        const bool merge = is_v && !fresh && writes != 0xffffu;  // some of V's codes stay
        uint32_t w[16][W];
        if (in_order) {
#pragma unroll
          for (int o = 0; o < 16; ++o) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[o][i] = 0;
            if (active) load_words<W>(x, w[o]);
            x += stride;
          }
        } else {
#pragma unroll
          for (int o = 0; o < 16; ++o) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[o][i] = 0;
            if (active && writes >> o & 1) load_words<W>(x + (int64_t)(at[o >> 2] >> (8 * (o & 3)) & 0xff) * stride, w[o]);
          }
        }
        uint32_t bad;
        const int e = max(scale_exponent(clean(w, bad)), k_was);
        const bool shift = !fresh && e > k_was;  // (warp-uniform)
        const __half2 f = __float2half2_rn(e - k_was > 24 ? 0.f : __uint_as_float(float_bits_of(k_was - e)));
        divide_words(w, e);
        if (!is_v) {
          if (shift) {  // the codes of the block's other tokens, 16 bytes a step
#pragma unroll 1
            for (int i = lane; i < D; i += 32) {  // word i: group of 8 tokens, 16 dims, token
              if (writes >> ((i / (D / 2)) * 8 + i % 8) & 1) continue;
              uint4 *c = reinterpret_cast<uint4 *>(kc) + i;
              uint4 v = *c;
              v.x = shift_codes(v.x, f); v.y = shift_codes(v.y, f); v.z = shift_codes(v.z, f); v.w = shift_codes(v.w, f);
              *c = v;
            }
          }
          const uint32_t stores = !active ? 0 : fresh ? 0xffffu : writes;
#pragma unroll
          for (int o = 0; o < 16; ++o) {
            if (!(stores >> o & 1)) continue;
            uint8_t *row = kc + (o / 8) * 8 * D + (o % 8) * 16;
            uint32_t c[W];
#pragma unroll
            for (int i = 0; i < W; ++i) c[i] = ptx::pack_e4m3x2(low_of(w[o][i]), high_of(w[o][i]));
            store_codes<W>(row, lane * DL, c);
          }
        } else {
          // a lane's dims, 16 tokens each
          auto codes4 = [&](int d, int i) {  // of dim d, tokens 4 i ...
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = d & 1 ? high_of(w[4 * i + j][d / 2]) : low_of(w[4 * i + j][d / 2]);
            return ptx::pack_e4m3x2(y[0], y[1]) | ptx::pack_e4m3x2(y[2], y[3]) << 16;
          };
          if (!active) {
          } else if (merge && !shift && __popc(writes) <= 2) {
            // two tokens: their bytes alone
#pragma unroll
            for (int o = 0; o < 16; ++o) {
              if (!(writes >> o & 1)) continue;
#pragma unroll
              for (int i = 0; i < W; ++i) {
                const uint32_t c = ptx::pack_e4m3x2(low_of(w[o][i]), high_of(w[o][i]));
                vc[(lane * DL + 2 * i) * 16 + o] = (uint8_t)c;
                vc[(lane * DL + 2 * i + 1) * 16 + o] = (uint8_t)(c >> 8);
              }
            }
          } else if (!merge) {
#pragma unroll
            for (int d = 0; d < DL; ++d)
              *reinterpret_cast<uint4 *>(vc + (lane * DL + d) * 16) = make_uint4(codes4(d, 0), codes4(d, 1), codes4(d, 2), codes4(d, 3));
          } else {
            uint32_t mask[4];  // bytes of the tokens that the call writes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t nib = writes >> (4 * i) & 15u;
              mask[i] = ((nib & 1) | (nib & 2) << 7 | (nib & 4) << 14 | (nib & 8) << 21) * 0xffu;
            }
            uint4 rows[DL];
#pragma unroll
            for (int d = 0; d < DL; ++d) rows[d] = *reinterpret_cast<const uint4 *>(vc + (lane * DL + d) * 16);
#pragma unroll
            for (int d = 0; d < DL; ++d) {
              uint32_t held[4] = {rows[d].x, rows[d].y, rows[d].z, rows[d].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (shift) held[i] = shift_codes(held[i], f);
                held[i] = (codes4(d, i) & mask[i]) | (held[i] & ~mask[i]);
              }
              *reinterpret_cast<uint4 *>(vc + (lane * DL + d) * 16) = make_uint4(held[0], held[1], held[2], held[3]);
            }
          }
        }
        if (lane == 0) {
          (is_v ? tail->sv : tail->sk) = float_bits_of(e);
          (is_v ? tail->vbad : tail->kbad) = (uint16_t)((was_bad & ~writes) | bad);
          if (is_v) tail->zero = 0;
        }
      }
    }
  }
}

struct ReadParams {
  const uint8_t *cache;
  const int *slots;
  __nv_bfloat16 *k, *v;
  int64_t kh, kt, vh, vt;  // element strides of head and token
  int64_t nslots;
  int T, H, shift;
  int window;  // tokens of a warp
  int share;   // (head, side) pairs of a warp
  int *status;
};

// Two codes as bfloat16: a code times a power of two is exact.
__device__ __forceinline__ uint32_t values2(uint32_t codes, float scale) {
  const uint32_t h = halves_of_e4m3x2(codes);
  __half2 x;
  memcpy(&x, &h, 4);
  const float2 y = __half22float2(x);
  return ptx::pack_bf16x2(y.x * scale, y.y * scale);
}

template <int W>
__device__ __forceinline__ void store_words(__nv_bfloat16 *to, const uint32_t (&w)[W]) {
  if constexpr (W == 4)
    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (W == 2)
    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
  else
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t *>(to)[i] = w[i];
}

// A warp has runs of tokens whose slots follow one another in a block (16 tokens at
// most), of K or V of some heads: K's rows as they are, V's rows of 16 tokens
// turned in registers.
template <int G>
__global__ void __launch_bounds__(kThreads) attn_kv8_read_kernel(const ReadParams p) {
  constexpr int D = G * 64, DL = lane_dims(G), W = DL / 2;
  constexpr uint32_t kNaN2 = 0x7fff7fffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool active = D % (32 * DL) == 0 || lane < D / DL;  // the lane has dims
  const int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * p.window;
  if (base >= p.T) return;
  // lane 0: the token before the window, lane 1 on: the window and the 15 tokens behind it
  const int64_t mine = base - 1 + lane;
  int slot = mine >= 0 && mine < p.T && lane < p.window + 16 ? p.slots[mine] : -1;
  if (slot < -1 || slot >= p.nslots) {
    atomicCAS(p.status, 0, kStatusDevice);
    slot = -1;
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  const uint32_t goes_on = __ballot_sync(0xffffffffu, lane > 0 && before >= 0 && slot == before + 1 && (slot & 15) != 0);
  uint32_t heads = __ballot_sync(0xffffffffu, lane > 0 && lane <= p.window && mine < p.T) & ~goes_on;
  const int P = 1 << p.shift, u0 = blockIdx.y * p.share, u1 = min(u0 + p.share, 2 * p.H);
  for (; heads; heads &= heads - 1) {
    const int head = __ffs(heads) - 1, s = __shfl_sync(0xffffffffu, slot, head);
    const int64_t t0 = base - 1 + head;
    const int off = s & 15, n = s < 0 ? 1 : __ffs(~(goes_on >> head >> 1));  // tokens of the run
    const int block = (s & (P - 1)) >> 4;
    for (int u = u0; u < u1; ++u) {
      const int h = u >> 1;
      const bool is_v = u & 1;
      __nv_bfloat16 *to = (is_v ? p.v : p.k) + (int64_t)h * (is_v ? p.vh : p.kh) + lane * DL;
      const int64_t stride = is_v ? p.vt : p.kt;
      to += t0 * stride;
      if (!active) continue;
      if (s < 0) {
        const uint32_t zero[W] = {};
        store_words<W>(to, zero);
        continue;
      }
      const uint8_t *page = p.cache + ((int64_t)(s >> p.shift) * p.H + h) * kv8_page_bytes(D, P);
      const uint8_t *kc = page + block * 16 * D, *vc = page + P * D + block * kv8_block_bytes(D);
      const Kv8Tail tail = *reinterpret_cast<const Kv8Tail *>(vc + D * 16);
      to -= off * stride;
      const uint32_t reads = (0xffffffffu >> (32 - n)) << off;
      if (!is_v) {
        const float scale = __uint_as_float(tail.sk);
        uint32_t c[16][W];
        const int d = lane * DL;
#pragma unroll
        for (int o = 0; o < 16; ++o) {
          if (!(reads >> o & 1)) continue;
          const uint8_t *row = kc + (o / 8) * 8 * D + (o % 8) * 16;
          if constexpr (W == 4) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row + (d / 16) * 128 + d % 16);
            c[o][0] = x.x; c[o][1] = x.x >> 16; c[o][2] = x.y; c[o][3] = x.y >> 16;
          } else if constexpr (W == 2) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(row + (d / 16) * 128 + d % 16);
            c[o][0] = x; c[o][1] = x >> 16;
          } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
              c[o][i] = *reinterpret_cast<const uint16_t *>(row + ((d + 2 * i) / 16) * 128 + (d + 2 * i) % 16);
          }
        }
#pragma unroll
        for (int o = 0; o < 16; ++o) {
          if (!(reads >> o & 1)) continue;
          uint32_t y[W];
#pragma unroll
          for (int i = 0; i < W; ++i) y[i] = tail.kbad >> o & 1 ? kNaN2 : values2(c[o][i], scale);
          store_words<W>(to + o * stride, y);
        }
      } else {
        const float scale = __uint_as_float(tail.sv);
        uint32_t rows[DL][4];
#pragma unroll
        for (int d = 0; d < DL; ++d) {
          const uint4 x = *reinterpret_cast<const uint4 *>(vc + (lane * DL + d) * 16);
          rows[d][0] = x.x; rows[d][1] = x.y; rows[d][2] = x.z; rows[d][3] = x.w;
        }
#pragma unroll
        for (int o = 0; o < 16; ++o) {
          if (!(reads >> o & 1)) continue;
          uint32_t y[W];
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const uint32_t two = __byte_perm(rows[2 * i][o >> 2], rows[2 * i + 1][o >> 2], (o & 3) | (4 + (o & 3)) << 4);
            y[i] = tail.vbad >> o & 1 ? kNaN2 : values2(two, scale);
          }
          store_words<W>(to + o * stride, y);
        }
      }
    }
  }
}

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The checks append and read share.
int check_cache(const void *cache, int num_pages, int H, int D, int P, int T, const int *slots) {
  if (T > 0x7fffffff - 4 * kThreads) return ATTN_ERR_ARG;  // a CTA's tokens are numbered past the last
  if (num_pages < 0 || T < 0 || H < 1 || H > 65535 || kv4_page_shift(P) < 0) return ATTN_ERR_ARG;
  if (D < 64 || D > ATTN_KV8_MAX_HEAD_DIM || D % 64 != 0) return ATTN_ERR_ARG;
  if ((int64_t)num_pages * P > 0x7fffffffLL) return ATTN_ERR_ARG;  // slots are 32-bit
  if (T == 0) return ATTN_OK;
  if (!slots || (num_pages > 0 && !cache)) return ATTN_ERR_ARG;
  if (off16(cache) || (reinterpret_cast<uintptr_t>(slots) & 3u)) return ATTN_ERR_ALIGN;
  return ATTN_OK;
}

// Strides of one [T, H, D] view.
int check_view(const void *x, long long t, long long h) {
  if (!x || t < 0 || h < 0) return ATTN_ERR_ARG;
  return off16(x) || t % 8 || h % 8 ? ATTN_ERR_ALIGN : ATTN_OK;
}

// The CTAs for windows of `window` tokens a warp, the (head, side) pairs spread over gridDim.y. Single tokens of many
// requests each have a block of their own, which a warp takes one after the other, so a window is short where there
// are few tokens; a prompt's tokens share blocks. Windows of 1 / 4 / 16 tokens, us (8 heads of 128):
//   append, 64 requests of one token 3.2 / 6.8 / 16.5, 256 of one 7.0 / 7.2 / 21.2, 1024 of one 15.3 / 17.5 / 21.6,
//     64 of 16 tokens 9.6 / 7.1 / 5.4, 512 of 4 24.0 / 15.5 / 15.0, 16384 tokens of 8 45 / 38 / 20;
//   read, 1024 slots 4.8 / 3.9 / 4.8, 4096 10.2 / 7.8 / 8.8, 5003 (16 heads of 64) 16.4 / 10.2 / 7.1, 16399 33 / 26 / 16.5.
dim3 cache_grid(int T, int H, int sms, int window, int *share) {
  const int x = (T + kWarps * window - 1) / (kWarps * window);
  const int64_t most = 8 * (int64_t)sms;  // CTAs, about
  int64_t y = (most + x - 1) / x;
  y = y < 1 ? 1 : y > 2 * H ? 2 * H : y;
  *share = (int)((2 * H + y - 1) / y);
  return dim3((unsigned)x, (unsigned)((2 * H + *share - 1) / *share));
}

template <typename F>
void by_head_dim(int D, F &&f) {
  switch (D / 64) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    default: f(std::integral_constant<int, 4>()); break;
  }
}

}  // namespace
}  // namespace attn

extern "C" {

long long attn_kv8_page_bytes(int D, int page_size) {
  if (D < 64 || D > ATTN_KV8_MAX_HEAD_DIM || D % 64 != 0 || attn::kv4_page_shift(page_size) < 0) return ATTN_ERR_ARG;
  return attn::kv8_page_bytes(D, page_size);
}

int attn_kv8_append(const void *k, long long k_stride_t, long long k_stride_h, const void *v, long long v_stride_t,
                    long long v_stride_h, const int *slots, void *cache, int num_pages, int T, int Hkv, int D,
                    int page_size, attn_stream_t stream) {
  using namespace attn;
  int rc = check_cache(cache, num_pages, Hkv, D, page_size, T, slots);
  if (rc != ATTN_OK || T == 0) return rc;
  if ((rc = check_view(k, k_stride_t, k_stride_h)) != ATTN_OK) return rc;
  if ((rc = check_view(v, v_stride_t, v_stride_h)) != ATTN_OK) return rc;
  int device = 0, sms = 0;
  AppendParams p{};
  if ((rc = current_device(&device, &sms, &p.status)) != ATTN_OK) return rc;
  p.k = static_cast<const __nv_bfloat16 *>(k);
  p.v = static_cast<const __nv_bfloat16 *>(v);
  p.kt = k_stride_t; p.kh = k_stride_h; p.vt = v_stride_t; p.vh = v_stride_h;
  p.slots = slots;
  p.cache = static_cast<uint8_t *>(cache);
  p.nslots = (int64_t)num_pages * page_size;
  p.T = T; p.H = Hkv; p.shift = kv4_page_shift(page_size);
  p.window = T <= 256 ? 1 : T <= 4096 ? 4 : kMostWindow;
  const dim3 grid = cache_grid(T, Hkv, sms, p.window, &p.share);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  by_head_dim(D, [&](auto g) { attn_kv8_append_kernel<g.value><<<grid, kThreads, 0, st>>>(p); });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

int attn_kv8_read(const void *cache, int num_pages, const int *slots, void *k, long long k_stride_h,
                  long long k_stride_t, void *v, long long v_stride_h, long long v_stride_t, int T, int Hkv, int D,
                  int page_size, attn_stream_t stream) {
  using namespace attn;
  int rc = check_cache(cache, num_pages, Hkv, D, page_size, T, slots);
  if (rc != ATTN_OK || T == 0) return rc;
  if ((rc = check_view(k, k_stride_t, k_stride_h)) != ATTN_OK) return rc;
  if ((rc = check_view(v, v_stride_t, v_stride_h)) != ATTN_OK) return rc;
  int device = 0, sms = 0;
  ReadParams p{};
  if ((rc = current_device(&device, &sms, &p.status)) != ATTN_OK) return rc;
  p.cache = static_cast<const uint8_t *>(cache);
  p.slots = slots;
  p.k = static_cast<__nv_bfloat16 *>(k);
  p.v = static_cast<__nv_bfloat16 *>(v);
  p.kh = k_stride_h; p.kt = k_stride_t; p.vh = v_stride_h; p.vt = v_stride_t;
  p.nslots = (int64_t)num_pages * page_size;
  p.T = T; p.H = Hkv; p.shift = kv4_page_shift(page_size);
  p.window = T <= 4096 ? 4 : kMostWindow;
  const dim3 grid = cache_grid(T, Hkv, sms, p.window, &p.share);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  by_head_dim(D, [&](auto g) { attn_kv8_read_kernel<g.value><<<grid, kThreads, 0, st>>>(p); });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // extern "C"
