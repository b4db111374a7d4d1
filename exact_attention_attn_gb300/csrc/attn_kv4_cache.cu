// The 4-bit KV cache: quantising tokens into their slots, and reading slots
// back as bfloat16.
//
// Per token, kv head and 64 dims:  m = min x,  s = (max x - m) / 15 as bfloat16
// (of the float32 product ((max x - m) / 16) (16 / 15)),
// c = rint((x - m) / s) in 0 .. 15 (0 where s = 0); the cache holds c in four
// bits and (s, m) as bfloat16.  m is one of the bfloat16 inputs, so it is
// held exactly; s is rounded to nearest once.  A group that holds an infinity
// or a NaN gets s = m = NaN, so that attention over it is NaN as it would be
// over the unquantised values.
//
// The differences are formed on x / 16, so that max - min of finite values
// stays finite; the factor is a power of two and leaves every result alone.
// The quotient comes from one reciprocal of the group's scale, corrected by its
// exact residual (q0 = d r, q = q0 + (d - q0 s) r: Markstein's correction, IBM
// J. Res. Dev. 34, 1990), three operations instead of a division's ten; groups
// whose scale is so small or large that these could leave the normal range
// divide.
//
// Eight threads share a group (16 bytes of bfloat16 each, one 4-byte word of
// codes); 32 consecutive tokens share a CTA, so that a warp writes four
// neighbouring rows and pairs.  Bytes: 2 + 0.5625 a value.  Bound: the issue of
// instructions for append (16384 tokens of 8 heads of 128, 86 MB: 19.4 us, 4.4
// TB/s, issue slots 74 % busy before the last reduction; 36 us as first written,
// with divisions), HBM for read (the same 86 MB in 12.7 us, 6.8 TB/s).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 8;  // tokens of a CTA

struct AppendParams {
  const __nv_bfloat16 *k, *v;
  int64_t kt, kh, vt, vh;  // element strides of token and head
  const int *slots;
  uint8_t *cache;
  int64_t nslots;
  int T, H, G, shift;
  int share;  // (head, group) pairs of a CTA
  int *status;
};

// Codes and pair of one group of 64 values, 8 of them (w) in each of 8 lanes.
__device__ __forceinline__ void quantise8(const uint4 &w, uint32_t &codes, uint32_t &pair) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  __nv_bfloat162 h[4];
  memcpy(h, ws, sizeof(ws));
  // minimum and maximum of the lane's values, NaN where there is one
  __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
  __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  __nv_bfloat162 a = __halves2bfloat162(__low2bfloat16(lo2), __hneg(__low2bfloat16(hi2)));
  __nv_bfloat162 b = __halves2bfloat162(__high2bfloat16(lo2), __hneg(__high2bfloat16(hi2)));
  __nv_bfloat162 r = __hmin2_nan(a, b);  // (min, -max): one minimum reduces both
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    uint32_t u;
    memcpy(&u, &r, 4);
    u = __shfl_xor_sync(0xffffffffu, u, o);
    __nv_bfloat162 t;
    memcpy(&t, &u, 4);
    r = __hmin2_nan(r, t);
  }
  const float lo = __low2float(r) * 0.0625f, hi = -__high2float(r) * 0.0625f;
  // ((max - min) / 16) / (15 / 16), by the reciprocal: one product, whose rounding also decides where the value is
  // halfway between two bfloat16 numbers
  const float d = hi - lo;
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(d, 1.f / 0.9375f));
  const float s = __bfloat162float(sb) * 0.0625f;
  uint16_t sbits, mbits;
  memcpy(&sbits, &sb, 2);
  const __nv_bfloat16 mb = __low2bfloat16(r);
  memcpy(&mbits, &mb, 2);
  codes = 0;
  if (!(d < INFINITY)) {
    pair = 0x7fff7fffu;  // NaN, NaN
    return;
  }
  pair = sbits | ((uint32_t)mbits << 16);
  if (s == 0.f) return;
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
  if (s < 0x1p-90f || s > 0x1p90f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float(i & 1 ? ws[i >> 1] & 0xffff0000u : ws[i >> 1] << 16);
      const float q = fminf(fmaf(x, 0.0625f, -lo) / s, 15.f);  // a subnormal scale may be rounded down by a third
      codes |= (__float_as_uint(q + kMagic) & 15u) << (4 * i);
    }
    return;
  }
  // Two values per packed operation.  With inv = 1 / s to a few units in its last
  // place, the residual e - q0 s is exact, so its correction leaves an error far
  // below the last place of the quotient (and none where the quotient is a short
  // number).  The quotient is at most 15 (1 + 2^-8), so no code passes 15.
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const uint64_t k16 = ptx::f2_pack(0.0625f, 0.0625f), nlo = ptx::f2_pack(-lo, -lo), ns = ptx::f2_pack(-s, -s);
  const uint64_t vi = ptx::f2_pack(inv, inv), zero = ptx::f2_pack(0.f, 0.f), magic = ptx::f2_pack(kMagic, kMagic);
  uint32_t sum = 0, base = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = ptx::f2_pack(__uint_as_float(ws[i] << 16), __uint_as_float(ws[i] & 0xffff0000u));
    const uint64_t e = ptx::f2_fma(x, k16, nlo);
    const uint64_t q0 = ptx::f2_fma(e, vi, zero);
    const uint64_t q = ptx::f2_fma(ptx::f2_fma(q0, ns, e), vi, q0);
    float t0, t1;
    ptx::f2_unpack(ptx::f2_add(q, magic), t0, t1);
    // the bits of 1.5 * 2^23 + c are those of 1.5 * 2^23, plus c: they are summed in place and taken off once
    sum += __float_as_uint(t0) * (1u << (8 * i)) + __float_as_uint(t1) * (16u << (8 * i));
    base += 0x4b400000u * (1u << (8 * i)) + 0x4b400000u * (16u << (8 * i));
  }
  codes = sum - base;
}

__global__ void __launch_bounds__(kThreads) attn_kv4_append_kernel(const AppendParams p) {
  const int t = blockIdx.x * kTokens + (threadIdx.x >> 3), sub = threadIdx.x & 7;
  int slot = t < p.T ? p.slots[t] : -1;
  if (slot >= p.nslots || slot < -1) {  // no such slot: not written
    atomicCAS(p.status, 0, kStatusDevice);
    slot = -1;
  }
  const int P = 1 << p.shift, row = slot & (P - 1), side = kv4_side_bytes(p.G, P);
  // The CTA's groups, one after the other: (head, group) pairs [hg, end).  The
  // addresses advance by additions (a multiplication and a division for each
  // group were a third of the instructions).  Lanes without a slot stay for the
  // shuffles, on zeros.
  int hg = blockIdx.y * p.share;
  const int end = min(hg + p.share, p.H * p.G);
  int h = hg / p.G, g = hg - h * p.G;
  const __nv_bfloat16 *k = p.k + (int64_t)t * p.kt + (int64_t)h * p.kh + g * kKv4Group + sub * 8;
  const __nv_bfloat16 *v = p.v + (int64_t)t * p.vt + (int64_t)h * p.vh + g * kKv4Group + sub * 8;
  const int64_t k_next = p.kh - (p.G - 1) * kKv4Group, v_next = p.vh - (p.G - 1) * kKv4Group;  // to the next head
  uint8_t *head = p.cache + ((int64_t)(slot >> p.shift) * p.H + h) * kv4_page_bytes(p.G, P);
  for (; hg < end; ++hg) {
    uint4 wk = make_uint4(0, 0, 0, 0), wv = wk;
    if (slot >= 0) {
      wk = *reinterpret_cast<const uint4 *>(k);
      wv = *reinterpret_cast<const uint4 *>(v);
    }
    uint32_t ck, pk, cv, pv;
    quantise8(wk, ck, pk);
    quantise8(wv, cv, pv);
    if (slot >= 0) {
      uint8_t *codes = head + (g * P + row) * kKv4RowBytes + sub * 4;
      uint8_t *pairs = head + kv4_codes_bytes(p.G, P) + (g * P + row) * kKv4PairBytes;
      *reinterpret_cast<uint32_t *>(codes) = ck;
      *reinterpret_cast<uint32_t *>(codes + side) = cv;
      if (sub == 0) {
        *reinterpret_cast<uint32_t *>(pairs) = pk;
        *reinterpret_cast<uint32_t *>(pairs + side) = pv;
      }
    }
    if (++g == p.G) {
      g = 0;
      k += k_next;
      v += v_next;
      head += kv4_page_bytes(p.G, P);
    } else {
      k += kKv4Group;
      v += kKv4Group;
    }
  }
}

struct ReadParams {
  const uint8_t *cache;
  const int *slots;
  __nv_bfloat16 *k, *v;
  int64_t kh, kt, vh, vt;  // element strides of head and token
  int64_t nslots;
  int T, H, G, shift;
  int share;  // (head, group) pairs of a CTA
  int *status;
};

// The 8 values of a word of codes.  A code behind the exponent of 2^23 is the
// float 2^23 + c, so a byte permutation and a subtraction convert it (the
// conversion instruction has a quarter of their rate).
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t pair) {
  const float s = __uint_as_float(pair << 16), m = __uint_as_float(pair & 0xffff0000u);
  const uint64_t s2 = ptx::f2_pack(s, s), m2 = ptx::f2_pack(m, m), bias = ptx::f2_pack(-8388608.f, -8388608.f);
  const uint32_t even = codes & 0x0f0f0f0fu, odd = (codes >> 4) & 0x0f0f0f0fu;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c0 = __uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440u + i));
    const float c1 = __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440u + i));
    // c * s is exact: one rounding, then bfloat16's
    const uint64_t x = ptx::f2_fma(ptx::f2_add(ptx::f2_pack(c0, c1), bias), s2, m2);
    float x0, x1;
    ptx::f2_unpack(x, x0, x1);
    out[i] = ptx::pack_bf16x2(x0, x1);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kThreads) attn_kv4_read_kernel(const ReadParams p) {
  const int t = blockIdx.x * kTokens + (threadIdx.x >> 3), sub = threadIdx.x & 7;
  if (t >= p.T) return;
  int slot = p.slots[t];
  if (slot >= p.nslots || slot < -1) {
    atomicCAS(p.status, 0, kStatusDevice);
    slot = -1;
  }
  const int P = 1 << p.shift, row = slot & (P - 1), side = kv4_side_bytes(p.G, P);
  int hg = blockIdx.y * p.share;
  const int end = min(hg + p.share, p.H * p.G);
  int h = hg / p.G, g = hg - h * p.G;
  __nv_bfloat16 *k = p.k + (int64_t)t * p.kt + (int64_t)h * p.kh + g * kKv4Group + sub * 8;
  __nv_bfloat16 *v = p.v + (int64_t)t * p.vt + (int64_t)h * p.vh + g * kKv4Group + sub * 8;
  const int64_t k_next = p.kh - (p.G - 1) * kKv4Group, v_next = p.vh - (p.G - 1) * kKv4Group;  // to the next head
  const uint8_t *head = p.cache + ((int64_t)(slot >> p.shift) * p.H + h) * kv4_page_bytes(p.G, P);
#pragma unroll 2
  for (; hg < end; ++hg) {
    uint32_t ck = 0, cv = 0, pk = 0, pv = 0;  // the pair (0, 0) stands for zeros
    if (slot >= 0) {
      const uint8_t *codes = head + (g * P + row) * kKv4RowBytes + sub * 4;
      const uint8_t *pairs = head + kv4_codes_bytes(p.G, P) + (g * P + row) * kKv4PairBytes;
      ck = *reinterpret_cast<const uint32_t *>(codes);
      cv = *reinterpret_cast<const uint32_t *>(codes + side);
      pk = *reinterpret_cast<const uint32_t *>(pairs);
      pv = *reinterpret_cast<const uint32_t *>(pairs + side);
    }
    *reinterpret_cast<uint4 *>(k) = values8(ck, pk);
    *reinterpret_cast<uint4 *>(v) = values8(cv, pv);
    if (++g == p.G) {
      g = 0;
      k += k_next;
      v += v_next;
      head += kv4_page_bytes(p.G, P);
    } else {
      k += kKv4Group;
      v += kKv4Group;
    }
  }
}

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The checks append and read share.
int check_cache(const void *cache, int num_pages, int H, int D, int P, int T, const int *slots) {
  if (T > 0x7fffffff - kTokens) return ATTN_ERR_ARG;  // a CTA's tokens are numbered past the last
  if (num_pages < 0 || T < 0 || H < 1 || H > 65535 || kv4_page_shift(P) < 0) return ATTN_ERR_ARG;
  if (D < 64 || D > ATTN_MAX_HEAD_DIM || D % 64 != 0) return ATTN_ERR_ARG;
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

// 32 tokens a CTA; the (head, group) pairs are spread over gridDim.y CTAs, as
// many as give each SM 8 CTAs (4 and 16: within 3 % either way).
dim3 cache_grid(int T, int HG, int sms, int *share) {
  const int x = (T + kTokens - 1) / kTokens;
  int y = (8 * sms + x - 1) / x;
  y = y < 1 ? 1 : y > HG ? HG : y;
  *share = (HG + y - 1) / y;
  return dim3((unsigned)x, (unsigned)((HG + *share - 1) / *share));
}

}  // namespace
}  // namespace attn

extern "C" {

long long attn_kv4_page_bytes(int D, int page_size) {
  if (D < 64 || D > ATTN_MAX_HEAD_DIM || D % 64 != 0 || attn::kv4_page_shift(page_size) < 0) return ATTN_ERR_ARG;
  return attn::kv4_page_bytes(D / 64, page_size);
}

int attn_kv4_append(const void *k, long long k_stride_t, long long k_stride_h, const void *v, long long v_stride_t,
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
  p.T = T; p.H = Hkv; p.G = D / 64; p.shift = kv4_page_shift(page_size);
  const dim3 grid = cache_grid(T, Hkv * p.G, sms, &p.share);
  attn_kv4_append_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

int attn_kv4_read(const void *cache, int num_pages, const int *slots, void *k, long long k_stride_h,
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
  p.T = T; p.H = Hkv; p.G = D / 64; p.shift = kv4_page_shift(page_size);
  const dim3 grid = cache_grid(T, Hkv * p.G, sms, &p.share);
  attn_kv4_read_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // extern "C"
