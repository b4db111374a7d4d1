// Rotary positions with several axes (time, height, width, ...) on q and k in
// one launch, forward and backward.
//
// Frequency i of a head's first rot dims turns the pair (x1, x2) by the angle
// pos[axis(i)] * theta_i:
//     y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin,
// the pair being dims (i, i + rot/2) or, with adjacent pairs, (2i, 2i + 1);
// dims from rot on pass through.  The matrix is a rotation, so the gradient is
// the rotation by the opposite angle.
//
// The angle.  A float32 angle of position 10^6 is off by 0.03 rad, and float64
// arithmetic is scarce on this chip.  The table holds theta_i / (2 pi) modulo
// one turn as a 64-bit binary fraction f, rounded to nearest from the exact
// value (whole turns of a large theta take no bits of it), so pos * f modulo
// 2^64 (one integer multiply, wrapping) is the angle in turns without any
// rounding but the table's: |pos| * 2^-65, at most 2^-34 turns for an int32
// position.  Its upper 32 bits, read as a signed number, are the angle in
// [-1/2, 1/2) turns; sincospif takes it as x = 2 * turns, a float32: 2^-26 turns.
//
// Work split.  A CTA takes NT tokens of one batch row, forms their rot/2 cos
// and sin once in shared memory, and each thread then holds the 8 pairs of one
// (token, 16-dim task) in registers while it walks over its share of the
// heads: the trigonometry is paid once per token, not once per head, and the
// rest is 16-byte loads and stores (bound: HBM, 4 bytes per element).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "attn.h"
#include "attn_internal.h"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxRot = ATTN_MAX_HEAD_DIM;

struct RopeTensor {
  const __nv_bfloat16 *x;
  __nv_bfloat16 *y;
  int64_t xb, xh, xn, yb, yh, yn;  // element strides of batch, head, token
  int heads;
};

struct RopeParams {
  RopeTensor t[2];  // q, k
  const int *pos;
  int64_t pos_a, pos_b;  // element strides of axis and batch
  const longlong2 *table;
  int N, D, rot, axes, adjacent;
  float sign;  // +1 forward, -1 backward
  int nt, lanes;  // tokens and head lanes per CTA
  int nblocks;    // CTAs per batch row
  int *status;
};

__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(ws[i] << 16);
    f[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 w;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  memcpy(&w, h, sizeof(w));
  return w;
}

template <bool ADJ>
__global__ void __launch_bounds__(kThreads) attn_rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs[];  // [nt][rot / 2]
  const int half = p.rot >> 1, tasks = p.D >> 4, rtasks = p.rot >> 4;
  const int b = blockIdx.x / p.nblocks, n0 = (blockIdx.x % p.nblocks) * p.nt;
  const int task = threadIdx.x % tasks, rest = threadIdx.x / tasks;
  const int nl = rest % p.nt, lane = rest / p.nt, n = n0 + nl;
  const bool active = lane < p.lanes && n < p.N;
  const bool turn = task < rtasks;
  // the task's two chunks of 8 dims
  const int d0 = turn && !ADJ ? task * 8 : task * 16, d1 = turn && !ADJ ? task * 8 + half : task * 16 + 8;
  for (int i = threadIdx.x; i < p.nt * half; i += kThreads) {
    const int m = n0 + i / half;
    if (m >= p.N) break;
    const longlong2 e = p.table[i % half];
    int axis = (int)e.y;
    if ((unsigned long long)e.y >= (unsigned long long)p.axes) {  // not a table of this call's axes
      atomicCAS(p.status, 0, kStatusDevice);
      axis = 0;
    }
    const int64_t pos = p.pos[axis * p.pos_a + b * p.pos_b + m];
    const uint64_t turns = (uint64_t)pos * (uint64_t)e.x;
    float s, c;
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c, p.sign * s);
  }
  __syncthreads();
  if (!active) return;
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = cs[nl * half + task * 8 + i];
      c[i] = v.x;
      s[i] = v.y;
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const RopeTensor &t = p.t[w];
    if (t.heads == 0 || (!turn && t.x == t.y)) continue;  // in place: the passed dims are there already
    const __nv_bfloat16 *x = t.x + b * t.xb + n * t.xn;
    __nv_bfloat16 *y = t.y + b * t.yb + n * t.yn;
#pragma unroll 1
    for (int h = lane; h < t.heads; h += p.lanes) {
      uint4 u = *reinterpret_cast<const uint4 *>(x + h * t.xh + d0);
      uint4 v = *reinterpret_cast<const uint4 *>(x + h * t.xh + d1);
      if (turn) {
        float a[8], e[8], r0[8], r1[8];
        unpack8(u, a);
        unpack8(v, e);
        if (ADJ) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            r0[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
            r0[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
            r1[2 * i] = e[2 * i] * c[i + 4] - e[2 * i + 1] * s[i + 4];
            r1[2 * i + 1] = e[2 * i + 1] * c[i + 4] + e[2 * i] * s[i + 4];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r0[i] = a[i] * c[i] - e[i] * s[i];
            r1[i] = e[i] * c[i] + a[i] * s[i];
          }
        }
        u = pack8(r0);
        v = pack8(r1);
      }
      *reinterpret_cast<uint4 *>(y + h * t.yh + d0) = u;
      *reinterpret_cast<uint4 *>(y + h * t.yh + d1) = v;
    }
  }
}

// 1 / (2 pi) to kTurnWords * 32 binary places, most significant word last; a
// double's whole turns (up to 2^971 of its last bits) are taken off by it.
constexpr int kTurnWords = 40;

// A number below 2^32 in fixed point: word kFixed - 1 is its whole part.
constexpr int kFixed = 45;
struct Fixed {
  uint32_t w[kFixed];
};

void divide(Fixed &a, uint32_t by) {
  uint64_t rest = 0;
  for (int i = kFixed - 1; i >= 0; --i) {
    rest = rest << 32 | a.w[i];
    a.w[i] = (uint32_t)(rest / by);
    rest %= by;
  }
}

// a += sign * times * b
void add(Fixed &a, const Fixed &b, int sign, uint32_t times) {
  int64_t carry = 0;
  for (int i = 0; i < kFixed; ++i) {
    carry += (int64_t)a.w[i] + sign * (int64_t)((uint64_t)b.w[i] * times);
    a.w[i] = (uint32_t)carry;
    carry >>= 32;
  }
}

bool below(const Fixed &a, const Fixed &b) {
  for (int i = kFixed - 1; i >= 0; --i)
    if (a.w[i] != b.w[i]) return a.w[i] < b.w[i];
  return false;
}

// a += sign * times * arctan(1 / k), by its series in 1 / k
void add_arctan(Fixed &a, uint32_t k, int sign, uint32_t times) {
  Fixed power{};
  power.w[kFixed - 1] = 1;
  divide(power, k);
  const Fixed zero{};
  for (uint32_t n = 1; below(zero, power); n += 2, sign = -sign) {
    Fixed term = power;
    divide(term, n);
    add(a, term, sign, times);
    divide(power, k * k);
  }
}

struct PerTurn {
  uint32_t w[kTurnWords];
  PerTurn() : w{} {
    Fixed turn{}, rest{};  // 2 pi = 32 arctan(1/5) - 8 arctan(1/239) (Machin)
    add_arctan(turn, 5, 1, 32);
    add_arctan(turn, 239, -1, 8);
    rest.w[kFixed - 1] = 1;
    for (int bit = kTurnWords * 32 - 1; bit >= 0; --bit) {  // long division of 1
      add(rest, Fixed(rest), 1, 1);
      if (below(rest, turn)) continue;
      add(rest, turn, -1, 1);
      w[bit / 32] |= 1u << (bit % 32);
    }
  }
};

// x / (2 pi) modulo 1 as a 64-bit fraction, to nearest.
uint64_t turns_of(double x) {
  static const PerTurn per;
  int e;
  const uint64_t m = (uint64_t)ldexp(frexp(fabs(x), &e), 53);  // |x| = m 2^(e - 53)
  uint32_t product[kTurnWords + 3] = {};  // m / (2 pi)
  unsigned __int128 carry = 0;
  for (int i = 0; i < kTurnWords + 3; ++i) {
    if (i < kTurnWords) carry += (unsigned __int128)per.w[i] * m;
    product[i] = (uint32_t)carry;
    carry >>= 32;
  }
  // the fraction's bits begin at this one of the product (those of small numbers past its end)
  const int at = kTurnWords * 32 - (e - 53) - 64;
  auto bit = [&](int i) -> uint64_t { return i < (kTurnWords + 3) * 32 ? product[i / 32] >> (i % 32) & 1 : 0; };
  uint64_t f = bit(at - 1);
  for (int i = 0; i < 64; ++i) f += bit(at + i) << i;
  return x < 0 ? 0 - f : f;
}

bool bad_align(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Fills one tensor's part of the parameters; ATTN_OK, ATTN_ERR_ARG or ATTN_ERR_ALIGN.
int set_tensor(RopeTensor *t, const void *x, const long long *xs, void *y, const long long *ys, int heads) {
  if (!x || !y || !xs || !ys) return ATTN_ERR_ARG;
  if (bad_align(x) || bad_align(y)) return ATTN_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    if (xs[i] < 0 || ys[i] < 0) return ATTN_ERR_ARG;
    if (xs[i] % 8 || ys[i] % 8) return ATTN_ERR_ALIGN;
    if (x == y && xs[i] != ys[i]) return ATTN_ERR_ARG;  // in place only with the same layout
  }
  t->x = static_cast<const __nv_bfloat16 *>(x);
  t->y = static_cast<__nv_bfloat16 *>(y);
  t->xb = xs[0]; t->xh = xs[1]; t->xn = xs[2];
  t->yb = ys[0]; t->yh = ys[1]; t->yn = ys[2];
  t->heads = heads;
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_rope_table(const double *inv_freq, const int *axis, int n, int axes, long long *table) {
  if (n < 0 || n > attn::kMaxRot / 2 || axes < 1 || axes > ATTN_ROPE_MAX_AXES) return ATTN_ERR_ARG;
  if (n > 0 && (!inv_freq || !axis || !table)) return ATTN_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    if (!isfinite(inv_freq[i]) || axis[i] < 0 || axis[i] >= axes) return ATTN_ERR_ARG;
  }
  for (int i = 0; i < n; ++i) {
    const uint64_t f = attn::turns_of(inv_freq[i]);  // modulo one turn: positions are whole numbers
    memcpy(&table[2 * i], &f, sizeof(f));
    table[2 * i + 1] = axis[i];
  }
  return ATTN_OK;
}

int attn_rope(const void *q, const long long *q_strides, void *q_out, const long long *q_out_strides, int Hq,
              const void *k, const long long *k_strides, void *k_out, const long long *k_out_strides, int Hkv,
              const int *positions, long long pos_stride_axis, long long pos_stride_b, int axes,
              const long long *table, int B, int N, int D, int rot, int adjacent, int backward,
              attn_stream_t stream) {
  using namespace attn;
  if (B < 0 || N < 0 || Hq < 0 || Hkv < 0 || axes < 1 || axes > ATTN_ROPE_MAX_AXES) return ATTN_ERR_ARG;
  if (D < 64 || D > ATTN_MAX_HEAD_DIM || D % 64 != 0) return ATTN_ERR_ARG;
  if (rot < 16 || rot > D || rot % 16 != 0) return ATTN_ERR_ARG;
  if ((adjacent != 0 && adjacent != 1) || (backward != 0 && backward != 1)) return ATTN_ERR_ARG;
  if (pos_stride_axis < 0 || pos_stride_b < 0) return ATTN_ERR_ARG;
  const int64_t heads = (int64_t)Hq + Hkv, tokens = (int64_t)B * N;
  if (N > 0x7fffffff - 8) return ATTN_ERR_ARG;  // a CTA's tokens are numbered past the last
  if (tokens == 0 || heads == 0) return ATTN_OK;
  if (tokens > ((int64_t)1 << 40) / heads) return ATTN_ERR_ARG;
  if (!positions || !table) return ATTN_ERR_ARG;
  RopeParams p{};
  int rc;
  if (Hq > 0 && (rc = set_tensor(&p.t[0], q, q_strides, q_out, q_out_strides, Hq)) != ATTN_OK) return rc;
  if (Hkv > 0 && (rc = set_tensor(&p.t[1], k, k_strides, k_out, k_out_strides, Hkv)) != ATTN_OK) return rc;
  if (bad_align(table) || (reinterpret_cast<uintptr_t>(positions) & 3u)) return ATTN_ERR_ALIGN;
  int device = 0, sms = 0;
  int *status = nullptr;
  if ((rc = current_device(&device, &sms, &status)) != ATTN_OK) return rc;
  p.pos = positions;
  p.pos_a = pos_stride_axis;
  p.pos_b = pos_stride_b;
  p.table = reinterpret_cast<const longlong2 *>(table);
  p.N = N; p.D = D; p.rot = rot; p.axes = axes; p.adjacent = adjacent;
  p.sign = backward ? -1.f : 1.f;
  p.status = status;
  // Tokens per CTA: the most (a power of two up to 4) that leaves two CTAs per
  // SM; one token per CTA where there are few tokens.  Measured on q 32 and k 8
  // heads of 128, N 8192, B 2 (336 MB): CTAs of 128 threads and 4 tokens 56.1 us
  // (88 % of a plain copy's rate), 256 threads and 8 tokens 57.3, 512 threads
  // 69.5, 256 threads and 2 tokens 83.1; two heads of a thread in flight 62.5.
  const int tasks = D / 16, fit = kThreads / tasks;
  int nt = 1;
  while (nt < 4 && nt * 2 <= fit && (int64_t)B * ((N + 2 * nt - 1) / (2 * nt)) >= 2 * sms) nt *= 2;
  p.nt = nt;
  p.lanes = fit / nt;
  p.nblocks = (N + nt - 1) / nt;
  const int64_t grid = (int64_t)B * p.nblocks;
  if (grid > 0x7fffffffLL) return ATTN_ERR_ARG;
  const size_t smem = (size_t)nt * (rot / 2) * sizeof(float2);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (adjacent)
    attn_rope_kernel<true><<<(unsigned)grid, kThreads, smem, st>>>(p);
  else
    attn_rope_kernel<false><<<(unsigned)grid, kThreads, smem, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // extern "C"
