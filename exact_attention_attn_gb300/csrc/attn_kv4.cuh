// Layout of the 4-bit KV cache and the pieces its kernels share.
//
// The cache is [num_pages, Hkv, page_bytes].  A page of one kv head holds P
// tokens: K's codes [D/64][P][32 bytes], K's pairs [D/64][P][scale, minimum]
// (bfloat16), then V's codes and pairs.  Byte b of a 32-byte row holds dims 2b
// (low nibble) and 2b + 1 of the group of 64; the value of code c is
// scale * c + minimum.  Rows are grouped by 64 dims, not by token, so that the
// rows a warp reads together lie next to each other in shared memory (eight
// 32-byte rows: two 128-byte lines, no bank conflict), and a page of a head is
// one contiguous block, so that one bulk copy moves it.
#pragma once

#include <stdint.h>

namespace attn {

constexpr int kKv4Group = 64;
constexpr int kKv4RowBytes = 32;
constexpr int kKv4PairBytes = 4;

__host__ __device__ constexpr int kv4_codes_bytes(int G, int P) { return G * P * kKv4RowBytes; }
__host__ __device__ constexpr int kv4_side_bytes(int G, int P) { return G * P * (kKv4RowBytes + kKv4PairBytes); }
__host__ __device__ constexpr int kv4_page_bytes(int G, int P) { return 2 * kv4_side_bytes(G, P); }

// log2 of a page size the cache takes (16, 32 or 64 tokens), else -1.
inline int kv4_page_shift(int P) { return P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : -1; }

}  // namespace attn
