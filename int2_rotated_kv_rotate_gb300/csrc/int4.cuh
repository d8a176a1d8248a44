// The 4-bit pages.
#pragma once

#include <cstdint>

#include "oscar_internal.h"

namespace oscar {

constexpr int kInt4Row = kHeadDim / 2;  // 64 B of 4-bit codes per token
constexpr int kInt4Half = kPage / 2;    // tokens of a half page, the unit in which the decode copies

// A (page, kv-head) is two blocks of 32 tokens, each K codes, V codes, then K and V scale and zero
// words (ng a token), so that a warp's copy of a half page is one piece: 4352 or 5120 bytes.
__host__ __device__ constexpr int int4_half_bytes(int ng) { return 2 * kInt4Half * (kInt4Row + 4 * ng); }

// Byte in its (page, kv-head) of the word that holds channels 8 l .. 8 l + 7 (channel 8 l + i in bits
// 4 i .. 4 i + 3) of token t, K (kv 0) or V: word l / 4 of 16-byte chunk (l % 4) ^ (t / 2 % 4) of the
// token's row.  A lane of a score MMA reads a chunk, 8 channels of each group of 32; the exclusive or
// spreads the chunk that a value MMA reads of even tokens over the banks.
__host__ __device__ constexpr int int4_word(int t, int l, int kv, int ng) {
  return (t / kInt4Half) * int4_half_bytes(ng) + kv * (kInt4Half * kInt4Row) + (t % kInt4Half) * kInt4Row +
         16 * ((l & 3) ^ ((t >> 1) & 3)) + 4 * (l >> 2);
}
// And of the scale (low half) and zero word of its group g.
__host__ __device__ constexpr int int4_scale(int t, int g, int kv, int ng) {
  return (t / kInt4Half) * int4_half_bytes(ng) + 2 * kInt4Half * kInt4Row + 4 * ((kv * kInt4Half + t % kInt4Half) * ng + g);
}

}  // namespace oscar
