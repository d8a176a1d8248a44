// The 4-bit pages' rows.
#pragma once

#include <cstdint>

#include "oscar_internal.h"

namespace oscar {

constexpr int kInt4Row = kHeadDim / 2;  // 64 B of 4-bit codes per token

// Byte of the word that holds channels 8 l .. 8 l + 7 (channel 8 l + i in bits 4 i .. 4 i + 3) of
// token t in a page's block of rows: word l / 4 of 16-byte chunk (l % 4) ^ (t / 2 % 4).  A lane of
// a score MMA reads a chunk, 8 channels of each group of 32; the exclusive or spreads the chunk
// that a value MMA reads of even tokens over the banks.
__host__ __device__ constexpr int int4_word(int t, int l) {
  return t * kInt4Row + 16 * ((l & 3) ^ ((t >> 1) & 3)) + 4 * (l >> 2);
}

}  // namespace oscar
