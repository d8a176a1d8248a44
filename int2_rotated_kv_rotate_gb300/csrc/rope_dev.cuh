// The rotary phase, shared by the kernels that turn rows (rope.cu, append_rows.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace oscar {

// cos and sin of 2 pi (phase / 2^64).
__device__ __forceinline__ float2 turn(uint64_t phase) {
  const uint64_t q = (phase + (uint64_t(1) << 61)) >> 62;  // nearest quarter turn, mod 4
  const int64_t rest = int64_t(phase - (q << 62));         // within an eighth of a turn
  float s, c;
  sincospif(float(rest) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
  const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -a : a, (q & 2) ? -b : b);
}

}  // namespace oscar
