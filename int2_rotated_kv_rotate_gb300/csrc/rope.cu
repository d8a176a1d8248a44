// Rotary positions on queries and keys.
//
// Pair i of a row at position p turns by the angle 2 pi p t_i, t_i = f_i / (2 pi) turns a
// position: (a, b) -> mag (a cos - b sin, b cos + a sin).  The table holds t_i as a 64-bit
// fixed-point fraction of a turn, so p t_i modulo one turn is one wrapping integer product:
// exact for every position, with no fp64 and no range reduction of a large angle.  The top
// two bits (rounded) are the quadrant, and what is left is at most an eighth of a turn and
// converts to fp32 with a relative error of 2^-24.
//
// Elementwise and HBM-bound: every channel is read once and written once.  A CTA takes the
// rows of `rows_per_cta` positions: it computes their sines and cosines once into shared
// memory (one per row and pair, for all heads), then thread (head, unit) turns one unit of
// its head: 16 bytes of the first half with the 16 bytes that pair with them (half layout)
// or 16 bytes of adjacent pairs (interleaved).  A thread keeps its unit over the row's
// heads, so its sines and cosines stay in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"

namespace oscar {
namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }

template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T v[V];
};

// cos and sin of 2 pi (phase / 2^64).
__device__ __forceinline__ float2 turn(uint64_t phase) {
  const uint64_t q = (phase + (uint64_t(1) << 61)) >> 62;      // nearest quarter turn, mod 4
  const int32_t rest = int32_t(int64_t(phase - (q << 62)) >> 32);  // within an eighth of a turn
  float s, c;
  sincospif(float(rest) * 4.6566128730773926e-10f, &s, &c);  // 2^-31: half turns
  const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -a : a, (q & 2) ? -b : b);
}

// V: channels of a unit (16 bytes, or 1 where the layout or the rotary size does not allow
// vectors).  A unit of the half layout is V channels of the first half and their V
// partners; of the interleaved one, V channels (2 at V = 1).  Channels past rotary_dim are
// copied, VP at a time, unless the call works in place.
template <typename T, int V, int VP, bool INTERLEAVED>
__global__ void __launch_bounds__(512) rope_kernel(RopeParams p) {
  extern __shared__ __align__(16) float2 table[];  // [rows_per_cta][pairs]
  constexpr int kPairs = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;  // pairs of a unit
  const int pairs = p.rotary_dim / 2;
  const long long row0 = (long long)blockIdx.x * p.rows_per_cta;
  const int n_rows = int(min((long long)p.rows_per_cta, p.n_rows - row0));
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < n_rows * pairs; e += blockDim.x) {
    const int r = e / pairs, i = e - r * pairs;
    const long long pos = p.positions64 ? reinterpret_cast<const long long*>(p.positions)[row0 + r]
                                        : (long long)(reinterpret_cast<const int*>(p.positions)[row0 + r]);
    float2 cs = turn(uint64_t(pos) * p.steps[i]);
    table[e] = make_float2(cs.x * p.magnitude, (p.transpose ? -cs.y : cs.y) * p.magnitude);
  }
  __syncthreads();
  const int unit = threadIdx.x % p.units, lane = threadIdx.x / p.units;
  if (lane >= p.head_lanes) return;  // threads past the last whole head
  const int H = p.x[0].n_heads + p.x[1].n_heads;
  for (int r = 0; r < n_rows; ++r) {
    float2 cs[kPairs];
    const bool turns = unit < p.turn_units;
    if (turns) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) cs[j] = table[r * pairs + unit * kPairs + j];
    }
    for (int h = lane; h < H; h += p.head_lanes) {
      const int z = h >= p.x[0].n_heads;
      const RopeTensor& x = p.x[z];
      const int hh = z ? h - p.x[0].n_heads : h;
      const T* in = static_cast<const T*>(x.in) + (row0 + r) * x.in_row + (long long)hh * x.in_head;
      T* out = static_cast<T*>(x.out) + (row0 + r) * x.out_row + (long long)hh * x.out_head;
      if (turns) {
        if constexpr (INTERLEAVED) {
          using W = Vec<T, 2 * kPairs>;
          W w;
          if constexpr (V > 1) w = *reinterpret_cast<const W*>(in + unit * 2 * kPairs);
          else {
            w.v[0] = in[2 * unit];
            w.v[1] = in[2 * unit + 1];
          }
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const float a = to_f32(w.v[2 * j]), b = to_f32(w.v[2 * j + 1]);
            w.v[2 * j] = from_f32<T>(a * cs[j].x - b * cs[j].y);
            w.v[2 * j + 1] = from_f32<T>(b * cs[j].x + a * cs[j].y);
          }
          if constexpr (V > 1) *reinterpret_cast<W*>(out + unit * 2 * kPairs) = w;
          else {
            out[2 * unit] = w.v[0];
            out[2 * unit + 1] = w.v[1];
          }
        } else {
          using W = Vec<T, V>;
          W a = *reinterpret_cast<const W*>(in + unit * V);
          W b = *reinterpret_cast<const W*>(in + pairs + unit * V);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float u = to_f32(a.v[j]), v = to_f32(b.v[j]);
            a.v[j] = from_f32<T>(u * cs[j].x - v * cs[j].y);
            b.v[j] = from_f32<T>(v * cs[j].x + u * cs[j].y);
          }
          *reinterpret_cast<W*>(out + unit * V) = a;
          *reinterpret_cast<W*>(out + pairs + unit * V) = b;
        }
      } else if (in != out) {  // channels past rotary_dim
        const int c = p.rotary_dim + (unit - p.turn_units) * VP;
        *reinterpret_cast<Vec<T, VP>*>(out + c) = *reinterpret_cast<const Vec<T, VP>*>(in + c);
      }
    }
  }
}

template <typename T>
int launch_t(RopeParams p, bool aligned, int n_sm, void* stream, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int pairs = p.rotary_dim / 2, rest = p.head_dim - p.rotary_dim;
  const bool vec = aligned && (p.interleaved ? p.rotary_dim : pairs) % V == 0;
  const bool vec_rest = aligned && p.rotary_dim % V == 0 && rest % V == 0;
  p.turn_units = vec ? (p.interleaved ? p.rotary_dim / V : pairs / V) : pairs;
  p.units = p.turn_units + rest / (vec_rest ? V : 1);
  const int H = p.x[0].n_heads + p.x[1].n_heads;
  // Lanes of heads that fill a CTA of about 320 threads with no ragged last pass.
  const int want = p.units < 320 ? 320 / p.units : 1;
  const int passes = (H + want - 1) / want;
  p.head_lanes = (H + passes - 1) / passes;
  const int threads = (p.units * p.head_lanes + 31) / 32 * 32;
  // Few rows: one a CTA, to spread them.  Many: four share the table's barrier.
  p.rows_per_cta = p.n_rows >= 16LL * n_sm ? 4 : 1;
  const size_t smem = size_t(p.rows_per_cta) * pairs * sizeof(float2);
  const long long grid = (p.n_rows + p.rows_per_cta - 1) / p.rows_per_cta;
  auto go = [&](auto kernel) { return launch_ex(kernel, dim3(unsigned(grid)), dim3(threads), smem, stream, p); };
  int e;
  if (p.interleaved) {
    if (vec) e = vec_rest ? go(rope_kernel<T, V, V, true>) : go(rope_kernel<T, V, 1, true>);
    else e = vec_rest ? go(rope_kernel<T, 1, V, true>) : go(rope_kernel<T, 1, 1, true>);
  } else {
    if (vec) e = vec_rest ? go(rope_kernel<T, V, V, false>) : go(rope_kernel<T, V, 1, false>);
    else e = vec_rest ? go(rope_kernel<T, 1, V, false>) : go(rope_kernel<T, 1, 1, false>);
  }
  if (!e) *launches += 1;
  return e;
}

}  // namespace

int launch_rope(const RopeParams& p, int dtype, bool aligned, int n_sm, void* stream, int* launches) {
  if (dtype == OSCAR_DTYPE_BF16) return launch_t<__nv_bfloat16>(p, aligned, n_sm, stream, launches);
  if (dtype == OSCAR_DTYPE_F16) return launch_t<__half>(p, aligned, n_sm, stream, launches);
  if (dtype == OSCAR_DTYPE_F32) return launch_t<float>(p, aligned, n_sm, stream, launches);
  return int(cudaErrorInvalidValue);
}

}  // namespace oscar
