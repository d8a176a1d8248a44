// Rotary positions on queries and keys.
//
// Pair i of a row at position p turns by the angle 2 pi p t_i, t_i = f_i / (2 pi) turns a
// position: (a, b) -> mag (a cos - b sin, b cos + a sin).  The table holds t_i as a 64-bit
// fixed-point fraction of a turn, so p t_i modulo one turn is one wrapping integer product:
// exact for every position, with no fp64 and no range reduction of a large angle.  The top
// two bits (rounded) are the quadrant, and what is left is at most an eighth of a turn and
// converts to fp32, all of its bits at once, with a relative error of 2^-24.
//
// Elementwise and HBM-bound: every channel is read once and written once.  A CTA takes the
// rows of `rows_per_cta` positions and some 320 threads' worth of heads.  It computes its
// rows' sines and cosines once into shared memory (one per row and pair, for all heads),
// then thread (head, unit) walks down the rows with one unit of its head: 16 bytes of the
// first half with the 16 bytes that pair with them (half layout), or 16 bytes of adjacent
// pairs (interleaved).  Two rows are loaded before the first is stored.  Walking the rows
// with a fixed head costs one pointer step a row; walking the heads of a row, and holding
// the sines in registers, spent more on addresses than it saved (8192 rows of 40 heads with
// 96 turning channels: 54 against 41 us).  Measured: 5.8 TB/s on 16384 rows of 72 bf16
// heads (104 us), 6.0 TB/s on 4099 rows of 40 fp32 heads (28.1 us); one row 1.6 us in a graph;
// without vectors, 8192 rows of 40 bf16 heads with 18 turning channels 50 us (31 with 128).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
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

// V channels at p: one access where VEC (aligned to it), else one by one.
template <typename T, int V, bool VEC>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  Vec<T, V> w;
  if constexpr (VEC) w = *reinterpret_cast<const Vec<T, V>*>(p);
  else {
#pragma unroll
    for (int i = 0; i < V; ++i) w.v[i] = p[i];
  }
  return w;
}
template <typename T, int V, bool VEC>
__device__ __forceinline__ void store(T* p, const Vec<T, V>& w) {
  if constexpr (VEC) *reinterpret_cast<Vec<T, V>*>(p) = w;
  else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = w.v[i];
  }
}

// cos and sin of 2 pi (phase / 2^64).
__device__ __forceinline__ float2 turn(uint64_t phase) {
  const uint64_t q = (phase + (uint64_t(1) << 61)) >> 62;  // nearest quarter turn, mod 4
  const int64_t rest = int64_t(phase - (q << 62));         // within an eighth of a turn
  float s, c;
  sincospif(float(rest) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
  const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -a : a, (q & 2) ? -b : b);
}

constexpr int kBatch = 2;  // rows that a thread loads before it stores the first
// CTAs of 512 threads whose registers an SM has to hold.  The half layout keeps two vectors
// a row, for which 40 registers spill (138 against 107 us on 16384 rows of 72 bf16 heads);
// the interleaved one needs no more (98 against 104 us).
constexpr int kPerSMHalf = 2, kPerSMInterleaved = 3;

// V: channels of a vector, 16 bytes of them, or 1 where strides or sizes do not allow
// vectors.  A unit that turns is V channels of the first half and their V partners (half
// layout) or V channels (interleaved; 2 at V = 1).  Channels past rotary_dim are copied by
// units of their own, unless the call works in place: 16 bytes each; at V = 1 first single
// channels up to pass_from, then 16 bytes each if pass_from < head_dim.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(512, INTERLEAVED ? kPerSMInterleaved : kPerSMHalf)
    rope_kernel(RopeParams p) {
  extern __shared__ __align__(16) float2 table[];  // [rows_per_cta][pairs], see slot()
  constexpr int kPairs = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;  // pairs of a unit
  constexpr int kChannels = INTERLEAVED ? 2 * kPairs : V;        // channels of one of its vectors
  constexpr bool kVec = V > 1;
  constexpr int kWide = 16 / sizeof(T);
  const int pairs = p.rotary_dim / 2;
  const unsigned block = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;  // a row block's chunks run together
  const long long row0 = (long long)block * p.rows_per_cta;
  const int n_rows = int(min((long long)p.rows_per_cta, p.n_rows - row0));
  const int unit = threadIdx.x % p.units, head = chunk * p.head_lanes + threadIdx.x / p.units;
  const int z = head >= p.x[0].n_heads;
  const RopeTensor& x = p.x[z];
  const int h = z ? head - p.x[0].n_heads : head;
  bool mine = threadIdx.x / p.units < p.head_lanes && h < x.n_heads;
  const bool turns = unit < p.turn_units;
  const bool single = !turns && unit - p.turn_units < p.pass_from - p.rotary_dim;
  const int c0 = turns    ? unit * kChannels
                 : single ? p.rotary_dim + unit - p.turn_units
                          : p.pass_from + (unit - p.turn_units - (p.pass_from - p.rotary_dim)) * kWide;
  const T* in = static_cast<const T*>(x.in) + row0 * x.in_row + h * x.in_head + c0;
  T* out = static_cast<T*>(x.out) + row0 * x.out_row + h * x.out_head + c0;
  // The pairs of a unit in twos of 16 bytes, the twos of all units side by side: a warp's
  // 16-byte reads fall in different banks.
  auto slot = [&](int r, int u, int j) {
    if constexpr (kPairs == 1) return r * pairs + u;
    return r * pairs + ((j >> 1) * p.turn_units + u) * 2 + (j & 1);
  };
  Vec<T, kChannels> a[kBatch], b[kBatch];
  auto fetch = [&](int r) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (r + k < n_rows) {
        a[k] = load<T, kChannels, kVec>(in + k * x.in_row);
        if constexpr (!INTERLEAVED)
          if (turns) b[k] = load<T, kChannels, kVec>(in + k * x.in_row + pairs);
      }
  };
  if (!turns && static_cast<const void*>(in) == static_cast<const void*>(out)) mine = false;  // in place: nothing to copy
  pdl_wait();
  pdl_trigger();
  if (mine && (kVec || turns)) fetch(0);  // in flight while the table is made
  for (int e = threadIdx.x; e < n_rows * pairs; e += blockDim.x) {
    const int r = e / pairs, i = e - r * pairs;
    const long long pos = p.positions64 ? reinterpret_cast<const long long*>(p.positions)[row0 + r]
                                        : (long long)(reinterpret_cast<const int*>(p.positions)[row0 + r]);
    const float2 cs = turn(uint64_t(pos) * p.steps[i]);
    table[slot(r, i / kPairs, i % kPairs)] =
        make_float2(cs.x * p.magnitude, (p.transpose ? -cs.y : cs.y) * p.magnitude);
  }
  __syncthreads();
  if (!mine) return;
  if constexpr (!kVec) {
    if (!turns) {  // single channels and 16-byte vectors past rotary_dim
      for (int r = 0; r < n_rows; ++r, in += x.in_row, out += x.out_row) {
        if (single) *out = *in;
        else store<T, kWide, true>(out, load<T, kWide, true>(in));
      }
      return;
    }
  }
  for (int r = 0; r < n_rows; r += kBatch) {
    if (r) fetch(r);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r + k >= n_rows) break;
      T* o = out + k * x.out_row;
      if (turns) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 cs = table[slot(r + k, unit, j)];
          T& tu = INTERLEAVED ? a[k].v[2 * j] : a[k].v[j];
          T& tv = INTERLEAVED ? a[k].v[2 * j + 1] : b[k].v[j];
          const float u = to_f32(tu), v = to_f32(tv);
          tu = from_f32<T>(u * cs.x - v * cs.y);
          tv = from_f32<T>(v * cs.x + u * cs.y);
        }
      }
      store<T, kChannels, kVec>(o, a[k]);
      if constexpr (!INTERLEAVED)
        if (turns) store<T, kChannels, kVec>(o + pairs, b[k]);
    }
    in += kBatch * x.in_row;
    out += kBatch * x.out_row;
  }
}

template <typename T>
int launch_t(RopeParams p, bool aligned, int n_sm, void* stream, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int pairs = p.rotary_dim / 2, rest = p.head_dim - p.rotary_dim;
  const bool vec = aligned && (p.interleaved ? p.rotary_dim : pairs) % V == 0 && rest % V == 0;
  p.turn_units = vec ? (p.interleaved ? p.rotary_dim / V : pairs / V) : pairs;
  const int up = (p.rotary_dim + V - 1) / V * V;  // the first channel past the turning ones on 16 bytes
  p.pass_from = vec ? p.rotary_dim : aligned && up < p.head_dim && p.head_dim % V == 0 ? up : p.head_dim;
  p.units = p.turn_units + (p.pass_from - p.rotary_dim) + (p.head_dim - p.pass_from) / V;
  // CTAs of about 320 threads: whole heads, evenly over the CTAs of a row block
  const int H = p.x[0].n_heads + p.x[1].n_heads;
  const int most = p.units < 320 ? 320 / p.units : 1;
  p.chunks = (H + most - 1) / most;
  p.head_lanes = (H + p.chunks - 1) / p.chunks;
  const int threads = (p.units * p.head_lanes + 31) / 32 * 32;
  // Rows of a CTA: full waves of CTAs of at most 16 rows.  4099 rows of 40 bf16 heads: 16.9 us
  // in one wave of 9 rows a CTA, 18.9 and 21.5 us with 4 and 8 (a ragged second wave); 16384
  // rows of 72 heads: 112, 107 and 109 us with 4, 8 and 16.
  const int per_sm = p.interleaved ? kPerSMInterleaved : kPerSMHalf;
  const long long wave = std::max<long long>(1, (long long)n_sm * (512 * per_sm / threads) / p.chunks);
  const long long waves = (p.n_rows + 16 * wave - 1) / (16 * wave);
  p.rows_per_cta = int((p.n_rows + waves * wave - 1) / (waves * wave));
  const size_t smem = size_t(p.rows_per_cta) * pairs * sizeof(float2);
  const long long grid = (p.n_rows + p.rows_per_cta - 1) / p.rows_per_cta * p.chunks;
  if (grid > 0x7fffffffLL) return int(cudaErrorInvalidConfiguration);
  auto go = [&](auto kernel) { return launch_ex(kernel, dim3(unsigned(grid)), dim3(threads), smem, stream, p); };
  int e;
  if (p.interleaved) e = vec ? go(rope_kernel<T, V, true>) : go(rope_kernel<T, 1, true>);
  else e = vec ? go(rope_kernel<T, V, false>) : go(rope_kernel<T, 1, false>);
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
