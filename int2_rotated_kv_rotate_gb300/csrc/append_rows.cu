// Appending rows to the paged caches of one launch's own: keys turned by their rotary positions
// on the way (and the queries of the same tokens), into BF16 pages or, quantised, into 4-bit
// pages; the 4-bit pages' plain append and their rows read back.
//
// Sixteen lanes take a row of a head, 8 channels (16 bytes) each.  A channel's rotary partner is
// in the same lane (interleaved pairs) or, in the half layout, in the lane rotary_dim / 16 away,
// from which it comes by shuffles; the minimum and maximum of a quantisation group are over 4 or
// 16 lanes.  So a row is read once, whatever is done to it.  A CTA takes the append plan's items
// (up to 16 tokens of a request), makes its rows' sines and cosines once for all heads, and each
// half-warp walks down the rows of its head, kBatch rows in flight.
//
// Rotary: the row that is stored is the turned one rounded to bf16, as by RotaryEmbedding and an
// append after it, bit for bit.
// HBM-bound when there are many rows, 61 us (5.5 TB/s) for 13635 rows of 32 + 8 + 8 heads; 64 registers a thread,
// four CTAs an SM (384 threads at 56 registers spill: 93 us).
//
// 4 bits, per token and group of 32 or 128 channels: s = bf16((max - min) / 15), z = bf16(min)
// (exact), code = clamp(rint((x - z) / s), 0, 15), every operation in fp32, 0 where s = 0.  The
// extremes are found on packed bf16, the rest in pairs of fp32 by products with approximate
// reciprocals; the few rows for which that is not known to give the definition's bits are taken
// again, as it stands, after the item's others.  (With divisions and single operations 8192 tokens of 8
// kv-heads took 42 us; 20 now, 2.3 TB/s.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "int4.cuh"
#include "oscar_internal.h"
#include "packed.cuh"
#include "rope_dev.cuh"

namespace oscar {
namespace {

constexpr int kBatch = 4;       // rows that a half-warp loads before it stores the first
constexpr int kItemRows = 16;   // of an append item at most
constexpr int kMaxThreads = 256;
constexpr int kPerSM = 4;

// Values past this count as it (and NaN as it): differences and their fifteenths stay finite.
constexpr float kInt4Limit = 8.507059173023462e37f;  // 2^126

__device__ __forceinline__ uint4 load8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = uint32_t(p[2 * i]) | (uint32_t(p[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(uint16_t* p, uint4 v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[2 * i] = uint16_t(w[i]);
    p[2 * i + 1] = uint16_t(w[i] >> 16);
  }
}

// Larger of each half, NaN where either is.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The definition as it stands, of the 8 channels of each of a half-warp's 16 lanes: codes (one word
// a lane) and the scale and zero point of the lane's group.  lanes: 4 or 16, those of a group.
__device__ __forceinline__ uint2 quantize8_plain(uint4 v, int lanes, unsigned mask) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
  float lo = kInt4Limit, hi = -kInt4Limit;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fmaxf(fminf(i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]), kInt4Limit), -kInt4Limit);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
  }
  const uint16_t s16 = bf16_rne(__fdiv_rn(hi - lo, 15.f));
  const float s = bf16_f32(s16);
  uint32_t codes = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= uint32_t(fminf(fmaxf(rintf(__fdiv_rn(x[i] - lo, s)), 0.f), 15.f)) << (4 * i);
  }
  return make_uint2(codes, uint32_t(s16) | (__float_as_uint(lo) & 0xffff0000u));  // (lo is one of the values, or 2^126)
}

// The same for most groups; `plain` says that this lane's is not known to be one of them: NaN or
// values past the limit, a scale below the normal numbers, or near a midpoint of bf16.
//
// The codes' quotients: t = d inv, d = fl(x - z), is off by 2^-22 of it at most (inv, which is within a unit in
// the last place, and the product); a step of residual correction, t + (d - t s) inv, leaves 2^-44 of
// error before its one rounding.  Only a quotient at or next to a half matters for rint.  Halves (up
// to 14.5) times s (8 bits) are exact, so d is one, and the step exact; or d differs from it by a unit in its
// last place or more, and then d / s is at least 2^-8 of a unit away from where its rounding would
// turn to or from the half (s / 2 times 2^k has 8 bits, so its units are over 2^-24 (1 + 2^-8) of it):
// the rounded sum falls on the side that the rounded quotient does.
__device__ __forceinline__ uint2 quantize8(uint4 v, int lanes, unsigned mask, bool& plain) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t up = w[0], down = w[0] ^ 0x80008000u;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    up = max_bf16x2(up, w[i]);
    down = max_bf16x2(down, w[i] ^ 0x80008000u);
  }
  uint32_t ends = max_bf16x2(permute(up, down, 0x5410), permute(up, down, 0x7632));  // (maximum, -minimum)
  ends = max_bf16x2(ends, __shfl_xor_sync(mask, ends, 1));
  ends = max_bf16x2(ends, __shfl_xor_sync(mask, ends, 2));
  if (lanes == 16) {
    ends = max_bf16x2(ends, __shfl_xor_sync(mask, ends, 4));
    ends = max_bf16x2(ends, __shfl_xor_sync(mask, ends, 8));
  }
  const float hi = bf16_lo(ends), neg_lo = bf16_hi(ends);
  const float fifteenth = (hi + neg_lo) * (1.f / 15.f);  // within 2 units in the last place
  const uint32_t s16 = pack_bf16(fifteenth, 0.f);
  const float s = bf16_lo(s16);
  // (4: units of the fp32 number around a midpoint; ends: 2^126 is 0x7e80; a scale of 0 by a span of 0 is none of them)
  plain = ((__float_as_uint(fifteenth) + 4u) & 0xffffu) - 0x8000u <= 8u || (ends & 0x7fffu) > 0x7e80u ||
          (ends & 0x7fff0000u) > 0x7e800000u || (s16 < 0x0080u && fifteenth != 0.f);
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));  // at most 1 unit in the last place off
  inv = s16 == 0u ? 0.f : inv;                           // the codes of a scale of 0
  // quotients in [0, 15 (1 + 2^-8)]: the nearest whole number is in the low bits of t + 1.5 * 2^23
  const uint64_t neg_lo2 = pack2(neg_lo, neg_lo), inv2 = pack2(inv, inv), neg_s2 = pack2(-s, -s), magic = pack2(12582912.f, 12582912.f);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t d = add2(pack2(bf16_lo(w[i]), bf16_hi(w[i])), neg_lo2);
    uint64_t t = mul2(d, inv2);
    t = fma2(fma2(t, neg_s2, d), inv2, t);
    const float2 bits = unpack2(add2(t, magic));
    c[2 * i] = __float_as_uint(bits.x);
    c[2 * i + 1] = __float_as_uint(bits.y);
  }
  // the low bytes of the even and of the odd channels
  const uint32_t even = permute(permute(c[0], c[2], 0x0040), permute(c[4], c[6], 0x0040), 0x5410);
  const uint32_t odds = permute(permute(c[1], c[3], 0x0040), permute(c[5], c[7], 0x0040), 0x5410);
  return make_uint2(even + 16u * odds, s16 | ((ends & 0xffff0000u) ^ 0x80000000u));
}

// How a lane finds the partners of its 8 channels: no turning; another lane's 8 (half layout,
// rotary_dim a multiple of 16); its own (interleaved); anywhere in the row.
enum Turn { kNoTurn, kLanes, kAdjacent, kAnywhere };

template <bool INT4, Turn TURN>
__global__ void __launch_bounds__(kMaxThreads, kPerSM) append_rows_kernel(KernelParams kp, int layer, AppendRowsParams p) {
  // The table, as the lanes multiply: a row's turned channels are X cx + (Y cy), the product in
  // brackets rounded first.  kLanes: X, Y are a channel of the first half and its partner of the
  // second, or the other way round, and two channels' factors (cx, cx, cy, cy) are 16 bytes, (cos,
  // cos, -sin, -sin) for the first half and (sin, sin, cos, cos) for the second, those of the lanes side
  // by side.  kAdjacent: X, Y are the two channels of a pair, and (cos, sin, -sin, cos) gives both.
  // kAnywhere: (cos, sin) of each pair.
  extern __shared__ __align__(16) float table[];  // [kItemRows][row_words]
  const int n_items = reinterpret_cast<const int*>(kp.base + kp.lay.append_counts)[0];
  const int l16 = threadIdx.x & 15, c0 = 8 * l16;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  const int head = int(blockIdx.y) * p.chunk_heads + int(threadIdx.x >> 4);
  const int Hq = p.q.n_heads, Hkv = kp.n_kv_heads;
  const bool mine = int(threadIdx.x >> 4) < p.chunk_heads && head < Hq + 2 * Hkv;
  const int kind = head < Hq ? 0 : head < Hq + Hkv ? 1 : 2;  // q, k, v
  const int h = kind == 0 ? head : kind == 1 ? head - Hq : head - Hq - Hkv;
  const uint16_t* in = static_cast<const uint16_t*>(kind == 0 ? p.q.in : kind == 1 ? p.k : p.v) +
                       (kind == 0 ? h * p.q.in_head : kind == 1 ? h * p.k_head : h * p.v_head) + c0;
  const long long in_row = kind == 0 ? p.q.in_row : kind == 1 ? p.k_row : p.v_row;
  const bool in_vec = kind == 0 ? p.q_in_vec : kind == 1 ? p.k_vec : p.v_vec;
  const int R = p.rotary_dim, pairs = R / 2, eighth = pairs >> 3;
  const int row_words = TURN == kAnywhere ? 2 * pairs : 4 * pairs;  // floats a row
  const bool turns = TURN != kNoTurn && kind != 2 && (TURN == kAnywhere || c0 < R);
  const bool first = c0 < pairs;
  const int other = TURN != kLanes || c0 >= R ? l16 : first ? l16 + eighth : l16 - eighth;
  const float* factors = table + (TURN == kLanes ? 4 * (first ? l16 : l16 - eighth + pairs / 2) : TURN == kAdjacent ? 2 * c0 : 0);
  // the head's keys or values in page 0 of the layer
  uint8_t* pool = kp.base;
  const int kv = kind == 2, ng = kHeadDim / (INT4 ? kp.group : kHeadDim);
  if (kind != 0) {
    if constexpr (!INT4) {
      pool += kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride + size_t(h) * kp.lay.bf16_head_stride +
              size_t(kv) * (kPage * kHeadDim * 2) + 16 * l16;
    } else {
      pool += kp.lay.codes + size_t(layer) * kp.lay.codes_layer_stride + size_t(h) * kp.lay.codes_head_stride;
    }
  }
  const unsigned page_stride = unsigned(INT4 ? kp.lay.codes_page_stride : kp.lay.bf16_page_stride);
  bool waited = false;
  for (int ix = blockIdx.x; ix < n_items * p.item_parts; ix += gridDim.x) {
    AppendItem it = reinterpret_cast<const AppendItem*>(kp.base + kp.lay.append_items)[ix / p.item_parts];
    if (p.item_parts > 1) {  // a part of the item's rows
      const int rows = kItemRows / p.item_parts, at = ix % p.item_parts * rows;
      it.begin += at;
      it.count = min(rows, it.count - at);
      if (it.count <= 0) continue;
    }
    const AppendReq a = reinterpret_cast<const AppendReq*>(kp.base + kp.lay.append_reqs)[it.req];
    const bool slot_ok = a.slot >= 0 && a.slot < kp.max_requests;
    if (!slot_ok && threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
    const long long row0 = (long long)a.x_offset + it.begin - a.L0;
    if (waited) __syncthreads();  // the table of the item before is read
    if (!waited && (TURN == kNoTurn || p.positions)) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    if constexpr (TURN != kNoTurn) {  // (the plan is older than the preceding kernel: places may be turned before the wait)
      for (int e = threadIdx.x; e < it.count * pairs; e += blockDim.x) {
        const int r = e / pairs, i = e - r * pairs;
        const long long pos = !p.positions ? (long long)(it.begin + r)
                              : p.positions64 ? reinterpret_cast<const long long*>(p.positions)[row0 + r]
                                              : (long long)(reinterpret_cast<const int*>(p.positions)[row0 + r]);
        const float2 cs = turn(uint64_t(pos) * p.steps[i]);
        const float c = cs.x * p.magnitude, si = cs.y * p.magnitude;
        float* row = table + r * row_words;
        if (TURN == kAdjacent) {
          reinterpret_cast<float4*>(row)[i] = make_float4(c, si, -si, c);
        } else if (TURN == kLanes) {  // channels 8 u + 2 j, + 1 of a half: twos (half, j, u)
          float* a0 = row + 4 * (((i >> 1) & 3) * eighth + (i >> 3)) + (i & 1);
          float* b0 = a0 + 2 * pairs;
          a0[0] = c, a0[2] = -si;
          b0[0] = si, b0[2] = c;
        } else {
          reinterpret_cast<float2*>(row)[i] = make_float2(c, si);
        }
      }
      if (!waited) {
        pdl_wait();
        pdl_trigger();
        waited = true;
      }
      __syncthreads();
    }
    if (!mine || !slot_ok) continue;
    // Where the rows go: the item's lie in one page or two.
    const int t0 = it.begin % kPage, crossing = kPage - t0;
    uint8_t *to = pool, *to_next = pool;
    long long to_row = kHeadDim * 2;  // bytes from row to row (4-bit rows are found by their token)
    bool ok = true, ok_next = true;
    if (kind == 0) {
      to = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.q.out) + row0 * p.q.out_row + h * p.q.out_head + c0);
      to_row = 2 * p.q.out_row;
    } else {
      const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(a.slot) * kp.max_pages_per_request;
      const int lp = it.begin / kPage;
      const int page = lp < kp.max_pages_per_request ? ptab[lp] : -1;
      const int next = it.count <= crossing ? page : lp + 1 < kp.max_pages_per_request ? ptab[lp + 1] : -1;
      ok = page >= 0 && page < kp.max_pages;
      ok_next = next >= 0 && next < kp.max_pages;
      if (l16 == 0 && !(ok && ok_next)) flag(kp, OSCAR_FLAG_BAD_PAGE);
      to += size_t(unsigned(ok ? page : 0)) * page_stride;
      to_next += size_t(unsigned(ok_next ? next : 0)) * page_stride;
      if constexpr (!INT4) {
        to += t0 * (kHeadDim * 2);
        to_next -= crossing * (kHeadDim * 2);
      }
    }
    uint32_t again = 0;  // bit r: this lane's group of row r is to be quantised as the definition stands
    auto put = [&](int r, uint4 v, auto plain) {
      if (TURN != kNoTurn && kind != 2) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (TURN == kAdjacent) {
          if (turns) {
            const float4* at = reinterpret_cast<const float4*>(factors + r * row_words);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 2 * i < R) {
                const float4 f = at[i];
                const float u = bf16_lo(w[i]), t = bf16_hi(w[i]);
                const float2 o = unpack2(fma2(pack2(u, u), pack2(f.x, f.y), mul2(pack2(t, t), pack2(f.z, f.w))));
                w[i] = pack_bf16(o.x, o.y);
              }
          }
        } else if constexpr (TURN == kLanes) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(mask, w[i], other, 16);
          if (turns) {
            const float4* at = reinterpret_cast<const float4*>(factors + r * row_words);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = at[i * eighth];
              const uint32_t X = first ? w[i] : y[i], Y = first ? y[i] : w[i];
              const float2 o = unpack2(fma2(pack2(bf16_lo(X), bf16_hi(X)), pack2(f.x, f.y),
                                           mul2(pack2(bf16_lo(Y), bf16_hi(Y)), pack2(f.z, f.w))));
              w[i] = pack_bf16(o.x, o.y);
            }
          }
        } else if constexpr (TURN == kAnywhere) {
          // read one by one, before any lane stores (q may be turned in place)
          const uint16_t* from = in + (row0 + r) * in_row - c0;
          const float2* row = reinterpret_cast<const float2*>(table + r * row_words);
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + i;
            o[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
            if (c < R) {
              const bool low = c < pairs;
              const float2 cs = row[low ? c : c - pairs];
              const float t = bf16_f32(from[low ? c + pairs : c - pairs]);
              o[i] = low ? fmaf(o[i], cs.x, -(t * cs.y)) : fmaf(t, cs.y, o[i] * cs.x);
            }
          }
          __syncwarp(mask);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = c0 + 2 * i < R ? pack_bf16(o[2 * i], o[2 * i + 1]) : w[i];
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      const bool behind = r >= crossing && kind != 0;
      if (!(behind ? ok_next : ok)) return;  // (flagged above)
      uint8_t* row = behind ? to_next : to;
      if (INT4 && kind != 0) {
        const int t = (t0 + r) % kPage, lanes = kp.group / 8;
        uint2 c;
        if constexpr (decltype(plain)::value) {
          c = quantize8_plain(v, lanes, mask);
        } else {
          bool leave;
          c = quantize8(v, lanes, mask, leave);
          again |= leave ? 1u << r : 0u;
        }
        *reinterpret_cast<uint32_t*>(row + int4_word(t, l16, kv, ng)) = c.x;
        if (l16 % lanes == 0) *reinterpret_cast<uint32_t*>(row + int4_scale(t, l16 / lanes, kv, ng)) = c.y;
      } else {
        store8(reinterpret_cast<uint16_t*>(row + r * to_row), v, kind != 0 || p.q_out_vec);
      }
    };
    const uint16_t* src = in + row0 * in_row;
    int r0 = 0;
    for (; r0 + kBatch <= it.count; r0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b, src += in_row) x[b] = load8(src, in_vec);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) put(r0 + b, x[b], std::false_type());
    }
    for (; r0 < it.count; ++r0, src += in_row) put(r0, load8(src, in_vec), std::false_type());
    if constexpr (INT4) {
      again = __reduce_or_sync(mask, again);
#pragma unroll 1
      for (; again; again &= again - 1) {
        const int r = __ffs(again) - 1;
        put(r, load8(in + (row0 + r) * in_row, in_vec), std::true_type());
      }
    }
  }
  if (!waited) {
    pdl_wait();
    pdl_trigger();
  }
}

// Tokens [begin, end) of a request's 4-bit rows as values: fmaf(code, s, z) in fp32, rounded to bf16
// where T is 16 bits.  Sixteen lanes a row, a head (K heads, then V heads) a half-warp, which walks
// down kItemRows tokens, eight of them in flight.  HBM-bound.
constexpr int kReadThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kReadThreads) int4_read_kernel(KernelParams kp, int layer, int slot, int begin, int end,
                                                                T* __restrict__ k_out, T* __restrict__ v_out) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15, ng = kHeadDim / kp.group, Hkv = kp.n_kv_heads;
  const int head = int(blockIdx.y) * (kReadThreads / 16) + int(threadIdx.x >> 4);
  if (head >= 2 * Hkv) return;
  const int kv = head >= Hkv, h = kv ? head - Hkv : head;
  const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(slot) * kp.max_pages_per_request;
  const uint8_t* pool = kp.base + kp.lay.codes + size_t(layer) * kp.lay.codes_layer_stride + size_t(h) * kp.lay.codes_head_stride;
  const int group = l16 / (kp.group / 8);
  T* out = (kv ? v_out : k_out) + size_t(h) * kHeadDim + 8 * l16;
  const long long row = (long long)Hkv * kHeadDim;
  const int shift = 4 * (l16 >> 2) + kv * (kInt4Half * kInt4Row), chunk = l16 & 3;
  // The tokens by sixteens of their places, each of which lies in one half page.
  for (int p0 = (begin / kItemRows + int(blockIdx.x)) * kItemRows; p0 < end; p0 += int(gridDim.x) * kItemRows) {
    const int lp = p0 / kPage, t0 = p0 % kPage;
    const int page = lp < kp.max_pages_per_request ? ptab[lp] : -1;
    const bool ok = page >= 0 && page < kp.max_pages;  // (else zeros, and the flag)
    if (!ok && l16 == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
    const uint8_t* at = pool + size_t(unsigned(ok ? page : 0)) * unsigned(kp.lay.codes_page_stride);
    const uint8_t* rows = at + int4_word(t0, 0, 0, ng) + shift;
    const uint32_t* szs = reinterpret_cast<const uint32_t*>(at + int4_scale(t0, group, kv, ng));
    T* to = out + (long long)(p0 - begin) * row;  // (rows before begin are not touched)
    auto word = [&](int r) { return ok ? *reinterpret_cast<const uint32_t*>(rows + r * kInt4Row + 16 * (chunk ^ ((r >> 1) & 3))) : 0u; };
    auto scale = [&](int r) { return ok ? szs[r * ng] : 0u; };
    auto put = [&](int r, uint32_t w, uint32_t sz) {
      const float s = bf16_lo(sz), z = bf16_hi(sz);
      // a code as the low byte of 2^23: its value by a subtraction
      const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
      const uint64_t ss = pack2(s, s), zz = pack2(z, z), base = pack2(-8388608.f, -8388608.f);
      float2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = unpack2(fma2(add2(pack2(__uint_as_float(permute(even, 0x4b000000u, 0x7650 + i)),
                                     __uint_as_float(permute(odd, 0x4b000000u, 0x7650 + i))),
                                base),
                           ss, zz));
      T* p = to + r * row;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y),
                                                  pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
      } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
      }
    };
    if (begin <= p0 && p0 + kItemRows <= end) {
#pragma unroll
      for (int r = 0; r < kItemRows; r += 2 * kBatch) {
        uint32_t w[2 * kBatch], sz[2 * kBatch];
#pragma unroll
        for (int b = 0; b < 2 * kBatch; ++b) {
          w[b] = word(r + b);
          sz[b] = scale(r + b);
        }
#pragma unroll
        for (int b = 0; b < 2 * kBatch; ++b) put(r + b, w[b], sz[b]);
      }
    } else {
#pragma unroll 1
      for (int r = max(0, begin - p0); r < min(kItemRows, end - p0); ++r) put(r, word(r), scale(r));
    }
  }
}

}  // namespace

int launch_append_rows(const KernelParams& kp, int layer, AppendRowsParams p, bool int4, bool rope, int n_items, long long n_rows,
                       int n_sm, void* stream, int* launches) {
  // whole heads, evenly over the CTAs of an item, an even number of them in each (full warps)
  const int H = p.q.n_heads + 2 * kp.n_kv_heads, most = kMaxThreads / 16;
  const int chunks = (H + most - 1) / most;
  p.chunk_heads = ((H + chunks - 1) / chunks + 1) / 2 * 2;
  // Where whole items would leave every SM less than four CTAs, halves of them, if most have so many
  // rows (8192 rows of 16 heads into 4-bit pages: 21.3 against 19.7 us).
  p.item_parts = !rope && (long long)n_items * chunks < 4LL * n_sm && n_rows > 8LL * n_items ? 2 : 1;
  const dim3 grid(n_items * p.item_parts, chunks), block(16 * p.chunk_heads);
  const size_t smem = rope ? size_t(kItemRows) * (p.rotary_dim / 2) * sizeof(float4) : 0;
  auto go = [&](auto kernel) { return launch_ex(kernel, grid, block, smem, stream, kp, layer, p); };
  int e;
  if (!rope) e = go(append_rows_kernel<true, kNoTurn>);
  else if (p.interleaved) e = int4 ? go(append_rows_kernel<true, kAdjacent>) : go(append_rows_kernel<false, kAdjacent>);
  else if (p.rotary_dim % 16 == 0) e = int4 ? go(append_rows_kernel<true, kLanes>) : go(append_rows_kernel<false, kLanes>);
  else e = int4 ? go(append_rows_kernel<true, kAnywhere>) : go(append_rows_kernel<false, kAnywhere>);
  if (!e) *launches += 1;
  return e;
}

int launch_int4_read(const KernelParams& kp, int layer, int slot, int begin, int end, void* k_out, void* v_out, bool f32,
                     int n_sm, void* stream, int* launches) {
  const dim3 grid(std::min((end + kItemRows - 1) / kItemRows - begin / kItemRows, 16 * n_sm),
                  (2 * kp.n_kv_heads + kReadThreads / 16 - 1) / (kReadThreads / 16));
  const int e = f32 ? launch_ex(int4_read_kernel<float>, grid, dim3(kReadThreads), 0, stream, kp, layer, slot, begin, end,
                                static_cast<float*>(k_out), static_cast<float*>(v_out))
                    : launch_ex(int4_read_kernel<uint16_t>, grid, dim3(kReadThreads), 0, stream, kp, layer, slot, begin, end,
                                static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out));
  if (!e) *launches += 1;
  return e;
}

}  // namespace oscar
