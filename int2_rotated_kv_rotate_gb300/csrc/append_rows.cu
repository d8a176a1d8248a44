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
//
// 4 bits, per token and group of 32 or 128 channels: s = bf16((max - min) / 15), z = bf16(min)
// (exact), code = clamp(rint((x - z) / s), 0, 15), every operation in fp32, 0 where s = 0.  The
// quotient is taken as a product with 1 / s, which is off by 3 units in the last place at most;
// where it falls so near to a half that this could matter, the division itself decides.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "int4.cuh"
#include "oscar_internal.h"
#include "rope_dev.cuh"

namespace oscar {
namespace {

constexpr int kBatch = 4;       // rows that a half-warp loads before it stores the first
constexpr int kItemRows = 16;   // of an append item at most
constexpr int kMaxThreads = 512;

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

// The 8 channels of each of a half-warp's 16 lanes as codes (one word a lane) and the scale and
// zero point of the lane's group.  lanes: 4 or 16, those of a group.
__device__ __forceinline__ uint32_t quantize8(uint4 v, int lanes, unsigned mask, uint32_t& sz) {
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
  sz = uint32_t(s16) | (__float_as_uint(lo) & 0xffff0000u);  // (lo is one of the bf16 values, or 2^126)
  uint32_t codes = 0;
  if (s > 0.f) {
    const float inv = __fdiv_rn(1.f, s);
    bool near_half = !(inv < INFINITY);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = (x[i] - lo) * inv, c = rintf(t);
      near_half |= fabsf(t - c) > 0.5f - 1.52587890625e-5f;  // 2^-16: 16 * 3 units of 2^-24, and as much again
      codes |= uint32_t(fminf(fmaxf(c, 0.f), 15.f)) << (4 * i);
    }
    if (near_half) {
      codes = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        codes |= uint32_t(fminf(fmaxf(rintf(__fdiv_rn(x[i] - lo, s)), 0.f), 15.f)) << (4 * i);
    }
  }
  return codes;
}

template <bool INT4, bool ROPE>
__global__ void __launch_bounds__(kMaxThreads, 2) append_rows_kernel(KernelParams kp, int layer, AppendRowsParams p) {
  extern __shared__ __align__(16) float2 table[];  // [kItemRows][pairs], see slot()
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
  const int R = p.rotary_dim, pairs = R / 2;
  // the pairs in twos of 16 bytes; the twos of a lane's channels 8 of them apart (half layout) or
  // side by side, so that lanes read different banks
  auto slot = [&](int r, int pair) {
    if (p.interleaved || (pairs & 7)) return r * pairs + pair;
    return r * pairs + (((pair >> 1) & 3) * (pairs >> 3) + (pair >> 3)) * 2 + (pair & 1);
  };
  bool waited = false;
  for (int ix = blockIdx.x; ix < n_items; ix += gridDim.x) {
    const AppendItem it = reinterpret_cast<const AppendItem*>(kp.base + kp.lay.append_items)[ix];
    const AppendReq a = reinterpret_cast<const AppendReq*>(kp.base + kp.lay.append_reqs)[it.req];
    const bool slot_ok = a.slot >= 0 && a.slot < kp.max_requests;
    if (!slot_ok && threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
    const long long row0 = (long long)a.x_offset + it.begin - a.L0;
    if (waited) __syncthreads();  // the table of the item before is read
    if (!waited && (!ROPE || p.positions)) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    if constexpr (ROPE) {  // (the plan is older than the preceding kernel: places may be turned before the wait)
      for (int e = threadIdx.x; e < it.count * pairs; e += blockDim.x) {
        const int r = e / pairs, i = e - r * pairs;
        const long long pos = !p.positions ? (long long)(it.begin + r)
                              : p.positions64 ? reinterpret_cast<const long long*>(p.positions)[row0 + r]
                                              : (long long)(reinterpret_cast<const int*>(p.positions)[row0 + r]);
        const float2 cs = turn(uint64_t(pos) * p.steps[i]);
        table[slot(r, i)] = make_float2(cs.x * p.magnitude, cs.y * p.magnitude);
      }
      if (!waited) {
        pdl_wait();
        pdl_trigger();
        waited = true;
      }
      __syncthreads();
    }
    if (!mine || !slot_ok) continue;
    const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(a.slot) * kp.max_pages_per_request;
    const uint16_t* src = in + row0 * in_row;
    for (int r0 = 0; r0 < it.count; r0 += kBatch, src += kBatch * in_row) {
      uint4 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (r0 + b < it.count) x[b] = load8(src + b * in_row, in_vec);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b;
        if (r >= it.count) break;
        uint4 v = x[b];
        if (ROPE && kind != 2) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w}, y[4] = {0u, 0u, 0u, 0u};
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 2 * i < R) {
                const float2 cs = table[slot(r, c0 / 2 + i)];
                const float u = bf16_lo(w[i]), t = bf16_hi(w[i]);
                w[i] = pack_bf16(fmaf(u, cs.x, -(t * cs.y)), fmaf(u, cs.y, t * cs.x));
              }
          } else if (!(pairs & 7)) {
            const bool first = c0 < pairs;
            const int other = c0 >= R ? l16 : first ? l16 + (pairs >> 3) : l16 - (pairs >> 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(mask, w[i], other, 16);
            if (c0 < R) {
              const int pair0 = first ? c0 : c0 - pairs;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 cs = *reinterpret_cast<const float4*>(&table[slot(r, pair0 + 2 * i)]);
                const float u0 = bf16_lo(w[i]), u1 = bf16_hi(w[i]), t0 = bf16_lo(y[i]), t1 = bf16_hi(y[i]);
                // (a cos - (b sin) in the first half, a sin + (b cos) in the second: the one in
                // brackets is rounded first)
                w[i] = pack_bf16(first ? fmaf(u0, cs.x, -(t0 * cs.y)) : fmaf(t0, cs.y, u0 * cs.x),
                                 first ? fmaf(u1, cs.z, -(t1 * cs.w)) : fmaf(t1, cs.w, u1 * cs.z));
              }
            }
          } else {  // partners anywhere in the row: read one by one, before any lane stores (q may be turned in place)
            const uint16_t* row = src + b * in_row - c0;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int c = c0 + i;
              o[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
              if (c < R) {
                const bool first = c < pairs;
                const float2 cs = table[slot(r, first ? c : c - pairs)];
                const float t = bf16_f32(row[first ? c + pairs : c - pairs]);
                o[i] = first ? fmaf(o[i], cs.x, -(t * cs.y)) : fmaf(t, cs.y, o[i] * cs.x);
              }
            }
            __syncwarp(mask);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = c0 + 2 * i < R ? pack_bf16(o[2 * i], o[2 * i + 1]) : w[i];
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (kind == 0) {
          store8(static_cast<uint16_t*>(p.q.out) + (row0 + r) * p.q.out_row + h * p.q.out_head + c0, v, p.q_out_vec);
          continue;
        }
        const int pos = it.begin + r, lp = pos / kPage;
        const int phys = lp < kp.max_pages_per_request ? ptab[lp] : -1;
        if (phys < 0 || phys >= kp.max_pages) {
          if (l16 == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
          continue;
        }
        const int t = pos % kPage;
        if constexpr (!INT4) {
          uint8_t* dst = kp.base + kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride +
                         size_t(phys) * kp.lay.bf16_page_stride + size_t(h) * kp.lay.bf16_head_stride +
                         size_t(kind - 1) * (kPage * kHeadDim * 2) + size_t(t) * (kHeadDim * 2);
          reinterpret_cast<uint4*>(dst)[l16] = v;
        } else {
          const int ng = kHeadDim / kp.group;
          uint32_t sz;
          const uint32_t codes = quantize8(v, kp.group / 8, mask, sz);
          uint8_t* row = kp.base + kp.lay.codes + size_t(layer) * kp.lay.codes_layer_stride +
                         size_t(phys) * kp.lay.codes_page_stride + size_t(h) * kp.lay.codes_head_stride +
                         size_t(kind - 1) * (kPage * kInt4Row);
          *reinterpret_cast<uint32_t*>(row + int4_word(t, l16)) = codes;
          if (l16 % (kp.group / 8) == 0) {
            uint32_t* szs = reinterpret_cast<uint32_t*>(
                kp.base + kp.lay.sz + size_t(layer) * kp.lay.sz_layer_stride + size_t(phys) * kp.lay.sz_page_stride +
                size_t(h) * kp.lay.sz_head_stride + size_t(kind - 1) * (kPage * ng * 4));
            szs[t * ng + l16 / (kp.group / 8)] = sz;
          }
        }
      }
    }
  }
  if (!waited) {
    pdl_wait();
    pdl_trigger();
  }
}

// Tokens [begin, end) of a request's 4-bit rows as values: fmaf(code, s, z) in fp32, rounded to bf16
// where T is 16 bits.  Sixteen lanes a row of a head, the heads of a token side by side (K, then V).
template <typename T>
__global__ void __launch_bounds__(256) int4_read_kernel(KernelParams kp, int layer, int slot, int begin, int end,
                                                        T* __restrict__ k_out, T* __restrict__ v_out) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15, ng = kHeadDim / kp.group, Hkv = kp.n_kv_heads;
  const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(slot) * kp.max_pages_per_request;
  const long long rows = (long long)(end - begin) * 2 * Hkv;
  for (long long e = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); e < rows; e += (long long)gridDim.x * 16) {
    const int hh = int(e % (2 * Hkv)), pos = begin + int(e / (2 * Hkv));
    const int kv = hh >= Hkv, h = kv ? hh - Hkv : hh, t = pos % kPage;
    const int lp = pos / kPage;
    const int phys = lp < kp.max_pages_per_request ? ptab[lp] : -1;
    T* out = (kv ? v_out : k_out) + ((long long)(pos - begin) * Hkv + h) * kHeadDim + 8 * l16;
    float x[8];
    if (phys < 0 || phys >= kp.max_pages) {
      if (l16 == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    } else {
      const uint8_t* row = kp.base + kp.lay.codes + size_t(layer) * kp.lay.codes_layer_stride +
                           size_t(phys) * kp.lay.codes_page_stride + size_t(h) * kp.lay.codes_head_stride +
                           size_t(kv) * (kPage * kInt4Row);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + int4_word(t, l16));
      const uint32_t sz = reinterpret_cast<const uint32_t*>(
          kp.base + kp.lay.sz + size_t(layer) * kp.lay.sz_layer_stride + size_t(phys) * kp.lay.sz_page_stride +
          size_t(h) * kp.lay.sz_head_stride + size_t(kv) * (kPage * ng * 4))[t * ng + l16 / (kp.group / 8)];
      const float s = bf16_lo(sz), z = bf16_hi(sz);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(float((w >> (4 * i)) & 15u), s, z);
    }
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(out) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
      reinterpret_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

}  // namespace

int launch_append_rows(const KernelParams& kp, int layer, AppendRowsParams p, bool int4, bool rope, int n_items, void* stream,
                       int* launches) {
  // whole heads, evenly over the CTAs of an item, an even number of them in each (full warps)
  const int H = p.q.n_heads + 2 * kp.n_kv_heads, most = kMaxThreads / 16;
  const int chunks = (H + most - 1) / most;
  p.chunk_heads = ((H + chunks - 1) / chunks + 1) / 2 * 2;
  const dim3 grid(n_items, chunks), block(16 * p.chunk_heads);
  const size_t smem = rope ? size_t(kItemRows) * (p.rotary_dim / 2) * sizeof(float2) : 0;
  int e;
  if (int4) e = rope ? launch_ex(append_rows_kernel<true, true>, grid, block, smem, stream, kp, layer, p)
                     : launch_ex(append_rows_kernel<true, false>, grid, block, smem, stream, kp, layer, p);
  else e = launch_ex(append_rows_kernel<false, true>, grid, block, smem, stream, kp, layer, p);
  if (!e) *launches += 1;
  return e;
}

int launch_int4_read(const KernelParams& kp, int layer, int slot, int begin, int end, void* k_out, void* v_out, bool f32,
                     int n_sm, void* stream, int* launches) {
  const long long rows = (long long)(end - begin) * 2 * kp.n_kv_heads;
  const unsigned grid = unsigned(std::min<long long>((rows + 15) / 16, 16LL * n_sm));
  const int e = f32 ? launch_ex(int4_read_kernel<float>, dim3(grid), dim3(256), 0, stream, kp, layer, slot, begin, end,
                                static_cast<float*>(k_out), static_cast<float*>(v_out))
                    : launch_ex(int4_read_kernel<uint16_t>, dim3(grid), dim3(256), 0, stream, kp, layer, slot, begin, end,
                                static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out));
  if (!e) *launches += 1;
  return e;
}

}  // namespace oscar
