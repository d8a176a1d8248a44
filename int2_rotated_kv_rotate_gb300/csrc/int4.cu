// Decode attention over 4-bit pages (OSCAR_FORMAT_INT4): split-K over the plan's page ranges, the
// codes taken by the tensor cores in their stored form, as the 2-bit decode does.
//
// Persistent-style grid, 8 warps a CTA, two CTAs an SM; warp w takes every eighth half page (32
// tokens) of an item, which bulk copies bring into stages of its own (no block barriers in the
// loop).  Per 16 tokens, with mma.sync m16n8k16 (fp16 in, fp32 accumulate):
//   scores  S[t, h] = sum_c code_K[t, c] q'[c, h]; q.k = s (q . code) + z sum(q) per group, in
//           fp32.  q' is q (bf16, 8 bits) times a power of two of its head, exact in fp16 down to 2^-26 of
//           the head's largest channel;
//   values  O[c, h] += sum_t code_V[c, t] P'[t, h], P' = p s_V u_h (fp16), and sum_t p z_V in
//           fp32.  u_h, a power of two (weights of 1 stay exact), makes the head's largest p s_V so far 64
//           or more: a token counts by what it adds, not by its scale, and one that is hardly attended
//           costs the others nothing.  P' is rounded to 11 bits, 2^-11 of each token's share (the output's
//           own rounding: 2^-8 of all), or, where it is subnormal, by up to 2^-25, 2^-31 of the
//           largest share.
//           u_h rises as the p s_V of what came before fall, when the head's maximum rises; a half page
//           with a scale above 65000 / u_h is looked through for its largest p s_V.
// A nibble masked in place (w & 0x000f000f, or << 4) is an fp16 subnormal, code * 2^-24 or 16 code *
// 2^-24: one AND turns two codes into an MMA operand (one shift in four ANDs, and a byte permute in
// four for the values, whose pairs are two tokens' codes of a channel).  The 16 is folded into q'
// or into the output row's factor.
//
// Eight query heads fill the 8 columns of an MMA.  Four stand in them twice: of the scores, the lanes of
// the first columns take the block's first 8 tokens and those of the second its others, so that
// no lane's scaling and softmax is idle; of the values, the second columns sum the products of the second
// tokens (B is 0 elsewhere), and both are added at the end.
//
// Bound by HBM at 136 bytes (group 128) or 160 (group 32) a token and kv-head, and near it by a warp's
// latency over its half pages: 8 x 100000 tokens of 8 kv-heads, G = 4, 163 us (5.3 TB/s) and 195 to 198 us (5.2);
// G = 8 177 and 227; one request of 32768 tokens 14.0 to 15.1 and 15.7 us.  Where every half page holds a scale far
// above what is attended, 8 to 9 % more.  A CTA alone on an SM runs at 0.6 of the rate of
// two; 128 registers leave no room for a third.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "int4.cuh"
#include "oscar_internal.h"
#include "packed.cuh"

namespace oscar {
namespace {

constexpr int NW = 8, kThreads = 32 * NW;
constexpr int kUnit = kInt4Half;  // tokens of a stage

template <int G, int GROUP>
struct Shape4 {
  static constexpr int NG = kHeadDim / GROUP;
  static constexpr int kCodeBytes = kUnit * kInt4Row;  // K; the same of V behind them
  static constexpr int kSzBytes = kUnit * NG * 4;
  static constexpr int kStageBytes = 2 * kCodeBytes + 2 * kSzBytes;
  static constexpr int kStages = GROUP == 32 ? 2 : 3;  // two CTAs an SM
  static constexpr int kPipe = NW * kStages * kStageBytes;
  static constexpr int kQs = kPipe;                                // fp32 [G][kQRow]
  static constexpr int kBars = (kQs + G * kQRow * 4 + 15) / 16 * 16;  // NW * kStages barriers, the slab's
  static constexpr int kCtl = kBars + (NW * kStages + 1) * 8;      // last, next, poison
  static constexpr int kSmemBytes = kCtl + 16;
  static constexpr int kSlabSlots = kPipe / PartialSlot<G>::kBytes;
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert((NW * G * (kHeadDim + 4) + 8) * 4 <= kPipe, "per-warp results reuse the stages");
  static_assert(kStageBytes == int4_half_bytes(NG) && kStageBytes % 16 == 0, "bulk copies");
};

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The P' of the head's largest p s so far is kLeastPeak / 2 or more, none is above kMostP (fp16 ends at
// 65504), and u at most 2^113 (values below 2^-106 in all), so that its inverse is normal.
constexpr float kLeastPeak = 128.f, kMostP = 65000.f, kMostUp = 1.0384593717069655e34f;
__device__ __forceinline__ float rcp(float x) {  // at most 1 unit in the last place off
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Of a normal x > 0: the power of two in [x / 2, x], and a power of two's inverse.
__device__ __forceinline__ float pow2_floor(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

template <int G, int GROUP>
__global__ void __launch_bounds__(kThreads, 2) int4_split_kernel(KernelParams kp, int layer, const uint16_t* __restrict__ q,
                                                                 uint8_t* __restrict__ partials, uint16_t* __restrict__ out,
                                                                 float* __restrict__ out_f32) {
  using C = Shape4<G, GROUP>;
  constexpr int NG = C::NG, ST = C::kStages;
  constexpr int NI = G == 8 ? 2 : 1;      // tokens of a block of 16 whose scores a lane has
  constexpr int kLane0 = G == 8 ? 4 : 2;  // lanes with the same heads: from lane bit kLane0 on
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + C::kQs);
  uint64_t* all_bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* slab_bar = all_bars + NW * ST;
  int* s_last = reinterpret_cast<int*>(smem + C::kCtl);
  int* s_next = s_last + 1;
  int* s_poison = s_last + 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int col = G == 8 ? gid : gid & 3;               // the head of column gid
  const int head_lane = G == 8 ? 2 * tig : 2 * (tig & 1);  // the heads of this lane's scores: that and the next
  const int i_lane = G == 8 ? 0 : tig >> 1;              // G = 4: its tokens are gid + 8 i_lane of a block
  if (threadIdx.x == 0) {
    for (int i = 0; i <= NW * ST; ++i) mbar_init(smem_u32(&all_bars[i]), 1);
    *s_poison = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint8_t* pipe = smem + size_t(warp) * ST * C::kStageBytes;
  uint64_t* bars = all_bars + warp * ST;
  uint32_t phase_bits = 0, slab_phase = 0;  // bit st: parity of the next completion of stage st
  // The plan and the page table were uploaded before the preceding kernels, and no kernel of the
  // step writes the rows below H_pre, so the first item's pages wholly below it are copied before
  // the wait on the preceding kernel.
  const int n_items = reinterpret_cast<const int*>(kp.base + kp.lay.decode_counts)[0];
  const WorkQueue wq{reinterpret_cast<unsigned*>(kp.base + kp.lay.sched), n_items, 0, n_items};
  const float scale = kLog2e * rsqrtf(float(kHeadDim));
  bool waited = false;
  // (a CTA whose copies did not land takes no further work: *s_poison, written before the item's
  // last barriers)
  for (int ix = wq.first(); ix >= 0; ix = *s_poison ? -1 : wq.next(s_next)) {
    const DecodeItem it = reinterpret_cast<const DecodeItem*>(kp.base + kp.lay.decode_items)[ix];
    const DecodeReq dr = reinterpret_cast<const DecodeReq*>(kp.base + kp.lay.decode_reqs)[it.req];
    const bool slot_ok = dr.slot >= 0 && dr.slot < kp.max_requests;
    if (!slot_ok && threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
    const int t0 = it.begin * kPage, t1 = slot_ok && it.kind == 0 ? min(it.end * kPage, dr.L) : t0;
    const int n_units = t1 > t0 ? (t1 - t0 + kUnit - 1) / kUnit : 0;
    const int n_my = n_units > warp ? (n_units - warp + NW - 1) / NW : 0;
    // The warp's half pages: half warp % 2 of pages begin + warp / 2, + 4, ..
    static_assert(NW % 2 == 0, "a warp's half pages are the same half of their pages");
    const int page0 = it.begin + warp / 2, half = warp & 1;
    const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) +
                      size_t(slot_ok ? dr.slot : 0) * kp.max_pages_per_request + page0;
    const uint8_t* halves = kp.base + kp.lay.codes + size_t(layer) * kp.lay.codes_layer_stride +
                            size_t(it.kvh) * kp.lay.codes_head_stride + half * C::kStageBytes;
    // copy of the warp's k-th half page into stage k % ST; false (none) if the page id is out of range
    auto issue = [&](int k) -> bool {
      const int phys = page0 + NW / 2 * k < kp.max_pages_per_request ? ptab[NW / 2 * k] : -1;
      if (phys < 0 || phys >= kp.max_pages) return false;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&bars[k % ST]);
        fence_proxy_async();
        mbar_expect_tx(bar, C::kStageBytes);
        bulk_g2s(smem_u32(pipe + (k % ST) * C::kStageBytes), halves + size_t(unsigned(phys)) * unsigned(kp.lay.codes_page_stride),
                 C::kStageBytes, bar);
      }
      return true;
    };
    uint32_t ok_mask = 0;  // bit st: a copy into stage st is in flight
    int issued = 0;
    for (; issued < min(ST, n_my); ++issued) {
      if (!waited && (page0 + NW / 2 * issued + 1) * kPage > dr.H_pre) break;
      if (issue(issued)) ok_mask |= 1u << issued;
    }
    const size_t head0 = size_t(it.req) * kp.n_q_heads + size_t(it.kvh) * G;
    if (!waited) {
      if (threadIdx.x < 2 * G) prefetch_l2(q + head0 * kHeadDim + 64 * threadIdx.x);
      pdl_wait();
      pdl_trigger();
      waited = true;
      for (; issued < min(ST, n_my); ++issued)
        if (issue(issued)) ok_mask |= 1u << issued;
    }
    for (int e = threadIdx.x; e < G * kHeadDim; e += kThreads)
      qs[(e / kHeadDim) * kQRow + e % kHeadDim] = bf16_f32(q[head0 * kHeadDim + e]);
    __syncthreads();
    // ---- q' as score-MMA B fragments: column gid = head, channels 32 g + 8 tig + {n, n + 4}
    uint32_t bq[8][2];
    float back = 0.f;  // of column gid's head: what a product of codes and q' is short of, with the scale
    {
      float top = 0.f, x[4][8];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int n = 0; n < 8; n += 4) {
          const float4 v = *reinterpret_cast<const float4*>(qs + col * kQRow + 32 * g + 8 * tig + n);
          x[g][n] = v.x;
          x[g][n + 1] = v.y;
          x[g][n + 2] = v.z;
          x[g][n + 3] = v.w;
          top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(13 - exponent of the largest); the exponent is held in [-110, 100], so that this and its
      // inverse with the 2^24 stay in range
      const int ex = min(max(int((__float_as_uint(top) >> 23) & 255u) - 127, -110), 100);
      const float up = __uint_as_float(uint32_t(127 + 13 - ex) << 23);
      back = scale * __uint_as_float(uint32_t(127 + 24 - 13 + ex) << 23);
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float f = n & 1 ? up * 0.0625f : up;
          bq[2 * g + (n >> 1)][n & 1] = half2_bits(x[g][n] * f, x[g][n + 4] * f);
        }
    }
    float bk[2], qz[2][NG];
#pragma unroll
    for (int j = 0; j < 2; ++j) bk[j] = __shfl_sync(0xffffffffu, back, 4 * (head_lane + j));
    {
      // sums of q over the groups: lanes of column gid have theirs, then as above
      float sum[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        sum[g] = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) sum[g] += qs[col * kQRow + 32 * g + 8 * tig + n];
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          qz[j][g] = scale * __shfl_sync(0xffffffffu, NG == 4 ? sum[g] : (sum[0] + sum[1]) + (sum[2] + sum[3]), 4 * (head_lane + j));
    }
    // ---- the warp's half pages
    float m_run[2] = {-INFINITY, -INFINITY}, muse[2] = {0.f, 0.f}, l_part[2] = {0.f, 0.f}, zv[2][NG], oacc[8][4];
    float u[2] = {kMostUp, kMostUp};  // of this lane's two heads, before it is rounded down to a power of two
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < NG; ++g) zv[j][g] = 0.f;
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[f][e] = 0.f;
    bool broken = false;
    for (int k = 0; k < n_my; ++k) {
      const int st = k % ST;
      if ((ok_mask >> st) & 1u) {
        if (!mbar_wait(smem_u32(&bars[st]), (phase_bits >> st) & 1u)) {
          if (lane == 0) flag(kp, OSCAR_FLAG_TIMEOUT);
          broken = true;
          break;
        }
        phase_bits ^= 1u << st;
        ok_mask &= ~(1u << st);
      } else {  // a page that was not copied contributes nothing
        if (lane == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
        __syncwarp();
        if (k + ST < n_my && issue(k + ST)) ok_mask |= 1u << st;
        continue;
      }
      const int valid = t1 - (t0 + (warp + NW * k) * kUnit);  // tokens of the unit (32 or more: all)
      const uint8_t* stage = pipe + st * C::kStageBytes;
      const uint8_t* kc = stage + 16 * (tig ^ ((gid >> 1) & 3));
      const uint8_t* vc = stage + C::kCodeBytes + 16 * ((gid >> 1) ^ tig);
      const uint32_t* ksz = reinterpret_cast<const uint32_t*>(stage + 2 * C::kCodeBytes);
      const uint32_t* vsz = ksz + kUnit * NG;
      float lg[2][NI][2];  // block, token, head
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int ta = 16 * b + gid;
        const uint4 va = *reinterpret_cast<const uint4*>(kc + ta * kInt4Row);
        const uint4 vb = *reinterpret_cast<const uint4*>(kc + (ta + 8) * kInt4Row);
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        constexpr int NA = NG == 4 ? 4 : 2;  // at group 128 two chains of products
        float acc[NA][4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float(&a)[4] = acc[NG == 4 ? g : g & 1];
          if (g < NA) mma_f16_16816_first(a, wa[g] & kLow, wb[g] & kLow, wa[g] & kHigh, wb[g] & kHigh, bq[2 * g][0], bq[2 * g][1]);
          else mma_f16_16816(a, wa[g] & kLow, wb[g] & kLow, wa[g] & kHigh, wb[g] & kHigh, bq[2 * g][0], bq[2 * g][1]);
          const uint32_t sa = wa[g] >> 8, sb = wb[g] >> 8;
          mma_f16_16816(a, sa & kLow, sb & kLow, sa & kHigh, sb & kHigh, bq[2 * g + 1][0], bq[2 * g + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint32_t sz[NG];
          const uint32_t* at = ksz + (ta + 8 * (G == 8 ? i : i_lane)) * NG;
          if constexpr (NG == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            sz[0] = v.x, sz[1] = v.y, sz[2] = v.z, sz[3] = v.w;
          } else {
            sz[0] = *at;
          }
          float sum[2] = {0.f, 0.f}, off[2] = {0.f, 0.f};
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float s = bf16_lo(sz[g]), z = bf16_hi(sz[g]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              auto product = [&](int k) { return G == 8 ? acc[k][2 * i + j] : i_lane ? acc[k][2 + j] : acc[k][j]; };
              const float T = NG == 4 ? product(g) : product(0) + product(1);
              sum[j] = fmaf(T, s, sum[j]);
              off[j] = fmaf(z, qz[j][g], off[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) lg[b][i][j] = fmaf(sum[j], bk[j], off[j]);
        }
      }
      if (valid < kUnit) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (16 * b + 8 * (G == 8 ? i : i_lane) + gid >= valid) lg[b][i][0] = lg[b][i][1] = -INFINITY;
      }
      // ---- scales of the values, and the references of the maximum and of the scales
      uint32_t szv[2][NI][NG];
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t* at = vsz + (16 * b + 8 * (G == 8 ? i : i_lane) + gid) * NG;
          if constexpr (NG == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            szv[b][i][0] = v.x, szv[b][i][1] = v.y, szv[b][i][2] = v.z, szv[b][i][3] = v.w;
          } else {
            szv[b][i][0] = *at;
          }
          // (what lies behind the last token may be anything, and is multiplied by a weight of 0)
          if (valid < kUnit && 16 * b + 8 * (G == 8 ? i : i_lane) + gid >= valid)
#pragma unroll
            for (int g = 0; g < NG; ++g) szv[b][i][g] = 0u;
#pragma unroll
          for (int g = 0; g < NG; ++g) top = fmaxf(top, bf16_lo(szv[b][i][g]));
        }
      float mloc[2];
      bool rise = false, over = top * fmaxf(u[0], u[1]) > kMostP;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mloc[j] = fmaxf(fmaxf(lg[0][0][j], lg[0][NI - 1][j]), fmaxf(lg[1][0][j], lg[1][NI - 1][j]));
        rise |= mloc[j] > m_run[j];
      }
      if (__any_sync(0xffffffffu, rise || over)) {
        float down[2];  // of O
#pragma unroll
        for (int j = 0; j < 2; ++j) down[j] = pow2_inverse(pow2_floor(u[j]));
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int o = kLane0; o < 32; o <<= 1) {
            mloc[0] = fmaxf(mloc[0], __shfl_xor_sync(0xffffffffu, mloc[0], o));
            mloc[1] = fmaxf(mloc[1], __shfl_xor_sync(0xffffffffu, mloc[1], o));
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mnew = fmaxf(m_run[j], mloc[j]);
            muse[j] = mnew == -INFINITY ? 0.f : mnew;
            const float alpha = ex2(m_run[j] - muse[j]);  // 0 while the reference was -inf
            m_run[j] = mnew;
            l_part[j] *= alpha;
#pragma unroll
            for (int g = 0; g < NG; ++g) zv[j][g] *= alpha;
            down[j] *= alpha;
            u[j] = fminf(u[j] * rcp(alpha), kMostUp);
          }
          over = top * fmaxf(u[0], u[1]) > kMostP;
        }
        if (__any_sync(0xffffffffu, over)) {
          float most[2] = {0.f, 0.f};  // of p s
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              float s = bf16_lo(szv[b][i][0]);
#pragma unroll
              for (int g = 1; g < NG; ++g) s = fmaxf(s, bf16_lo(szv[b][i][g]));
#pragma unroll
              for (int j = 0; j < 2; ++j) most[j] = fmaxf(most[j], ex2(lg[b][i][j] - muse[j]) * s);
            }
#pragma unroll
          for (int o = kLane0; o < 32; o <<= 1) {
            most[0] = fmaxf(most[0], __shfl_xor_sync(0xffffffffu, most[0], o));
            most[1] = fmaxf(most[1], __shfl_xor_sync(0xffffffffu, most[1], o));
          }
          // (a scale is below 2^124, so u above 2^-118)
#pragma unroll
          for (int j = 0; j < 2; ++j) u[j] = fminf(u[j], kLeastPeak * rcp(fmaxf(most[j], kLeastPeak / kMostUp)));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) down[j] *= pow2_floor(u[j]);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          oacc[f][0] *= down[0];
          oacc[f][1] *= down[1];
          oacc[f][2] *= down[0];
          oacc[f][3] *= down[1];
        }
      }
      // ---- values
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float p[NI][2];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[i][j] = ex2(lg[b][i][j] - muse[j]);  // masked: exactly 0
            l_part[j] += p[i][j];
          }
        uint32_t bp[NG][2];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float p0 = p[i][0] * pow2_floor(u[0]), p1 = p[i][1] * pow2_floor(u[1]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float s = bf16_lo(szv[b][i][g]), z = bf16_hi(szv[b][i][g]);
            const uint32_t x = movmatrix_trans(half2_bits(p0 * s, p1 * s));
            if constexpr (G == 8) {
              bp[g][i] = x;
            } else {  // lanes of the first columns have the first tokens
              bp[g][0] = gid < 4 ? x : 0u;
              bp[g][1] = gid < 4 ? 0u : x;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) zv[j][g] = fmaf(p[i][j], z, zv[j][g]);
          }
        }
        // tokens 2 tig, + 1, + 8, + 9 of the block; chunk gid / 2 of each, its half gid % 2
        const uint8_t* at = vc + (16 * b + 2 * tig) * kInt4Row;
        const uint4 a = *reinterpret_cast<const uint4*>(at), a1 = *reinterpret_cast<const uint4*>(at + kInt4Row);
        const uint4 c = *reinterpret_cast<const uint4*>(at + 8 * kInt4Row), c1 = *reinterpret_cast<const uint4*>(at + 9 * kInt4Row);
        const uint32_t wA[4] = {a.x, a.y, a.z, a.w}, wB[4] = {a1.x, a1.y, a1.z, a1.w};
        const uint32_t wC[4] = {c.x, c.y, c.z, c.w}, wD[4] = {c1.x, c1.y, c1.z, c1.w};
        const uint32_t sel = gid & 1 ? 0x7632u : 0x5410u;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t X = permute(wA[g], wB[g], sel), Y = permute(wC[g], wD[g], sel);
          const int gg = NG == 4 ? g : 0;
          mma_f16_16816(oacc[2 * g], X & kLow, X & kHigh, Y & kLow, Y & kHigh, bp[gg][0], bp[gg][1]);
          const uint32_t X8 = X >> 8, Y8 = Y >> 8;
          mma_f16_16816(oacc[2 * g + 1], X8 & kLow, X8 & kHigh, Y8 & kLow, Y8 & kHigh, bp[gg][0], bp[gg][1]);
        }
      }
      __syncwarp();
      if (k + ST < n_my && issue(k + ST)) ok_mask |= 1u << st;
    }
    if (broken) {
      // copies still in flight land (bounded) before the stages are reused or the CTA exits
      bool drained = true;
      for (int st = 0; st < ST; ++st)
        if ((ok_mask >> st) & 1u) {
          if (mbar_wait(smem_u32(&bars[st]), (phase_bits >> st) & 1u)) phase_bits ^= 1u << st;
          else drained = false;
        }
      if (!drained && lane == 0) *s_poison = 1;
    }
    // ---- the warps' sums into the partial
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = kLane0; o < 32; o <<= 1) {
        l_part[j] += __shfl_xor_sync(0xffffffffu, l_part[j], o);
#pragma unroll
        for (int g = 0; g < NG; ++g) zv[j][g] += __shfl_xor_sync(0xffffffffu, zv[j][g], o);
      }
    if constexpr (G == 4) {  // the two halves of the tokens
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[f][e] += __shfl_xor_sync(0xffffffffu, oacc[f][e], 2);
    }
    __syncthreads();  // every warp is done with its stages
    float* wm = reinterpret_cast<float*>(smem);  // [NW][G] maxima
    float* wl = wm + NW * G;                     // [NW][G] denominators
    float* wo = wl + NW * G;                     // [NW][G][kRow]
    constexpr int kRow = kHeadDim + 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int head = head_lane + j;
      if (G == 8 || tig < 2) {
        if (gid == 0) {
          wm[warp * G + head] = broken ? -INFINITY : m_run[j];
          wl[warp * G + head] = broken ? 0.f : l_part[j];
        }
        float* mine = wo + (warp * G + head) * kRow + 4 * gid;
        const float r = pow2_inverse(pow2_floor(u[j]));
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          // rows gid: 2^-24 a code; rows gid + 8: 2^-20
          const float z = zv[j][NG == 4 ? f >> 1 : 0];
          mine[32 * (f >> 1) + 2 * (f & 1)] = fmaf(oacc[f][j] * 16777216.f, r, z);
          mine[32 * (f >> 1) + 2 * (f & 1) + 1] = fmaf(oacc[f][2 + j] * 1048576.f, r, z);
        }
      }
    }
    __syncthreads();
    uint8_t* part = partials + size_t(it.slot) * PartialSlot<G>::kBytes;
    for (int e = threadIdx.x; e < G * kHeadDim; e += kThreads) {
      const int h = e / kHeadDim, c = e % kHeadDim;
      float ms = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) ms = fmaxf(ms, wm[w * G + h]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float lw = wl[w * G + h];
        if (lw == 0.f) continue;
        const float a = ex2(wm[w * G + h] - ms);
        l = fmaf(a, lw, l);
        o = fmaf(a, wo[(w * G + h) * kRow + c], o);
      }
      store_slot<G>(part, h, c, ms, l, o);
    }
    __syncthreads();  // read before the merge's copies or the next item's
    MergeAcc<G, kThreads> acc;
    if (merge_partial<G, kThreads>(kp, it, it.head_count, partials, acc, s_last, smem, C::kSlabSlots, smem_u32(slab_bar), slab_phase,
                                   [] {})) {
      const int c = threadIdx.x & (kHeadDim - 1), hb = threadIdx.x / kHeadDim;
#pragma unroll
      for (int i = 0; i < MergeAcc<G, kThreads>::HPT; ++i) {
        const int h = hb + MergeAcc<G, kThreads>::kStride * i;
        const float o = merged(acc.L[i], acc.O[i]);
        out[(head0 + h) * kHeadDim + c] = bf16_rne(o);
        if (out_f32) out_f32[(head0 + h) * kHeadDim + c] = o;
      }
    }
    fence_proxy_async();  // generic use of the stages is over before later bulk copies
    __syncthreads();
  }
  if (!waited) {  // no item: the launch still orders itself after the preceding kernel
    pdl_wait();
    pdl_trigger();
  }
  wq.leave();
}

template <int G, int GROUP>
int resident_t(int n_sm) {
  static PerDevice resident;
  return resident.get([=] {
    int e = int(cudaFuncSetAttribute(int4_split_kernel<G, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Shape4<G, GROUP>::kSmemBytes));
    int per_sm = 0;
    if (!e)
      e = int(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, int4_split_kernel<G, GROUP>, kThreads,
                                                            Shape4<G, GROUP>::kSmemBytes));
    return e ? -e : (per_sm > 0 ? per_sm : 1) * n_sm;
  });
}

template <int G, int GROUP>
int launch_t(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, uint8_t* partials, int n_sm,
             void* stream, int* launches) {
  const int resident = resident_t<G, GROUP>(n_sm);
  if (resident < 0) return -resident;
  const int e = launch_ex(int4_split_kernel<G, GROUP>, dim3(resident), dim3(kThreads), size_t(Shape4<G, GROUP>::kSmemBytes),
                          stream, kp, layer, static_cast<const uint16_t*>(q), partials, static_cast<uint16_t*>(out), out_f32);
  if (!e) *launches += 1;
  return e;
}

}  // namespace

int int4_decode_resident_ctas(int gqa, int group, int n_sm) {
  if (gqa == 4) return group == 32 ? resident_t<4, 32>(n_sm) : resident_t<4, 128>(n_sm);
  if (gqa == 8) return group == 32 ? resident_t<8, 32>(n_sm) : resident_t<8, 128>(n_sm);
  return n_sm;
}

int launch_int4_decode(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, uint8_t* ws,
                       const DecodeWorkspace& wl, int n_sm, void* stream, int* launches) {
  uint8_t* partials = ws + wl.partials;
  if (kp.gqa == 4)
    return kp.group == 32 ? launch_t<4, 32>(kp, layer, q, out, out_f32, partials, n_sm, stream, launches)
                          : launch_t<4, 128>(kp, layer, q, out, out_f32, partials, n_sm, stream, launches);
  if (kp.gqa == 8)
    return kp.group == 32 ? launch_t<8, 32>(kp, layer, q, out, out_f32, partials, n_sm, stream, launches)
                          : launch_t<8, 128>(kp, layer, q, out, out_f32, partials, n_sm, stream, launches);
  return int(cudaErrorInvalidValue);
}

}  // namespace oscar
