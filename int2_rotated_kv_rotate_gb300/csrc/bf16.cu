// Uncompressed comparison: split-K decode attention over plain BF16 pages, no rotation.
// The pages' speed claims compare the INT2 kernel against BF16 decoding (OSCAR technical
// summary §4; the OScaR abstract compares against BF16 FlashDecoding-v2); this kernel is
// that comparison, on the same page tables and plans.
//
// Persistent-style grid: each CTA loops over work items (pages [p0, p1) of one (request,
// kv-head)); 64-token pages are staged by cp.async and attended with bf16 tensor-core
// MMAs (bf16_rows_mma); the last CTA of each (request, kv-head) merges the partials and
// stores bf16 (and optional fp32) output.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"

namespace oscar {
namespace {

// Row buffers of a CTA: chunks of 64 tokens, NBUF - 1 of them in flight while one is
// attended.  Plans of one wave (small steps, latency-bound) run the deeper pipeline
// (NBUF 3, two CTAs per SM); larger plans NBUF 2 (three CTAs per SM, more CTAs to overlap
// one another's prologues and merges).
template <int NBUF>
constexpr int kBf16PerSM = NBUF == 3 ? 2 : 3;  // (told to the compiler, which else keeps to fewer registers and spills)
template <int G, int NBUF>
constexpr int kBf16SlabSlots = Bf16Rows<4, NBUF>::kSmemBytes / PartialSlot<G>::kBytes;

// Where the scores of an item's (request, kv-head) begin.
template <int G>
__device__ __forceinline__ size_t score_offset(const KernelParams& kp, const DecodeItem& it, const DecodeReq& dr) {
  const long long base = reinterpret_cast<const long long*>(kp.base + kp.lay.score_base)[it.req];
  return (size_t(base) + size_t(it.kvh) * size_t(dr.L)) * G;
}

// WEIGHTS: the scores (log2 units) go to scores, fp32 [kv-head][L][G] of each plan request, and
// each head's (maximum, 1 / denominator) to ml, for bf16_weights_kernel.
// after_shared: the preceding launch attends the plan's shared runs.  It waited for its own
// predecessors before it let this one start, so q and the pages are final here, and only a
// merge, which reads the shared runs' partials, waits for its end: the private items of the
// SMs that it leaves free run beside it.
template <int G, int NBUF, bool WEIGHTS>
__global__ void __launch_bounds__(128, kBf16PerSM<NBUF>) bf16_split_kernel(KernelParams kp, int layer, const uint16_t* __restrict__ q,
                                                         uint8_t* __restrict__ partials, uint16_t* __restrict__ out,
                                                         float* __restrict__ out_f32, float* __restrict__ scores,
                                                         float2* __restrict__ ml, bool after_shared) {
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + Bf16Rows<4, NBUF>::kSmemBytes);
  int* s_last_p = reinterpret_cast<int*>(smem + Bf16Rows<4, NBUF>::kSmemBytes + G * kQRow * 4);
  uint64_t* slab_bar = reinterpret_cast<uint64_t*>(smem + Bf16Rows<4, NBUF>::kSmemBytes + G * kQRow * 4 + 16);
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(slab_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t slab_phase = 0;
  // The plan and the page table were uploaded before the preceding kernels, and no kernel
  // of the step writes the rows below H_pre (the length before the step's append), so the
  // first item copies those of its first chunks before the wait on the preceding kernel.
  const int n_items = reinterpret_cast<const int*>(kp.base + kp.lay.decode_counts)[0];
  const WorkQueue wq{reinterpret_cast<unsigned*>(kp.base + kp.lay.sched), n_items, 0, n_items};
  int* s_next = s_last_p + 1;
  bool waited = false;
  for (int ix = wq.first(); ix >= 0; ix = wq.next(s_next)) {
    const DecodeItem it = reinterpret_cast<const DecodeItem*>(kp.base + kp.lay.decode_items)[ix];
    const DecodeReq dr = reinterpret_cast<const DecodeReq*>(kp.base + kp.lay.decode_reqs)[it.req];
    const size_t head0 = size_t(it.req) * kp.n_q_heads + size_t(it.kvh) * G;
    uint8_t* part = partials + size_t(it.slot) * PartialSlot<G>::kBytes;
    const bool slot_ok = dr.slot >= 0 && dr.slot < kp.max_requests;
    if (!slot_ok && threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
    int t0 = 0, t1 = 0;
    if (slot_ok && it.kind == 0) {
      t0 = it.begin * kPage;
      t1 = min(it.end * kPage, dr.L);
    }
    const int* ptab =
        reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(slot_ok ? dr.slot : 0) * kp.max_pages_per_request;
    const uint8_t* head_base = kp.base + kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride +
                               size_t(it.kvh) * kp.lay.bf16_head_stride;
    // a bad page id reads page 0 of the pool instead and raises the flag
    auto page_of = [=](int u) -> const uint16_t* {
      int phys = ptab[u / kPage];
      if (phys < 0 || phys >= kp.max_pages) {
        flag(kp, OSCAR_FLAG_BAD_PAGE);
        phys = 0;
      }
      return reinterpret_cast<const uint16_t*>(head_base + size_t(phys) * kp.lay.bf16_page_stride);
    };
    auto rowK = [=](int u) { return page_of(u) + size_t(u % kPage) * kHeadDim; };
    auto rowV = [=](int u) { return page_of(u) + size_t(kPage + u % kPage) * kHeadDim; };
    int staged = 0;
    if (!waited) {
      if (threadIdx.x < 2 * G) prefetch_l2(q + head0 * kHeadDim + 64 * threadIdx.x);  // q's lines, loaded after the wait
      constexpr int kAheadTok = (NBUF > 1 ? NBUF - 1 : 1) * Bf16Rows<4, NBUF>::kChunk;
      const int upto = min(min(t1, dr.H_pre), t0 + kAheadTok);
      if (upto > t0) {
        bf16_prestage<4, NBUF>(rowK, rowV, t0, upto, smem);
        staged = upto - t0;
      }
      if (!after_shared) pdl_wait();
      pdl_trigger();
      waited = true;
    }
    for (int e = threadIdx.x; e < G * kHeadDim; e += 128) qs[(e / kHeadDim) * kQRow + e % kHeadDim] = bf16_f32(q[head0 * kHeadDim + e]);
    __syncthreads();
    float* sc = nullptr;
    if constexpr (WEIGHTS) sc = scores + score_offset<G>(kp, it, dr);
    auto keep = [=](int h, int u, float s) {
      if constexpr (WEIGHTS) sc[size_t(u) * G + h] = s;
    };
    auto nothing = [] {};
    bf16_rows_mma<G, 4, NBUF, decltype(rowK), decltype(rowV), decltype(nothing), decltype(keep), true>(
        rowK, rowV, t0, t1, qs, part, smem, staged, nothing, keep);

    MergeAcc<G, 128> acc;
    if (merge_partial<G, 128>(kp, it, it.head_count - dr.n_shared, partials, acc, s_last_p, smem, kBf16SlabSlots<G, NBUF>, smem_u32(slab_bar), slab_phase,
                              [&] {
                                if (after_shared) pdl_wait();
                              })) {
      const int c = threadIdx.x;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float r = acc.L[h] > 0.f ? acc.O[h] / acc.L[h] : 0.f;
        out[(head0 + h) * kHeadDim + c] = bf16_rne(r);
        if (out_f32) out_f32[(head0 + h) * kHeadDim + c] = r;
        if constexpr (WEIGHTS)
          if (c == h) ml[head0 + h] = acc.L[h] > 0.f ? make_float2(acc.M[h], 1.f / acc.L[h]) : make_float2(0.f, 0.f);
      }
    }
    fence_proxy_async();  // generic use of the buffers is over before later bulk copies
  }
  if (!waited) {  // no item: the launch still orders itself after the preceding kernel
    pdl_wait();
    pdl_trigger();
  }
  wq.leave();
}

// Second pass of the decode with weights: the softmax probabilities of each (request,
// kv-head)'s tokens, summed over its G query heads, added to their accumulated weights.
// Memory-bound: 4 G + 8 bytes a token (the K and V rows of the first pass are 512), four
// tokens a thread in flight: 25 us for 8 x 100000 tokens of 8 kv-heads (7 TB/s, the scores
// partly from L2).  Storing the scores costs the first pass 40 of its 577 us there; reading the
// keys a second time instead would cost 240.  The plan's items give the work, kPiece tokens of
// one at a time.
constexpr int kWeightsThreads = 128;
constexpr int kPiece = 4 * kWeightsThreads;

template <int G>
__global__ void __launch_bounds__(kWeightsThreads) bf16_weights_kernel(KernelParams kp, const float* __restrict__ scores,
                                                                       const float2* __restrict__ ml,
                                                                       const float* weights_in, float* weights_out) {
  const int n_items = reinterpret_cast<const int*>(kp.base + kp.lay.decode_counts)[0];
  for (int ix = blockIdx.x; ix < n_items; ix += gridDim.x) {
    const DecodeItem it = reinterpret_cast<const DecodeItem*>(kp.base + kp.lay.decode_items)[ix];
    const DecodeReq dr = reinterpret_cast<const DecodeReq*>(kp.base + kp.lay.decode_reqs)[it.req];
    if (dr.slot < 0 || dr.slot >= kp.max_requests || it.kind != 0) continue;
    const int t0 = it.begin * kPage, t1 = min(it.end * kPage, dr.L);
    if (t0 + int(blockIdx.y) * kPiece >= t1) continue;
    float2 head[G];
#pragma unroll
    for (int h = 0; h < G; ++h) head[h] = ml[size_t(it.req) * kp.n_q_heads + size_t(it.kvh) * G + h];
    const float* sc = scores + score_offset<G>(kp, it, dr);
    const size_t row = (size_t(dr.slot) * kp.n_kv_heads + it.kvh) * size_t(kp.weights_stride);
    for (int p = t0 + int(blockIdx.y) * kPiece; p < t1; p += int(gridDim.y) * kPiece) {
      float4 s[4][G / 4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = p + i * kWeightsThreads + int(threadIdx.x);
        if (t < t1) {
          w[i] = weights_in ? weights_in[row + t] : 0.f;
#pragma unroll
          for (int j = 0; j < G / 4; ++j) s[i][j] = reinterpret_cast<const float4*>(sc + size_t(t) * G)[j];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = p + i * kWeightsThreads + int(threadIdx.x);
        if (t < t1) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < G / 4; ++j) {
            sum = fmaf(ex2(s[i][j].x - head[4 * j].x), head[4 * j].y, sum);
            sum = fmaf(ex2(s[i][j].y - head[4 * j + 1].x), head[4 * j + 1].y, sum);
            sum = fmaf(ex2(s[i][j].z - head[4 * j + 2].x), head[4 * j + 2].y, sum);
            sum = fmaf(ex2(s[i][j].w - head[4 * j + 3].x), head[4 * j + 3].y, sum);
          }
          weights_out[row + t] = w[i] + sum;
        }
      }
    }
  }
}

constexpr int kBf16KernelSmem(int G, int nbuf) {
  return (nbuf == 3 ? Bf16Rows<4, 3>::kSmemBytes : Bf16Rows<4, 2>::kSmemBytes) + G * kQRow * 4 + 32;  // + flags, barrier
}

template <int G, int NBUF, bool WEIGHTS = false>
int resident_ctas(int n_sm) {
  static PerDevice resident;
  return resident.get([=] {
    int e = int(cudaFuncSetAttribute(bf16_split_kernel<G, NBUF, WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kBf16KernelSmem(G, NBUF)));
    int per_sm = 0;
    if (!e)
      e = int(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, bf16_split_kernel<G, NBUF, WEIGHTS>,
                                                            128, kBf16KernelSmem(G, NBUF)));
    return e ? -e : (per_sm > 0 ? per_sm : 1) * n_sm;
  });
}

template <int G, int NBUF>
int launch_t(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, uint8_t* ws,
             const DecodeWorkspace& wl, bool after_shared, int n_sm, void* stream, int* launches) {
  uint8_t* partials = ws + wl.partials;
  const int resident = resident_ctas<G, NBUF>(n_sm);
  if (resident < 0) return -resident;
  const int grid = resident;  // persistent-style: CTAs loop over the plan's items
  int e = launch_ex(bf16_split_kernel<G, NBUF, false>, dim3(grid), dim3(128), size_t(kBf16KernelSmem(G, NBUF)), stream,
                    kp, layer, static_cast<const uint16_t*>(q), partials, static_cast<uint16_t*>(out), out_f32,
                    static_cast<float*>(nullptr), static_cast<float2*>(nullptr), after_shared);
  if (!e) *launches += 1;
  return e;
}

template <int G, int NBUF>
int launch_weights_t(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, const float* w_in,
                     float* w_out, uint8_t* ws, const WeightsWorkspace& wl, int n_sm, void* stream, int* launches) {
  const int resident = resident_ctas<G, NBUF, true>(n_sm);
  if (resident < 0) return -resident;
  float* scores = reinterpret_cast<float*>(ws + wl.scores);
  float2* ml = reinterpret_cast<float2*>(ws + wl.ml);
  int e = launch_ex(bf16_split_kernel<G, NBUF, true>, dim3(resident), dim3(128), size_t(kBf16KernelSmem(G, NBUF)), stream,
                    kp, layer, static_cast<const uint16_t*>(q), ws + wl.partials, static_cast<uint16_t*>(out), out_f32,
                    scores, ml, false);
  if (e) return e;
  *launches += 1;
  // Not as a dependent launch: its CTAs would wait in the slots that the decode's leave free
  // (8 x 100000 tokens: 609 against 600 us; not measured on plans of one wave).
  bf16_weights_kernel<G><<<dim3(4 * n_sm, 4), kWeightsThreads, 0, static_cast<cudaStream_t>(stream)>>>(kp, scores, ml, w_in,
                                                                                                       w_out);
  e = int(cudaGetLastError());
  if (!e) *launches += 1;
  return e;
}

}  // namespace

int bf16_decode_resident_ctas(int gqa, bool deep, int n_sm) {
  if (gqa == 4) return deep ? resident_ctas<4, 3>(n_sm) : resident_ctas<4, 2>(n_sm);
  if (gqa == 8) return deep ? resident_ctas<8, 3>(n_sm) : resident_ctas<8, 2>(n_sm);
  return n_sm;
}

int launch_bf16_decode_weights(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32,
                               const float* w_in, float* w_out, uint8_t* ws, const WeightsWorkspace& wl, bool deep,
                               int n_sm, void* stream, int* launches) {
  if (kp.gqa == 4)
    return deep ? launch_weights_t<4, 3>(kp, layer, q, out, out_f32, w_in, w_out, ws, wl, n_sm, stream, launches)
                : launch_weights_t<4, 2>(kp, layer, q, out, out_f32, w_in, w_out, ws, wl, n_sm, stream, launches);
  if (kp.gqa == 8)
    return deep ? launch_weights_t<8, 3>(kp, layer, q, out, out_f32, w_in, w_out, ws, wl, n_sm, stream, launches)
                : launch_weights_t<8, 2>(kp, layer, q, out, out_f32, w_in, w_out, ws, wl, n_sm, stream, launches);
  return int(cudaErrorInvalidValue);
}

int launch_bf16_decode(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, uint8_t* ws,
                       const DecodeWorkspace& wl, bool deep, bool after_shared, int n_sm, void* stream,
                       int* launches) {
  if (kp.gqa == 4)
    return deep ? launch_t<4, 3>(kp, layer, q, out, out_f32, ws, wl, after_shared, n_sm, stream, launches)
                : launch_t<4, 2>(kp, layer, q, out, out_f32, ws, wl, after_shared, n_sm, stream, launches);
  if (kp.gqa == 8)
    return deep ? launch_t<8, 3>(kp, layer, q, out, out_f32, ws, wl, after_shared, n_sm, stream, launches)
                : launch_t<8, 2>(kp, layer, q, out, out_f32, ws, wl, after_shared, n_sm, stream, launches);
  return int(cudaErrorInvalidValue);
}

}  // namespace oscar
