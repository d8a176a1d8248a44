// Eviction from the BF16 cache by accumulated attention weight, per (request, kv-head) of one
// layer: the `keep` tokens with the greatest weight stay (equal weights: the earliest), in
// the order of their positions, and are copied into the request's new pages.
//
// evict_select_kernel, one cluster of kCluster CTAs per (request, kv-head): a radix select.
// A weight's key is its bits mapped so that unsigned order is numeric order; protected
// tokens (the sinks and the most recent ones) take the greatest key.  Three passes (11, 11
// and 10 bits) narrow down the key of the keep-th token: each CTA counts its slice of the
// row into a shared-memory histogram, and every CTA adds up the cluster's histograms through
// distributed shared memory and walks them from the top.  A last pass ranks every token:
// with g tokens above the threshold key before it and e equal to it, a kept token goes to
// index g + min(e, ties kept).  The row is read four times, from L2 after the first.
//
// evict_gather_kernel, one page of new tokens a CTA at a time: warp w copies eight tokens,
// half a warp the 256 bytes of a row of K, the other half those of V, all eight loaded
// before the first is stored.  HBM-bound: 1 KB a kept token and kv-head.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"

namespace oscar {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 4;
constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kTile = 4 * kThreads;  // tokens a CTA takes at once: four a thread

// Unsigned key in the numeric order of w: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the CTA of (x, y) packed in one 64-bit value; `total` is the CTA's.
__device__ __forceinline__ uint64_t block_inclusive(uint64_t v, uint64_t* s_warp, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the previous call's reads of s_warp are over
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const uint64_t s = s_warp[i];
    if (i < warp) before += s;
    total += s;
  }
  return v + before;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    evict_select_kernel(KernelParams kp, const float* __restrict__ weights, float* __restrict__ weights_out,
                        int* __restrict__ kept) {
  __shared__ uint32_t hist[3][kBins];
  __shared__ uint64_t s_warp[kThreads / 32];
  __shared__ uint64_t s_count;  // this CTA's tokens (above << 32 | equal) of the row
  __shared__ uint32_t s_digit, s_above;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank());
  pdl_wait();
  pdl_trigger();
  const int n_req = reinterpret_cast<const int*>(kp.base + kp.lay.evict_plan)[0];
  const EvictReq* reqs = reinterpret_cast<const EvictReq*>(kp.base + kp.lay.evict_plan + 256);
  const int n_rows = n_req * kp.n_kv_heads;
  const int stride = kp.weights_stride;
  for (int item = blockIdx.x / kCluster; item < n_rows; item += gridDim.x / kCluster) {
    const EvictReq rq = reqs[item / kp.n_kv_heads];
    const size_t row = (size_t(rq.slot) * kp.n_kv_heads + item % kp.n_kv_heads) * size_t(stride);
    const float* w = weights + row;
    float* w_out = weights_out + row;
    int* idx = kept + row;
    const int protect_from = rq.L - rq.n_recent;
    // this CTA's slice: whole tiles, in order
    const int tiles = (rq.L + kTile - 1) / kTile, per = (tiles + kCluster - 1) / kCluster;
    const int t0 = min(tiles, rank * per), t1 = min(tiles, t0 + per);
    auto tokens = [&](int tile, uint32_t (&key)[4], float (&val)[4]) {  // -> tokens there are
      const int t = tile * kTile + 4 * int(threadIdx.x);
      if (t >= rq.L) return 0;
      const float4 v = *reinterpret_cast<const float4*>(w + t);  // rows are whole pages long
      val[0] = v.x, val[1] = v.y, val[2] = v.z, val[3] = v.w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        key[i] = t + i < rq.n_sink || t + i >= protect_from ? 0xffffffffu : key_of(val[i]);
      return min(4, rq.L - t);
    };
    uint32_t edge = 0, ties = 0;  // the keep-th key; tokens equal to it that stay
    const bool all = rq.keep >= rq.L;
    if (!all && rq.keep > 0) {
      for (int e = threadIdx.x; e < 3 * kBins; e += kThreads) hist[0][e] = 0u;
      __syncthreads();
      uint32_t need = uint32_t(rq.keep);
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        for (int tile = t0; tile < t1; ++tile) {
          uint32_t key[4];
          float val[4];
          const int n = tokens(tile, key, val);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < n && (pass == 0 || (uint64_t(key[i]) >> (shift + (pass == 2 ? 10 : 11))) ==
                                           (uint64_t(edge) >> (shift + (pass == 2 ? 10 : 11)))))
              atomicAdd(&hist[pass][(key[i] >> shift) & mask], 1u);
        }
        cluster.sync();  // every CTA has counted
        // thread t: bins 4 t' .. 4 t' + 3 from the top
        const int b0 = kBins - 4 - 4 * int(threadIdx.x);
        uint32_t c[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
          const uint4 v = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&hist[pass][b0], r));
          c[0] += v.w, c[1] += v.z, c[2] += v.y, c[3] += v.x;
        }
        uint64_t total;
        const uint32_t mine = c[0] + c[1] + c[2] + c[3];
        const uint32_t upto = uint32_t(block_inclusive(mine, s_warp, total));
        if (upto >= need && upto - mine < need) {  // one thread: the keep-th token's bin is mine
          uint32_t above = upto - mine;
          int i = 0;
          while (above + c[i] < need) above += c[i++];
          s_digit = uint32_t(b0 + 3 - i);
          s_above = above;
        }
        __syncthreads();
        edge |= s_digit << shift;
        need -= s_above;
        __syncthreads();  // s_digit is written again by the next pass
      }
      ties = need;
    }
    // ---- ranks: tokens above the edge and equal to it, in the CTAs before this one
    uint64_t before = 0;
    if (!all && rq.keep > 0) {
      uint64_t count = 0;
      for (int tile = t0; tile < t1; ++tile) {
        uint32_t key[4];
        float val[4];
        const int n = tokens(tile, key, val);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < n) count += key[i] > edge ? uint64_t(1) << 32 : uint64_t(key[i] == edge);
      }
      uint64_t total;
      block_inclusive(count, s_warp, total);
      if (threadIdx.x == 0) s_count = total;
      cluster.sync();
      for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&s_count, r);
    }
    for (int tile = t0; tile < t1 && rq.keep > 0; ++tile) {
      uint32_t key[4];
      float val[4];
      const int n = tokens(tile, key, val), t = tile * kTile + 4 * int(threadIdx.x);
      if (all) {
        for (int i = 0; i < n; ++i) {
          w_out[t + i] = val[i];
          idx[t + i] = t + i;
        }
        continue;
      }
      uint64_t mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) mine += key[i] > edge ? uint64_t(1) << 32 : uint64_t(key[i] == edge);
      uint64_t total;
      uint64_t at = before + block_inclusive(mine, s_warp, total) - mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= n) break;
        const uint32_t above = uint32_t(at >> 32), equal = uint32_t(at);
        const int dst = int(above + min(equal, ties));
        if (key[i] > edge || (key[i] == edge && equal < ties)) {
          w_out[dst] = val[i];
          idx[dst] = t + i;
        }
        at += key[i] > edge ? uint64_t(1) << 32 : uint64_t(key[i] == edge);
      }
      before += total;
    }
    // new tokens start at weight zero: the rest of the row
    for (int t = min(rq.keep, rq.L) + rank * kThreads + int(threadIdx.x); t < stride; t += kCluster * kThreads) w_out[t] = 0.f;
    cluster.sync();  // no CTA leaves or counts the next row while its shared memory is read
  }
}

constexpr int kGatherThreads = 256;
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(KernelParams kp, int layer,
                                                                      const int* __restrict__ kept) {
  pdl_wait();
  pdl_trigger();
  const int n_req = reinterpret_cast<const int*>(kp.base + kp.lay.evict_plan)[0];
  const EvictReq* reqs = reinterpret_cast<const EvictReq*>(kp.base + kp.lay.evict_plan + 256);
  const int kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv = lane >> 4, seg = lane & 15;
  uint8_t* pool = kp.base + kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride +
                  size_t(kvh) * kp.lay.bf16_head_stride + size_t(kv) * (kPage * kHeadDim * 2) + seg * 16;
  for (int r = blockIdx.z; r < n_req; r += gridDim.z) {
    const EvictReq rq = reqs[r];
    if (rq.keep >= rq.L) continue;  // nothing moves
    const int* old_pages = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(rq.slot) * kp.max_pages_per_request;
    const int* new_pages = reinterpret_cast<const int*>(kp.base + kp.lay.evict_pages) + size_t(r) * kp.max_pages_per_request;
    const int* idx = kept + (size_t(rq.slot) * kp.n_kv_heads + kvh) * size_t(kp.weights_stride);
    for (int page = blockIdx.x; page * kPage < rq.keep; page += gridDim.x) {
      const int phys = new_pages[page];
      if (phys < 0 || phys >= kp.max_pages) {
        if (threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
        continue;
      }
      uint8_t* dst = pool + size_t(phys) * kp.lay.bf16_page_stride;
      const int row0 = 8 * warp, n = min(8, rq.keep - page * kPage - row0);
      uint4 v[8];
      bool ok[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ok[i] = false;
        if (i < n) {
          const int t = idx[page * kPage + row0 + i];
          const int from = t >= 0 && t < rq.L ? old_pages[t / kPage] : -1;
          if (from < 0 || from >= kp.max_pages) {
            if (lane == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
            continue;
          }
          ok[i] = true;
          v[i] = __ldcs(reinterpret_cast<const uint4*>(pool + size_t(from) * kp.lay.bf16_page_stride + size_t(t % kPage) * (kHeadDim * 2)));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (ok[i]) __stcs(reinterpret_cast<uint4*>(dst + size_t(row0 + i) * (kHeadDim * 2)), v[i]);
    }
  }
}

}  // namespace

int launch_evict(const KernelParams& kp, int layer, const float* weights, float* weights_out, int* kept, int n_req,
                 int max_keep_pages, int n_sm, void* stream, int* launches) {
  const int rows = n_req * kp.n_kv_heads;
  const int clusters = rows < 4 * n_sm ? rows : 4 * n_sm;
  int e = launch_ex(evict_select_kernel, dim3(kCluster * clusters), dim3(kThreads), 0, stream, kp, weights, weights_out,
                    kept);
  if (e) return e;
  *launches += 1;
  if (max_keep_pages <= 0) return 0;  // no request gives tokens up and keeps any
  const dim3 grid(unsigned(max_keep_pages), unsigned(kp.n_kv_heads), unsigned(n_req < 65535 ? n_req : 65535));
  e = launch_ex(evict_gather_kernel, grid, dim3(kGatherThreads), 0, stream, kp, layer, static_cast<const int*>(kept));
  if (!e) *launches += 1;
  return e;
}

}  // namespace oscar
