// Eviction from the BF16 cache by accumulated attention weight, per (request, kv-head) of one
// layer: the `keep` tokens with the greatest weight stay (equal weights: the earliest), in
// the order of their positions, and are copied into the request's new pages.
//
// evict_select_kernel, one cluster of CTAs per (request, kv-head): a radix select.  Each CTA
// keeps its slice of the row's keys in shared memory (what does not fit is read again from
// L2).
// A weight's key is its bits mapped so that unsigned order is numeric order; protected
// tokens (the sinks and the most recent ones) take the greatest key.  Three passes (11, 11
// and 10 bits) narrow down the key of the keep-th token: each CTA counts its slice of the
// row into a shared-memory histogram, and every CTA adds up the cluster's histograms through
// distributed shared memory and walks them from the top.  A last pass ranks every token:
// with g tokens above the threshold key before it and e equal to it, a kept token goes to
// index g + min(e, ties kept).
//
// evict_gather_kernel, one page of new tokens a CTA at a time: warp w copies eight tokens,
// half a warp the 256 bytes of a row of K, the other half those of V, all eight loaded
// before the first is stored.  HBM-bound: 1 KB a kept token and kv-head.
// 8 x 100000 tokens of 8 kv-heads to a quarter: selection 51 us, copy 238 us (1.64 GB, 6.9 TB/s).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"

namespace oscar {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kTile = 4 * kThreads;  // tokens a CTA takes at once: four a thread
// Unsigned key in the numeric order of w: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the CTA; `total` is the CTA's.  s_warp: two sets of a value a warp, used
// in turn, so that one barrier a call is enough.
template <typename T>
__device__ __forceinline__ T block_inclusive(T v, T (&s_warp)[2][kThreads / 32], int& turn, T& total) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) s_warp[turn][warp] = v;
  __syncthreads();
  T w = s_warp[turn][lane & (kWarps - 1)];
  turn ^= 1;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, w, d, kWarps);
    if ((lane & (kWarps - 1)) >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const T before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? v + before : v;
}

// slice_tiles: tiles whose keys the dynamic shared memory holds.
template <int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    evict_select_kernel(KernelParams kp, const float* __restrict__ weights, float* __restrict__ weights_out,
                        int* __restrict__ kept, int slice_tiles) {
  extern __shared__ __align__(16) uint4 slice[];  // [slice_tiles][kThreads]
  __shared__ uint32_t hist[3][kBins];
  __shared__ uint32_t s_warp[2][kThreads / 32];
  __shared__ uint64_t s_count;  // this CTA's tokens (above << 32 | equal) of the row
  __shared__ uint32_t s_digit[3], s_above[3];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCluster > 1 ? int(cluster.block_rank()) : 0;
  auto sync = [&] {
    if constexpr (kCluster > 1) cluster.sync();
    else __syncthreads();
  };
  int turn = 0;
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
    // this CTA's slice: whole tiles, in order; thread: tokens 4 t .. 4 t + 3 of each
    const int tiles = (rq.L + kTile - 1) / kTile, per = (tiles + kCluster - 1) / kCluster;
    const int t0 = min(tiles, rank * per), t1 = min(tiles, t0 + per);
    const bool all = rq.keep >= rq.L, choose = !all && rq.keep > 0;
    const int t_cached = min(t1, t0 + slice_tiles);
    auto token = [&](int tile) { return tile * kTile + 4 * int(threadIdx.x); };
    auto make_keys = [&](int tile) {  // (rows are whole pages long)
      const int t = token(tile), protect_from = rq.L - rq.n_recent;
      const float4 v = *reinterpret_cast<const float4*>(w + t);
      uint4 k = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
      if (t < rq.n_sink || t + 3 >= protect_from) {
        if (t < rq.n_sink || t >= protect_from) k.x = 0xffffffffu;
        if (t + 1 < rq.n_sink || t + 1 >= protect_from) k.y = 0xffffffffu;
        if (t + 2 < rq.n_sink || t + 2 >= protect_from) k.z = 0xffffffffu;
        if (t + 3 < rq.n_sink || t + 3 >= protect_from) k.w = 0xffffffffu;
      }
      return k;
    };
    auto keys = [&](int tile) { return tile < t_cached ? slice[(tile - t0) * kThreads + int(threadIdx.x)] : make_keys(tile); };
    // f(token, key) for each of the thread's tokens of a tile
    auto each = [&](int tile, auto f) {
      const int t = token(tile);
      if (t >= rq.L) return;
      const uint4 k = keys(tile);
      f(t, k.x);
      if (t + 1 < rq.L) f(t + 1, k.y);
      if (t + 2 < rq.L) f(t + 2, k.z);
      if (t + 3 < rq.L) f(t + 3, k.w);
    };
    uint32_t edge = 0, ties = 0;  // the keep-th key; tokens equal to it that stay
    uint32_t above_before = 0, equal_before = 0;
    if (choose) {
#pragma unroll 4
      for (int tile = t0; tile < t_cached; ++tile)
        if (token(tile) < rq.L) slice[(tile - t0) * kThreads + int(threadIdx.x)] = make_keys(tile);
      for (int e = threadIdx.x; e < 3 * kBins / 4; e += kThreads) reinterpret_cast<uint4*>(hist[0])[e] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      uint32_t need = uint32_t(rq.keep);
#pragma unroll
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
#pragma unroll 2
        for (int tile = t0; tile < t1; ++tile)
          each(tile, [&](int, uint32_t k) {
            if (pass == 0 || ((k ^ edge) >> (pass == 1 ? 21 : 10)) == 0u) atomicAdd(&hist[pass][(k >> shift) & mask], 1u);
          });
        sync();  // every CTA has counted
        // thread t: four bins, thread 0's the highest
        const int b0 = kBins - 4 - 4 * int(threadIdx.x);
        uint32_t c[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
          const uint32_t* h = kCluster > 1 ? cluster.map_shared_rank(&hist[pass][b0], r) : &hist[pass][b0];
          const uint4 v = *reinterpret_cast<const uint4*>(h);
          c[0] += v.w, c[1] += v.z, c[2] += v.y, c[3] += v.x;
        }
        uint32_t total;
        const uint32_t mine = c[0] + c[1] + c[2] + c[3];
        const uint32_t upto = block_inclusive(mine, s_warp, turn, total);
        if (upto >= need && upto - mine < need) {  // one thread: the keep-th token's bin is mine
          uint32_t above = upto - mine;
          int i = 0;
          while (above + c[i] < need) above += c[i++];
          s_digit[pass] = uint32_t(b0 + 3 - i);
          s_above[pass] = above;
        }
        __syncthreads();
        edge |= s_digit[pass] << shift;
        need -= s_above[pass];
      }
      ties = need;
      // ---- tokens above the edge and equal to it in the CTAs before this one
      if constexpr (kCluster > 1) {
        if (threadIdx.x == 0) s_count = 0;
        __syncthreads();
        uint32_t above = 0, equal = 0;
#pragma unroll 2
        for (int tile = t0; tile < t1; ++tile)
          each(tile, [&](int, uint32_t k) {
            above += k > edge;
            equal += k == edge;
          });
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if ((threadIdx.x & 31) == 0)
          atomicAdd(reinterpret_cast<unsigned long long*>(&s_count), (unsigned long long)above << 32 | equal);
        cluster.sync();
        uint64_t before = 0;
        for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&s_count, r);
        above_before = uint32_t(before >> 32);
        equal_before = uint32_t(before);
      }
      // ---- every token's rank: a tile holds at most 2048 of either, so both fit one word
      for (int tile = t0; tile < t1; ++tile) {
        const int t = token(tile);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < rq.L) v = *reinterpret_cast<const float4*>(w + t);
        uint32_t mine = 0;
        each(tile, [&](int, uint32_t k) { mine += k > edge ? 0x10000u : uint32_t(k == edge); });
        uint32_t total;
        const uint32_t at = block_inclusive(mine, s_warp, turn, total) - mine;
        uint32_t above = above_before + (at >> 16), equal = equal_before + (at & 0xffffu);
        each(tile, [&](int u, uint32_t k) {
          if (k > edge || (k == edge && equal < ties)) {
            const int dst = int(above + min(equal, ties));
            w_out[dst] = u == t ? v.x : u == t + 1 ? v.y : u == t + 2 ? v.z : v.w;
            idx[dst] = u;
          }
          above += k > edge;
          equal += k == edge;
        });
        above_before += total >> 16;
        equal_before += total & 0xffffu;
      }
    } else if (all) {
      for (int tile = t0; tile < t1; ++tile)
        for (int t = token(tile); t < min(token(tile) + 4, rq.L); ++t) {
          w_out[t] = w[t];
          idx[t] = t;
        }
    }
    // new tokens start at weight zero: the rest of the row
    for (int t = rq.keep + rank * kThreads + int(threadIdx.x); t < stride; t += kCluster * kThreads) w_out[t] = 0.f;
    sync();  // no CTA leaves or counts the next row while its shared memory is read
  }
}

constexpr int kGatherThreads = 256;
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(KernelParams kp, int layer,
                                                                      const int* __restrict__ kept) {
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

namespace {
template <int kCluster>
int launch_select(const KernelParams& kp, const float* weights, float* weights_out, int* kept, int n_req, int max_len,
                  int n_sm, void* stream) {
  constexpr int kTileBytes = kTile * 4, kMost = 10;  // of 8 KB: two CTAs an SM
  static PerDevice attr;
  const int ready = attr.get([] {
    const int e = int(cudaFuncSetAttribute(evict_select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMost * kTileBytes));
    return e ? -e : 1;
  });
  if (ready < 0) return -ready;
  const int tiles = (max_len + kTile - 1) / kTile, per = (tiles + kCluster - 1) / kCluster;
  const int slice_tiles = per < kMost ? per : kMost;
  const int rows = n_req * kp.n_kv_heads, clusters = rows < 8 * n_sm ? rows : 8 * n_sm;
  return launch_ex(evict_select_kernel<kCluster>, dim3(kCluster * clusters), dim3(kThreads),
                   size_t(slice_tiles) * kTileBytes, stream, kp, weights, weights_out, kept, slice_tiles);
}
}  // namespace

int launch_evict(const KernelParams& kp, int layer, const float* weights, float* weights_out, int* kept, int n_req,
                 int max_len, int max_keep_pages, int n_sm, void* stream, int* launches) {
  // CTAs of a row: as many as leave the launch one wave (two CTAs an SM), since a CTA's scans
  // and barriers take as long as some five tiles.  64 rows of 100000 tokens: 51 us with four,
  // 85 us with eight; 224 rows of up to 32768: 42 us with one, 57 us with four.
  const long long rows = (long long)n_req * kp.n_kv_heads, wave = 2LL * n_sm;
  const int tiles = (max_len + kTile - 1) / kTile;
  int e = rows * 4 > wave || tiles <= 2 ? launch_select<1>(kp, weights, weights_out, kept, n_req, max_len, n_sm, stream)
          : rows * 8 > wave             ? launch_select<4>(kp, weights, weights_out, kept, n_req, max_len, n_sm, stream)
                                        : launch_select<8>(kp, weights, weights_out, kept, n_req, max_len, n_sm, stream);
  if (e) return e;
  *launches += 1;
  // (also where no request gives tokens up: a captured launch serves later plans)
  const dim3 grid(unsigned(max_keep_pages > 0 ? max_keep_pages : 1), unsigned(kp.n_kv_heads), unsigned(n_req < 65535 ? n_req : 65535));
  // Not as a dependent launch: the selection's large shared memory would leave the copy, resident
  // before the SM is empty, little L1 for its loads in flight (361 against 300 us on 8 x 100000).
  evict_gather_kernel<<<grid, kGatherThreads, 0, static_cast<cudaStream_t>(stream)>>>(kp, layer, kept);
  e = int(cudaGetLastError());
  if (!e) *launches += 1;
  return e;
}

}  // namespace oscar
