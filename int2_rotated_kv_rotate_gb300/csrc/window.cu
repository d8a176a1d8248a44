// Attention over the BF16 pages within a sliding window and over the first tokens (sinks): the
// query at position p attends t <= p with t < n_sink or t > p - window (window 0: all t <= p).
//
// Requests with one query (a decode step): window_rows_kernel, the split-K decode of bf16.cu over
// the list of visible tokens (the sinks, then the window), so that neither the bytes nor the values
// of other tokens are touched.  HBM-bound, 512 bytes a visible token and kv-head.
//
// Requests with more (a prompt's chunk, drafted tokens): window_tile_kernel on the tcgen05 tensor
// cores.  A tile is the G heads of a kv-head for 256 / G neighbouring queries, two blocks of 128
// rows (row m: query m / G, head m % G), over the pages that any of them sees, 128 tokens (two pages,
// not always neighbours) a step:
//   S = Q K^T      M = 128 rows, N = 128 tokens, K = 128 channels, both from shared memory;
//   P = 2^(S - m)  one thread a row, the step's whole row in registers;
//   O += P V       M = 128, N = 128 channels, K = 128 tokens, P from tensor memory.
// P is bf16 (8 bits, up to 2^-8 of each weight, at random): as V is bf16 the tensor core takes no
// other type beside it, and a second product with P's lower half would be half as much work again;
// its error is about that of the output's own rounding.  Maxima, denominators and O are fp32, and the
// denominator is the sum of the weights before their rounding.  A row's reference m moves only
// when a score exceeds it by more than kRaise (base 2), so O is rarely rescaled.
//
// Masks cost nothing in steps that every row of a block sees whole.  In the others (the window's
// edge, the diagonal, the end) a row's visible tokens are 128 bits, and the step's values are looked
// over first: an infinity or NaN in a row of values that is hidden from some row would turn that
// row's 0 into NaN in the product, so it is replaced by 0 there, and added to the rows that do see
// it when O is complete (weights are positive, so the sum is that infinity or NaN).
//
// Roles: warp 0 copies pages (TMA, a ring of five stages of 32 KB: the keys and the values of two
// pages in turn), warps 1 and 2 issue the products of S of the two blocks, 4 and 5 those of O, and
// 8-11 and 12-15 are the blocks' softmax, one thread a row.   S of a page is in
// one of two buffers of 64 columns, P over it, so that S of the next page and O of the last one are
// computed beside a page's softmax.  An item of at most 128 rows has its even pages in one block
// and its odd ones in the other, which are joined through shared memory, or by the merge.
// Where few tiles would leave SMs idle, the plan cuts their pages into parts, whose partial results
// window_merge_kernel joins, in a fixed order.
//
// Measured, G = 4, 8 kv-heads: 2048 queries behind 32768 tokens 772 to 789 us (1.36 PFLOP/s), 2 x 8192 queries
// with windows of 4096 744 to 749 us (1.27; the tensor pipe is active 57 % of the time), 16 requests of 3 to 7 drafted tokens at
// G = 8 with windows of 2048 26 us.  A page and block takes some 650 cycles, its products 512.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"
#include "packed.cuh"
#include "tmem.cuh"

namespace oscar {
namespace {

__device__ __forceinline__ const int* plan_counts(const KernelParams& kp) {
  return reinterpret_cast<const int*>(kp.base + kp.lay.window_plan);
}
__device__ __forceinline__ const WindowReq* plan_reqs(const KernelParams& kp) {
  return reinterpret_cast<const WindowReq*>(kp.base + kp.lay.window_plan + 256);
}

// ---------------------------------------------------------------- one query a request
// Row buffers of a CTA, two of them in flight, and two CTAs an SM: 64 requests of 32768 tokens with
// windows of 4096 take 178 us (6.0 TB/s), with two buffers and three CTAs 189; at ragged lengths both 66 to 68
// (4.9 TB/s).
constexpr int NBUF = 3, kRowsPerSM = 2;
constexpr int kRowsSmem(int G) { return Bf16Rows<4, NBUF>::kSmemBytes + G * kQRow * 4 + 32; }  // + flags, barrier
template <int G>
constexpr int kRowsSlabSlots = Bf16Rows<4, NBUF>::kSmemBytes / PartialSlot<G>::kBytes;

template <int G>
__global__ void __launch_bounds__(128, kRowsPerSM)
    window_rows_kernel(KernelParams kp, int layer, const uint16_t* __restrict__ q, uint8_t* __restrict__ partials,
                       uint16_t* __restrict__ out, float* __restrict__ out_f32) {
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + Bf16Rows<4, NBUF>::kSmemBytes);
  int* s_last = reinterpret_cast<int*>(smem + Bf16Rows<4, NBUF>::kSmemBytes + G * kQRow * 4);
  int* s_next = s_last + 1;
  uint64_t* slab_bar = reinterpret_cast<uint64_t*>(smem + Bf16Rows<4, NBUF>::kSmemBytes + G * kQRow * 4 + 16);
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(slab_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t slab_phase = 0;
  const int* counts = plan_counts(kp);
  const DecodeItem* items = reinterpret_cast<const DecodeItem*>(kp.base + kp.lay.window_plan + counts[4]);
  const WorkQueue wq{reinterpret_cast<unsigned*>(kp.base + kp.lay.sched), counts[0], 0, counts[0]};
  bool waited = false;
  for (int ix = wq.first(); ix >= 0; ix = wq.next(s_next)) {
    const DecodeItem it = items[ix];
    const WindowReq wr = plan_reqs(kp)[it.req];
    const size_t head0 = size_t(wr.row) * kp.n_q_heads + size_t(it.kvh) * G;
    uint8_t* part = partials + size_t(it.slot) * PartialSlot<G>::kBytes;
    const bool slot_ok = wr.slot >= 0 && wr.slot < kp.max_requests;
    if (!slot_ok && threadIdx.x == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
    const int u0 = it.begin, u1 = slot_ok ? it.end : it.begin;
    const int* ptab =
        reinterpret_cast<const int*>(kp.base + kp.lay.page_table) + size_t(slot_ok ? wr.slot : 0) * kp.max_pages_per_request;
    const uint8_t* head_base = kp.base + kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride +
                               size_t(it.kvh) * kp.lay.bf16_head_stride;
    // token u of the list: a sink or one of the window; a bad page id reads page 0 of the pool
    // instead and raises the flag
    auto row_of = [=](int u, int kv) -> const uint16_t* {
      const int t = u < wr.sinks ? u : u + wr.skip, lp = t / kPage;
      int phys = lp < kp.max_pages_per_request ? ptab[lp] : -1;
      if (phys < 0 || phys >= kp.max_pages) {
        flag(kp, OSCAR_FLAG_BAD_PAGE);
        phys = 0;
      }
      return reinterpret_cast<const uint16_t*>(head_base + size_t(phys) * kp.lay.bf16_page_stride) +
             size_t(kv * kPage + t % kPage) * kHeadDim;
    };
    auto rowK = [=](int u) { return row_of(u, 0); };
    auto rowV = [=](int u) { return row_of(u, 1); };
    int staged = 0;
    if (!waited) {
      // rows that no kernel of the step writes are copied before the wait on the preceding kernel
      if (threadIdx.x < 2 * G) prefetch_l2(q + head0 * kHeadDim + 64 * threadIdx.x);
      constexpr int kAheadTok = (NBUF > 1 ? NBUF - 1 : 1) * Bf16Rows<4, NBUF>::kChunk;
      const int upto = min(min(u1, wr.u_pre), u0 + kAheadTok);
      if (upto > u0) {
        bf16_prestage<4, NBUF>(rowK, rowV, u0, upto, smem);
        staged = upto - u0;
      }
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    for (int e = threadIdx.x; e < G * kHeadDim; e += 128) qs[(e / kHeadDim) * kQRow + e % kHeadDim] = bf16_f32(q[head0 * kHeadDim + e]);
    __syncthreads();
    auto nothing = [] {};
    bf16_rows_mma<G, 4, NBUF, decltype(rowK), decltype(rowV), decltype(nothing), NoScores, true>(rowK, rowV, u0, u1, qs, part, smem,
                                                                                                 staged, nothing);
    MergeAcc<G, 128> acc;
    if (merge_partial<G, 128>(kp, it, it.head_count, partials, acc, s_last, smem, kRowsSlabSlots<G>, smem_u32(slab_bar),
                              slab_phase, [] {})) {
      const int c = threadIdx.x;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float r = merged(acc.L[h], acc.O[h]);
        out[(head0 + h) * kHeadDim + c] = bf16_rne(r);
        if (out_f32) out_f32[(head0 + h) * kHeadDim + c] = r;
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

// ---------------------------------------------------------------- several queries a request
constexpr int kStages = 5;
constexpr int kStep = 2 * kPage;                       // tokens of a step
constexpr int kStageBytes = kStep * kHeadDim * 2;      // keys or values of a step
constexpr int kHalf = kStageBytes / 2;                 // of 64 channels
constexpr int kBlockRows = 128;
constexpr int kQBlock = kBlockRows * kHeadDim * 2;
constexpr int kThreads = 512;
static_assert(kWindowRows == 2 * kBlockRows, "warps 8-11 and 12-15");
// Registers of a thread: 128 at the launch, then as the roles need them, the same in all.
constexpr int kRegsControl = 72, kRegsSoftmax = 184;
static_assert(2 * 128 * (kRegsControl + kRegsSoftmax) <= kThreads * 128, "registers of the launch");

struct Control {
  // Stage s's completion n is its n-th filling (leaving, which both blocks' warps report).
  uint64_t full[kStages], empty[kStages];
  // Completion n is item n of those in which the block has rows.
  uint64_t q_full[2];
  // Page n of the block has buffer n % 2, whose completion is n / 2: S is written, P is written, O
  // holds the pages up to n (and P is read).
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];
  // A split item that is a whole tile: block 0's rows have O, block 1's are in shared memory, block 0
  // has read them.  Completion n is the n-th such item.
  uint64_t join_ready, join_full, join_done;
  float2 join[kBlockRows];  // maximum and denominator of block 1's rows
  uint64_t drain[4];
  uint32_t tmem;
  int abort;
  int odd;  // an infinity or NaN was met among values that not every row of a tile sees (in any of the CTA's)
};
constexpr int kOffStages = 2 * kQBlock;
constexpr int kOffControl = kOffStages + kStages * kStageBytes;
constexpr int kTileSmem = kOffControl + int(sizeof(Control)) + 1024;  // + alignment to 1024
static_assert(kTileSmem <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns of block b: two buffers of S of 64 (P over the first 32 of each), O of 128.
constexpr uint32_t kBlockCols = 256, kColO = 128;

constexpr float kRaise = 32.f;

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The n lowest bits (n in any range).
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Everything a role needs of an item: the list of pages is sink_pages pages from 0, then those
// from window_page on; step i is list pages 2 i and 2 i + 1 (the last may have only one).
struct Work {
  WindowTile it;
  WindowReq rq;
  int rows, blocks, sink_pages, window_page, pages;
  // Pages of block b: all, or, split, every other one.
  __device__ int page0(int b) const { return first_page() + (it.split ? b : 0); }
  __device__ int stride() const { return it.split ? 2 : 1; }
  // Row r of block b in the tile.
  __device__ int row(int b, int r) const { return (it.split ? 0 : b * kBlockRows) + r; }
  __device__ int page(int j) const { return j < sink_pages ? j : window_page + j - sink_pages; }
  __device__ int first_page() const { return 2 * it.begin; }
  __device__ int end_page() const { return min(2 * it.end, pages); }
  // Tokens of list page j that the query at position p sees.
  __device__ uint64_t visible(int j, int p) const {
    if (j >= pages) return 0;
    const int t0 = page(j) * kPage;
    const uint64_t upto = low_bits(p - t0 + 1);
    if (rq.window == 0) return upto;
    return upto & (~low_bits(p - rq.window - t0 + 1) | low_bits(rq.n_sink - t0));
  }
  // Tokens that some query from position p0 to p1 sees.
  __device__ uint64_t seen(int j, int p0, int p1) const {
    if (j >= pages) return 0;
    const int t0 = page(j) * kPage;
    const uint64_t upto = low_bits(p1 - t0 + 1);
    if (rq.window == 0) return upto;
    return upto & (~low_bits(p0 - rq.window - t0 + 1) | low_bits(rq.n_sink - t0));
  }
  // Pages of the list of which every query from position p0 to p1 sees all: those of the window
  // between its edge for the last query and the diagonal of the first.  (Sink pages are not counted.)
  struct Range {
    int begin, end;
    __device__ bool has(int i) const { return i >= begin && i < end; }
  };
  __device__ Range whole(int p0, int p1) const {
    const int edge = rq.window > 0 ? max(0, p1 - rq.window + 1) : 0;          // first token that all see
    const int a = max((edge + kPage - 1) / kPage, window_page), b = (p0 + 1) / kPage;  // pages [a, b)
    return {sink_pages + a - window_page, min(sink_pages + b - window_page, pages)};
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    window_tile_kernel(KernelParams kp, int layer, const __grid_constant__ CUtensorMap map, const uint16_t* __restrict__ q,
                       uint8_t* __restrict__ parts, uint16_t* __restrict__ out, float* __restrict__ out_f32) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Control* ctl = reinterpret_cast<Control*>(smem + kOffControl);
  const uint32_t sq = smem_u32(smem), sst = sq + kOffStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->q_full[b]), kBlockRows);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&ctl->s_full[b][i]), 1);
        mbar_init(smem_u32(&ctl->p_full[b][i]), kBlockRows);
        mbar_init(smem_u32(&ctl->o_done[b][i]), 1);
      }
      mbar_init(smem_u32(&ctl->drain[b]), 1);
      mbar_init(smem_u32(&ctl->drain[2 + b]), 1);
    }
    mbar_init(smem_u32(&ctl->join_ready), kBlockRows);
    mbar_init(smem_u32(&ctl->join_full), kBlockRows);
    mbar_init(smem_u32(&ctl->join_done), kBlockRows);
    ctl->abort = ctl->odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem::alloc(smem_u32(&ctl->tmem), 512);
  tmem::fence_before();
  __syncthreads();
  tmem::fence_after();
  const uint32_t tm = ctl->tmem;
  // The plan is older than the preceding kernel: only those who read rows or queries, or write
  // results, wait for it, with their first item at hand.
  const int* counts = plan_counts(kp);
  const int G = kp.gqa;
  const int* first_item = reinterpret_cast<const int*>(kp.base + kp.lay.window_plan + counts[7]);  // of each CTA
  const int ix0 = int(blockIdx.x) < counts[3] ? first_item[blockIdx.x] : 0;
  const int ix1 = int(blockIdx.x) < counts[3] ? first_item[blockIdx.x + 1] : 0;
  const WindowTile* items = reinterpret_cast<const WindowTile*>(kp.base + kp.lay.window_plan + counts[5]);
  auto load_work = [&](int ix) {
    Work w;
    w.it = items[ix];
    w.rq = plan_reqs(kp)[w.it.req];
    w.rows = w.it.n_tok * G;
    const WindowPages p = window_pages(w.rq.first + w.it.tok0, w.it.n_tok, w.rq.n_sink, w.rq.window);
    w.sink_pages = p.sink_pages;
    w.window_page = p.window_page;
    w.pages = p.pages;
    w.blocks = (w.it.split ? w.end_page() - w.first_page() > 1 : w.rows > kBlockRows) ? 2 : 1;
    return w;
  };
  // Bounded wait of a whole warp for a barrier's completion `index`.  Every lane polls: one lane's
  // polls, with the warp brought together behind them, cost some 300 cycles of each of a page's three
  // hand-overs (2432 queries on 8192 tokens: 292 against 204 us, and 188 with try_wait from the first
  // poll on, as here).  After a wait that ran out MMAs
  // and stores of that page still go out, on memory of this CTA; the roles vote once a page, and
  // every role then leaves its loop.
  auto wait = [&](uint64_t& bar, uint32_t index) -> int {
    const uint32_t a = smem_u32(&bar), par = index & 1u;
    int done = mbar_try_wait(a, par);
    for (uint32_t i = 0; i < kWaitPolls && !done; ++i) {
      done = mbar_try_wait_for(a, par, 1000000u);
      if (!done && *reinterpret_cast<volatile int*>(&ctl->abort)) break;
    }
    if (!done) {
      *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
      flag(kp, OSCAR_FLAG_TIMEOUT);
    }
    return done;
  };
  auto all = [](int done) -> bool { return __all_sync(0xffffffffu, done); };
  if (ix0 == ix1) {  // no item: the launch still orders itself after the preceding kernel
    pdl_wait();
    pdl_trigger();
  }

  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      // ---------------------------------------------------------------- pages
      uint32_t n = 0, issued = 0;  // fillings of stages: keys and values of each step in turn
      bool ok = true;
      for (int ix = ix0; ok && ix < ix1; ++ix) {
        const Work w = load_work(ix);
        const bool slot_ok = w.rq.slot >= 0 && w.rq.slot < kp.max_requests;
        if (!slot_ok && lane == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
        const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) +
                          size_t(slot_ok ? w.rq.slot : 0) * kp.max_pages_per_request;
        if (ix == ix0) {
          pdl_wait();
          pdl_trigger();
        }
        // The first item's queries go before the pages: they would come behind the copies of five stages on
        // every SM (8192 queries, window 4096: 306 against 298 us).
        if (ix == ix0)
          for (int b = 0; ok && b < w.blocks; ++b) ok = all(wait(ctl->q_full[b], 0));
        for (int i = w.it.begin; ok && i < w.it.end; ++i) {
          const int two = min(2, w.pages - 2 * i);
          int y[2] = {0, 0};
          for (int j = 0; j < two; ++j) {
            const int lp = w.page(2 * i + j);
            int phys = lp < kp.max_pages_per_request ? ptab[lp] : -1;
            if (phys < 0 || phys >= kp.max_pages) {  // page 0 instead, and the flag
              if (lane == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
              phys = 0;
            }
            y[j] = ((layer * kp.max_pages + phys) * kp.n_kv_heads + w.it.kvh) * (2 * kPage);
          }
          for (int kv = 0; ok && kv < 2; ++kv, ++n) {
            const uint32_t st = n % kStages;
            const int done = n >= kStages ? wait(ctl->empty[st], n / kStages - 1) : 1;
            if (lane == 0 && done) {  // (lane 0 polled: no copy into a stage that was not left)
              const uint32_t bar = smem_u32(&ctl->full[st]), dst = sst + st * kStageBytes;
              mbar_expect_tx(bar, two * (kStageBytes / 2));
              for (int j = 0; j < two; ++j) {
                tma_load(dst + j * (kHalf / 2), &map, 0, y[j] + kv * kPage, bar);
                tma_load(dst + kHalf + j * (kHalf / 2), &map, 64, y[j] + kv * kPage, bar);
              }
            }
            if ((ok = all(done))) issued = n + 1;
          }
        }
      }
      // the last arrivals on the stages' barriers come before the CTA leaves
      for (uint32_t k = n > kStages ? n - kStages : 0; ok && k < n; ++k) ok = all(wait(ctl->empty[k % kStages], k / kStages));
      if (!ok)  // copies still in flight land first, too
        for (uint32_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
          mbar_wait(smem_u32(&ctl->full[k % kStages]), (k / kStages) & 1u);
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------------- S = Q K^T of block b
      const int b = warp - 1;
      constexpr uint32_t kIdS = tmem::idesc_bf16(kBlockRows, kPage, false);
      const uint64_t qb = tmem::sdesc_sw128(sq + b * kQBlock, 16, 1024), kd = tmem::sdesc_sw128(sst, 16, 1024);
      uint32_t f = 0, items_done = 0, n = 0;  // fillings; items and pages of the block
      bool ok = true;
      for (int ix = ix0; ok && ix < ix1; ++ix) {
        const Work w = load_work(ix);
        const bool here = b < w.blocks;
        if (here) ok = all(wait(ctl->q_full[b], items_done++));
        for (int i = w.it.begin; ok && i < w.it.end; ++i, f += 2) {
          const uint32_t st = f % kStages;
          const int j0 = 2 * i + (w.it.split ? b : 0), j1 = here ? min(w.it.split ? j0 + 1 : j0 + 2, w.pages) : 0;
          ok = all(wait(ctl->full[st], f / kStages));
          if (j0 >= j1 && lane == 0) mbar_arrive(smem_u32(&ctl->empty[st]));
          for (int j = j0; ok && j < j1; ++j, ++n) {
            const uint32_t buf = n & 1u;
            const int done = n >= 2 ? wait(ctl->o_done[b][buf], (n >> 1) - 1) : 1;
            tmem::fence_after();
            if (elect_one()) {
              const uint32_t d = tm + b * kBlockCols + buf * kPage;
              const uint64_t kb = kd + st * (kStageBytes >> 4) + (j & 1) * (kHalf / 2 / 16);
#pragma unroll
              for (int c = 0; c < 8; ++c)
                tmem::mma_ss(d, qb + ((c >> 2) * (kQBlock / 2) + (c & 3) * 32) / 16, kb + ((c >> 2) * kHalf + (c & 3) * 32) / 16,
                             kIdS, c > 0);
              tmem::commit(smem_u32(&ctl->s_full[b][buf]));
              if (j == j1 - 1) tmem::commit(smem_u32(&ctl->empty[st]));
            }
            ok = all(done);
          }
        }
      }
      if (!ok) {  // MMAs in flight end before the tensor memory is freed
        if (elect_one()) tmem::commit(smem_u32(&ctl->drain[b]));
        __syncwarp();
        mbar_wait(smem_u32(&ctl->drain[b]), 0);
      }
    } else if (warp == 4 || warp == 5) {
      // ---------------------------------------------------------------- O += P V of block b
      const int b = warp - 4;
      constexpr uint32_t kIdO = tmem::idesc_bf16(kBlockRows, kHeadDim, true);
      const uint64_t vd = tmem::sdesc_sw128(sst, kHalf, 1024);
      uint32_t f = 1, n = 0;
      bool ok = true;
      for (int ix = ix0; ok && ix < ix1; ++ix) {
        const Work w = load_work(ix);
        const bool here = b < w.blocks;
        for (int i = w.it.begin; ok && i < w.it.end; ++i, f += 2) {
          const uint32_t st = f % kStages;
          const int j0 = 2 * i + (w.it.split ? b : 0), j1 = here ? min(w.it.split ? j0 + 1 : j0 + 2, w.pages) : 0;
          ok = all(wait(ctl->full[st], f / kStages));
          if (j0 >= j1 && lane == 0) mbar_arrive(smem_u32(&ctl->empty[st]));
          for (int j = j0; ok && j < j1; ++j, ++n) {
            const uint32_t buf = n & 1u;
            const int done = wait(ctl->p_full[b][buf], n >> 1);
            tmem::fence_after();
            if (elect_one()) {
              const uint32_t a = tm + b * kBlockCols + buf * kPage, d = tm + b * kBlockCols + kColO;
              const uint64_t vb = vd + st * (kStageBytes >> 4) + (j & 1) * (kHalf / 2 / 16);
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem::mma_ts(d, a + 8 * c, vb + c * (2048 / 16), kIdO, j > w.page0(b) || c > 0);
              tmem::commit(smem_u32(&ctl->o_done[b][buf]));
              if (j == j1 - 1) tmem::commit(smem_u32(&ctl->empty[st]));
            }
            ok = all(done);
          }
        }
      }
      if (!ok) {
        if (elect_one()) tmem::commit(smem_u32(&ctl->drain[2 + b]));
        __syncwarp();
        mbar_wait(smem_u32(&ctl->drain[2 + b]), 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------------------------------------------------------- softmax of block b
    const int b = (warp - 8) >> 2, wq = warp & 3, r = (wq << 5) | lane;
    const float scale = kLog2e * rsqrtf(float(kHeadDim));
    const uint32_t tl = tm + b * kBlockCols + (uint32_t(32 * wq) << 16);
    uint32_t n = 0, nv = 1, joins = 0;  // pages of this block; fillings up to the item's first values; joined items
    bool ok = true;
    for (int ix = ix0; ok && ix < ix1; ++ix) {
      const Work w = load_work(ix);
      if (ix == ix0) pdl_wait();
      const int first = w.first_page(), end = w.end_page(), fillings = 2 * (w.it.end - w.it.begin);
      const int m = w.row(b, r);
      const bool mine = m < w.rows;
      uint8_t* slot = parts + size_t(w.it.slot < 0 ? 0 : w.it.slot + b) * kWindowSlotBytes;  // of a part, the block's
      if (b >= w.blocks) {
        if (w.it.split && w.it.slot >= 0 && mine) reinterpret_cast<float2*>(slot)[r] = make_float2(-INFINITY, 0.f);  // no page for this block
        nv += fillings;
        continue;
      }
      // ---- Q: rows 32 wq .. 32 wq + 31 of the block, two rows of 16 chunks at a time
      {
        // (rows past the tile's read its first row, and become zeros: with a branch around each load
        // they came one after the other, 10000 cycles)
        const int tok = mine ? m / G : 0, head = mine ? m % G : 0;
        const long long row = (long long)(w.rq.row + w.it.tok0 + tok) * kp.n_q_heads + w.it.kvh * G + head;
        const unsigned some = __ballot_sync(0xffffffffu, mine);
        uint4 v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const long long src = __shfl_sync(0xffffffffu, row, 2 * k + (lane >> 4));
          v[k] = reinterpret_cast<const uint4*>(q + size_t(src) * kHeadDim)[lane & 15];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (!((some >> (2 * k + (lane >> 4))) & 1u)) v[k] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int rr = 32 * wq + 2 * k + (lane >> 4), c = lane & 15;
          *reinterpret_cast<uint4*>(smem + b * kQBlock + (c >> 3) * (kQBlock / 2) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v[k];
        }
      }
      fence_proxy_async();
      mbar_arrive(smem_u32(&ctl->q_full[b]));
      // positions of the block's first and last query and of this row's
      const int first_pos = w.rq.first + w.it.tok0, last_pos = first_pos + w.it.n_tok - 1;
      const int p0 = first_pos + w.row(b, 0) / G, p1 = min(last_pos, p0 + kBlockRows / G - 1);
      const int pos = min(p0 + r / G, p1);
      // Pages that some row of the tile does not see whole: both blocks look over their values
      // (whoever comes first replaces what the other's product reads, too).
      const Work::Range whole_in_tile = w.whole(first_pos, last_pos), whole_in_block = w.whole(p0, p1);
      float m_ref = -INFINITY, l = 0.f;
      const bool idle = w.row(b, 32 * wq) >= w.rows;  // no query in this warp's rows: P is not needed
      for (int j = w.page0(b); j < end; j += w.stride(), ++n) {
        const uint32_t buf = n & 1u;
        const bool masked = !whole_in_block.has(j);
        int done = wait(ctl->s_full[b][buf], n >> 1);
        if (!whole_in_tile.has(j)) {
          const uint32_t f = nv + 2 * ((j - first) / 2), st = f % kStages;
          done &= wait(ctl->full[st], f / kStages);
          uint4* page = reinterpret_cast<uint4*>(smem + kOffStages + st * kStageBytes + (j & 1) * (kHalf / 2)) + r;
          // 512 chunks of 64 channels, then as many of the others; 0 times an infinity or NaN is NaN
          __nv_bfloat162 sum = __float2bfloat162_rn(0.f);
          const __nv_bfloat162 zero = sum;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 v = page[(k >> 2) * (kHalf / 16) + (k & 3) * kBlockRows];
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[e]), zero, sum);
          }
          if (*reinterpret_cast<const uint32_t*>(&sum) & 0x7fff7fffu) {
            const uint64_t seen = w.seen(j, first_pos, last_pos);
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              uint32_t* at = reinterpret_cast<uint32_t*>(page + (k >> 2) * (kHalf / 16) + (k & 3) * kBlockRows);
              const int t = ((k & 3) * kBlockRows + r) / 8;  // eight chunks a token
#pragma unroll 1
              for (int e = 0; e < 4; ++e) {
                const uint32_t x = at[e];
                const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
                if (!lo && !hi) continue;
                if ((seen >> t) & 1ull) {  // (not what lies behind the last token)
                  *reinterpret_cast<volatile int*>(&ctl->odd) = 1;  // first: the other block may find only the zeros
                  __threadfence_block();
                }
                at[e] = x & (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
              }
            }
          }
          fence_proxy_async();
        }
        if (idle) {
          mbar_arrive(smem_u32(&ctl->p_full[b][buf]));
          if (!(ok = all(done))) break;
          continue;
        }
        const uint32_t ts = tl + buf * kPage;
        tmem::fence_after();
        uint32_t s[2][32];
        tmem::ld_x32(ts, s[0]);
        tmem::ld_x32(ts + 32, s[1]);
        tmem::wait_ld();
        if (masked) {
          const uint64_t see = w.visible(j, pos);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t bits = uint32_t(see >> (32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((bits >> e) & 1u)) s[c][e] = 0xff800000u;  // -inf
          }
        }
        // The weights by the reference so far, and the page's maximum beside them; where some row's
        // is above its reference by more than kRaise (so is an item's first page), the references
        // move, and the weights are taken again.
        uint32_t pw[32];
        uint64_t l2, l3;
        for (bool again = false;; again = true) {
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t scale2 = pack2(scale, scale), minus_ref = pack2(-ref, -ref);
          l2 = l3 = pack2(0.f, 0.f);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t* x = e < 16 ? s[0] + 2 * e : s[1] + 2 * (e - 16);
            mx[e & 3] = max3(mx[e & 3], __uint_as_float(x[0]), __uint_as_float(x[1]));
            float2 p = unpack2(fma2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), scale2, minus_ref));
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            if (e & 1) l2 = add2(l2, pack2(p.x, p.y));
            else l3 = add2(l3, pack2(p.x, p.y));
            pw[e] = pack_bf16(p.x, p.y);
          }
          if (again) break;
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
          if (!__any_sync(0xffffffffu, top > m_ref + kRaise)) break;  // (also from -inf)
          // all rows of the warp to their maxima, so that the others' turns come less often
          const float f = top > m_ref ? ex2(m_ref - top) : 1.f;
          m_ref = fmaxf(m_ref, top);
          l *= f;
          if (j == w.page0(b)) continue;  // (O is not there yet)
          done &= wait(ctl->o_done[b][buf ^ 1u], (n - 1) >> 1);
          tmem::fence_after();
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            uint32_t o[32];
            tmem::ld_x32(tl + kColO + c, o);
            tmem::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem::st_x32(tl + kColO + c, o);
          }
        }
        tmem::st_x32(ts, pw);
        const float2 sums = unpack2(add2(l2, l3));
        l += sums.x + sums.y;
        tmem::wait_st();
        tmem::fence_before();
        mbar_arrive(smem_u32(&ctl->p_full[b][buf]));
        if (!(ok = all(done))) break;
      }
      nv += fillings;
      if (!ok) break;
      // ---- the rows' results
      if (!(ok = all(wait(ctl->o_done[b][(n - 1) & 1u], (n - 1) >> 1)))) break;
      tmem::fence_after();
      const bool whole_tile = w.it.slot < 0, join = w.it.split && whole_tile && w.blocks == 2;
      // Joined blocks: the second's rows go through the queries' memory, which no product reads any
      // more, 16-byte chunk c of row r at c ^ (r & 7) of its 512 bytes.
      float4* joined = reinterpret_cast<float4*>(smem) + r * (kHeadDim / 4);
      float f0 = 1.f, f1 = 0.f;  // what this row's O and the joined row's count
      if (join && b == 1) {
        if (!(ok = all(wait(ctl->join_ready, joins)))) break;
        ctl->join[r] = make_float2(l == 0.f ? -INFINITY : m_ref, l);
        if (!idle) {
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            uint32_t o[32];
            tmem::ld_x32(tl + kColO + c, o);
            tmem::wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              joined[(c / 4 + e) ^ (r & 7)] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                          __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
        tmem::fence_before();
        mbar_arrive(smem_u32(&ctl->join_full));
        if (!(ok = all(wait(ctl->join_done, joins++)))) break;
        continue;
      }
      if (join) {
        mbar_arrive(smem_u32(&ctl->join_ready));
        if (!(ok = all(wait(ctl->join_full, joins)))) break;
        const float2 ml = ctl->join[r];
        const float m0 = l == 0.f ? -INFINITY : m_ref, top = fmaxf(m0, ml.x);
        if (top != -INFINITY) {
          f0 = ex2(m0 - top);
          f1 = ex2(ml.x - top);
        }
        l = fmaf(l, f0, ml.y * f1);
      }
      // Read behind every look at the row's values: its own block's (o_done), and a joined block's, at
      // other pages (join_full).
      const bool odd = *reinterpret_cast<volatile int*>(&ctl->odd) != 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      const size_t row = size_t(w.rq.row + w.it.tok0 + m / G) * kp.n_q_heads + size_t(w.it.kvh) * G + m % G;
      float* part = reinterpret_cast<float*>(slot + kBlockRows * 8) + size_t(r) * kHeadDim;
      if (mine && !whole_tile) reinterpret_cast<float2*>(slot)[r] = make_float2(l == 0.f ? -INFINITY : m_ref, l);
      if (!idle) {
        uint32_t o[2][32];  // 32 columns on their way while the last 32 are stored
        tmem::ld_x32(tl + kColO, o[0]);
#pragma unroll
        for (int c = 0; c < kHeadDim; c += 32) {
          uint32_t(&cur)[32] = o[(c / 32) & 1];
          tmem::wait_ld();
          if (c + 32 < kHeadDim) tmem::ld_x32(tl + kColO + c + 32, o[(c / 32 + 1) & 1]);
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(cur[e]) * f0;
          if (join)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 y = joined[(c / 4 + e) ^ (r & 7)];
              x[4 * e] = fmaf(y.x, f1, x[4 * e]);
              x[4 * e + 1] = fmaf(y.y, f1, x[4 * e + 1]);
              x[4 * e + 2] = fmaf(y.z, f1, x[4 * e + 2]);
              x[4 * e + 3] = fmaf(y.w, f1, x[4 * e + 3]);
            }
          if (odd && mine) {  // infinities and NaN that this row sees of the pages that were looked over
            const bool slot_ok = w.rq.slot >= 0 && w.rq.slot < kp.max_requests;
            const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) +
                              size_t(slot_ok ? w.rq.slot : 0) * kp.max_pages_per_request;
#pragma unroll 1
            for (int j = join ? first : w.page0(b); j < end; j += join ? 1 : w.stride()) {
              if (whole_in_tile.has(j)) continue;
              const uint64_t see = w.visible(j, pos);
              const int lp = w.page(j);
              int phys = see && lp < kp.max_pages_per_request ? ptab[lp] : 0;
              if (phys < 0 || phys >= kp.max_pages) phys = 0;
              const uint16_t* v = reinterpret_cast<const uint16_t*>(
                                      kp.base + kp.lay.bf16_pages + size_t(layer) * kp.lay.bf16_layer_stride +
                                      size_t(phys) * kp.lay.bf16_page_stride + size_t(w.it.kvh) * kp.lay.bf16_head_stride) +
                                  kPage * kHeadDim + c;
#pragma unroll 1
              for (int t = 0; t < kPage; ++t)
                if ((see >> t) & 1ull)
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    const float y = bf16_f32(v[t * kHeadDim + e]);
                    if (!(fabsf(y) < INFINITY)) x[e] += y;
                  }
            }
          }
          if (mine) {
            if (whole_tile) {
              uint4* dst = reinterpret_cast<uint4*>(out + row * kHeadDim + c);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dst[e] = make_uint4(pack_bf16(x[8 * e], x[8 * e + 1]), pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                                    pack_bf16(x[8 * e + 4], x[8 * e + 5]), pack_bf16(x[8 * e + 6], x[8 * e + 7]));
            }
            float4* f = whole_tile ? (out_f32 ? reinterpret_cast<float4*>(out_f32 + row * kHeadDim + c) : nullptr)
                                   : reinterpret_cast<float4*>(part + c);
            if (f)
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
      }
      tmem::fence_before();  // O is read before the next item's first MMA writes it
      if (join) {  // and the joined rows before the next queries come there
        mbar_arrive(smem_u32(&ctl->join_done));
        if (!(ok = all(wait(ctl->join_done, joins++)))) break;
      }
    }
  }
  __syncwarp();
  tmem::fence_before();
  __syncthreads();
  tmem::fence_after();
  if (warp == 0) tmem::dealloc(tm, 512);
}

// Rows of tiles whose pages were cut into parts, a warp each: the parts' results by their maxima
// and denominators, in order.
constexpr int kMergeThreads = 256;
constexpr int kMergeSplit = 4;  // CTAs to a tile
__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(KernelParams kp, const uint8_t* __restrict__ parts,
                                                                     uint16_t* __restrict__ out, float* __restrict__ out_f32) {
  const int* counts = plan_counts(kp);  // (the plan is older than the preceding kernel)
  const WindowMerge* merges = reinterpret_cast<const WindowMerge*>(kp.base + kp.lay.window_plan + counts[6]);
  bool waited = false;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = kp.gqa;
  for (int e = blockIdx.x; e < counts[2] * kMergeSplit; e += gridDim.x) {
    const WindowMerge mg = merges[e / kMergeSplit];
    const WindowReq rq = plan_reqs(kp)[mg.req];
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    for (int m = (e % kMergeSplit) * (kMergeThreads / 32) + warp; m < mg.n_tok * G; m += kMergeSplit * (kMergeThreads / 32)) {
      // part k of block m / 128: slot first_slot + stride k + m / 128
      const size_t step = size_t(mg.stride) * kWindowSlotBytes;
      const uint8_t* slot = parts + size_t(mg.first_slot + m / kBlockRows) * kWindowSlotBytes;
      const int r = m % kBlockRows;
      // lane k: part k's maximum and denominator, 32 parts at a time; the rows of eight in flight
      float top = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < mg.n_parts; k0 += 32) {
        const int n = min(32, mg.n_parts - k0);
        const float2 ml = lane < n ? reinterpret_cast<const float2*>(slot + (k0 + lane) * step)[r] : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        mx = fmaxf(mx, top);
        const float ref = mx == -INFINITY ? 0.f : mx;  // (-inf: parts that are empty or NaN)
        const float old = ex2(top - ref);               // 0 at first
        top = mx;
        const float f = ml.y == 0.f ? 0.f : ex2(ml.x - ref) * ml.y;
        const unsigned some = __ballot_sync(0xffffffffu, ml.y != 0.f);
        float sum = f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = fmaf(l, old, sum);
        o.x *= old;
        o.y *= old;
        o.z *= old;
        o.w *= old;
        for (int k = 0; k < n; k += 8) {
          float4 x[8];
          float g[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g[i] = __shfl_sync(0xffffffffu, f, (k + i) & 31);
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k + i < n && ((some >> (k + i)) & 1u))  // (a part without a visible token has no row)
              x[i] = reinterpret_cast<const float4*>(slot + (k0 + k + i) * step + kBlockRows * 8)[r * (kHeadDim / 4) + lane];
            else g[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o.x = fmaf(g[i], x[i].x, o.x);
            o.y = fmaf(g[i], x[i].y, o.y);
            o.z = fmaf(g[i], x[i].z, o.z);
            o.w = fmaf(g[i], x[i].w, o.w);
          }
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const size_t row = size_t(rq.row + mg.tok0 + m / G) * kp.n_q_heads + size_t(mg.kvh) * G + m % G;
      const float4 y = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      reinterpret_cast<uint2*>(out + row * kHeadDim)[lane] = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
      if (out_f32) reinterpret_cast<float4*>(out_f32 + row * kHeadDim)[lane] = y;
    }
  }
  if (!waited) {
    pdl_wait();
    pdl_trigger();
  }
}

template <int G>
int resident_t(int n_sm) {
  static PerDevice resident;
  return resident.get([=] {
    int e = int(cudaFuncSetAttribute(window_rows_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem(G)));
    int per_sm = 0;
    if (!e) e = int(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, window_rows_kernel<G>, 128, kRowsSmem(G)));
    return e ? -e : (per_sm > 0 ? per_sm : 1) * n_sm;
  });
}

template <int G>
int launch_rows_t(const KernelParams& kp, int layer, const void* q, void* out, float* out_f32, uint8_t* partials, int n_sm,
                  void* stream, int* launches) {
  const int resident = resident_t<G>(n_sm);
  if (resident < 0) return -resident;
  const int e = launch_ex(window_rows_kernel<G>, dim3(resident), dim3(128), size_t(kRowsSmem(G)), stream, kp, layer,
                          static_cast<const uint16_t*>(q), partials, static_cast<uint16_t*>(out), out_f32);
  if (!e) *launches += 1;
  return e;
}

}  // namespace

int window_rows_resident_ctas(int gqa, int n_sm) { return gqa == 4 ? resident_t<4>(n_sm) : resident_t<8>(n_sm); }

int launch_window(const KernelParams& kp, int layer, const void* map, const void* q, void* out, float* out_f32, uint8_t* ws,
                  const WindowWorkspace& wl, bool rows, bool tiles, bool merges, int n_sm, void* stream, int* launches) {
  int e = 0;
  if (rows)
    e = kp.gqa == 4 ? launch_rows_t<4>(kp, layer, q, out, out_f32, ws + wl.rows, n_sm, stream, launches)
                    : launch_rows_t<8>(kp, layer, q, out, out_f32, ws + wl.rows, n_sm, stream, launches);
  if (!e && tiles) {
    static PerDevice attr;
    const int ready = attr.get([] {
      const int x = int(cudaFuncSetAttribute(window_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
      return x ? -x : 1;
    });
    if (ready < 0) return -ready;
    e = launch_ex(window_tile_kernel, dim3(n_sm), dim3(kThreads), size_t(kTileSmem), stream, kp, layer,
                  *static_cast<const CUtensorMap*>(map), static_cast<const uint16_t*>(q), ws + wl.tiles,
                  static_cast<uint16_t*>(out), out_f32);
    if (!e) *launches += 1;
  }
  if (!e && merges) {
    e = launch_ex(window_merge_kernel, dim3(4 * n_sm), dim3(kMergeThreads), 0, stream, kp,
                  static_cast<const uint8_t*>(ws + wl.tiles), static_cast<uint16_t*>(out), out_f32);
    if (!e) *launches += 1;
  }
  return e;
}

}  // namespace oscar
