// Decode attention over the runs of BF16 pages that several requests of a plan share: each
// run is read once for all of them.  The launch comes before the decode's own and writes the
// partial slots (maximum, denominator, output) that the decode's merge then joins with each
// request's private items.
//
// An item is a range of pages of one kv-head and up to 256 query rows: the G heads of the
// members that share it, 128 rows a block.  Per 64-token page, on the tcgen05 tensor cores:
//   S = Q K^T      M = 128 rows, N = 64 tokens, K = 128 channels: Q and the page's keys in
//                  shared memory, 128-byte swizzle, S in tensor memory;
//   P = 2^(S - m)  one thread a row: the whole row of the page in registers, so its maximum
//                  and sum need no other thread; P goes back as bf16 hi and lo halves (16
//                  bits, as the private items keep);
//   O += P V       M = 128, N = 128 channels, K = 64 tokens, hi then lo: P from tensor memory,
//                  the page's values in shared memory as they are stored (channels contiguous).
// The reference m of a row moves only when a score exceeds it by more than 32 (base 2), so O is
// rarely rescaled in tensor memory; p <= 2^32 loses nothing in bf16 and fp32, whose range is
// 2^127 (values up to 2^78 and 100000 tokens stay inside).
//
// Roles: warp 0 copies pages (TMA, kStages of them, keys and values apart), warp 1 issues the
// MMAs of S and warp 2 those of O (one warp for both spent 2700 cycles a page on its waits and
// issues), warps 4-7 and 8-11 are the softmax of two blocks: two row blocks over the same pages,
// or, for runs of at most 128 rows, the even and the odd pages of one row block, each with a
// partial slot of its own (one block's chain of S, softmax and O took 2400 cycles a page, more
// than the 1470 of an SM's share of the copy rate for its 32 KB).  S of a block's next page is
// computed as soon as its softmax has read this one's, beside O of the page before: a buffer of
// S and one of P a block, 512 tensor-memory columns in all.  (With P over S in two buffers, S of
// page n + 1 waited for O of page n - 1: 117.5 against 114.8 us a call on 64 requests of 33000
// shared tokens at GQA 8.)
//
// Measured (one launch, cold): 8 requests at GQA 4 on 65536 tokens of 8 kv-heads, 268 MB, 51.6 us
// (5.2 TB/s); 32 requests at GQA 8, 87.9 us, where a page and block takes 1500 cycles, 768 of the
// tensor pipe and about as many of shared memory for the MMAs' operands and the copies: neither
// is the bound; what is left is the chain of a block's S, softmax, P and O.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "oscar_internal.h"
#include "tmem.cuh"

namespace oscar {
namespace {

constexpr int kStages = 5;
constexpr int kBlockRows = 128;
constexpr int kPageKv = 2 * kPage * kHeadDim * 2;         // bytes of a page's K and V rows of a head
constexpr int kQBlock = kBlockRows * kHeadDim * 2;        // bytes of a row block of Q
constexpr int kThreads = 384;
constexpr int kBlocks = kSharedRows / kBlockRows;
static_assert(kBlocks == 2, "warps 4-7 and 8-11");

struct Control {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  // Completion n is item n of those in which the block has a page.  (A split item of one page
  // leaves block 1 none.  Arriving for it all the same, block 1 would run ahead over such items:
  // nothing there waits for the warp of S, which waits for each of them in order.)
  uint64_t q_full[kBlocks];
  // Completion n of each is page n of the block: S is written, S is read, P is written, P is
  // read and O holds the pages up to n.  Whoever waits for one of them waits for every page in
  // order, and none gets two ahead (a parity tells a completion from its neighbours only).
  uint64_t s_full[kBlocks], s_empty[kBlocks], p_full[kBlocks], o_done[kBlocks];
  uint64_t drain[2];
  uint32_t tmem;
  int abort;
};
constexpr int kOffStages = kBlocks * kQBlock;
constexpr int kOffControl = kOffStages + kStages * kPageKv;
constexpr int kSmemBytes = kOffControl + int(sizeof(Control)) + 1024;  // + alignment to 1024
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns of block b: S of 64, P of 64 (hi, lo), O of 128.
constexpr uint32_t kBlockCols = 256, kColP = 64, kColO = 128;

// A row's reference moves when a score exceeds it by this much (base 2).
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
// Two floats in one register pair, and sums and products of both at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Everything a role needs of an item.  Blocks are row blocks over all pages, or (split) the
// even and the odd pages of one row block.
struct Work {
  SharedItem it;
  int rows, blocks, pages;
  __device__ int pages_of(int b) const { return it.split ? (pages + 1 - b) / 2 : pages; }
  __device__ int row0(int b) const { return it.split ? 0 : b * kBlockRows; }
};

__global__ void __launch_bounds__(kThreads, 1)
    shared_kernel(KernelParams kp, int layer, const __grid_constant__ CUtensorMap map, const uint16_t* __restrict__ q,
                  uint8_t* __restrict__ partials) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Control* ctl = reinterpret_cast<Control*>(smem + kOffControl);
  const uint32_t sq = smem_u32(smem), sst = sq + kOffStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&ctl->k_full[i]), 1);
      mbar_init(smem_u32(&ctl->k_empty[i]), 1);
      mbar_init(smem_u32(&ctl->v_full[i]), 1);
      mbar_init(smem_u32(&ctl->v_empty[i]), 1);
    }
    for (int b = 0; b < kBlocks; ++b) {
      mbar_init(smem_u32(&ctl->q_full[b]), kBlockRows);
      mbar_init(smem_u32(&ctl->s_full[b]), 1);
      mbar_init(smem_u32(&ctl->s_empty[b]), kBlockRows);
      mbar_init(smem_u32(&ctl->p_full[b]), kBlockRows);
      mbar_init(smem_u32(&ctl->o_done[b]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctl->drain[i]), 1);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem::alloc(smem_u32(&ctl->tmem), 512);
  tmem::fence_before();
  __syncthreads();
  tmem::fence_after();
  const uint32_t tm = ctl->tmem;
  pdl_wait();
  pdl_trigger();
  const int n_items = reinterpret_cast<const int*>(kp.base + kp.lay.decode_counts)[3];
  const DecodeReq* reqs = reinterpret_cast<const DecodeReq*>(kp.base + kp.lay.decode_reqs);
  const int* order = reinterpret_cast<const int*>(kp.base + kp.lay.shared_order);
  const SharedItem* items = reinterpret_cast<const SharedItem*>(kp.base + kp.lay.shared_items);
  auto load_work = [&](int ix) {
    Work w;
    w.it = items[ix];
    w.rows = (w.it.hi - w.it.lo) * kp.gqa;
    w.blocks = w.it.split ? 2 : (w.rows + kBlockRows - 1) / kBlockRows;
    w.pages = w.it.end - w.it.begin;
    return w;
  };
  // Bounded wait of a whole warp for completions of one or two barriers (index: parity of the
  // completion).  Lane 0 polls the first, lane 1 the second: each polling lane costs the
  // barrier's bank a turn, and two waits one after the other twice a wait's 200 cycles.  The
  // __syncwarp orders what they saw before what the others do next; a vote would not.  Each lane
  // has its own poll's result: the roles vote once a page, where the warp meets anyway, so after
  // a wait that ran out MMAs and stores of that page still go out, on memory of this CTA, and
  // every role then leaves its loop.
  auto wait2 = [&](uint64_t& bar0, uint32_t index0, uint64_t& bar1, uint32_t index1) -> int {
    int done = 1;
    if (lane < 2) {
      const uint32_t a = lane ? smem_u32(&bar1) : smem_u32(&bar0), par = (lane ? index1 : index0) & 1u;
      done = mbar_try_wait(a, par);
      for (uint32_t i = 0; i < kWaitPolls && !done; ++i) {
        done = mbar_try_wait_for(a, par, 1000000u);
        if (!done && *reinterpret_cast<volatile int*>(&ctl->abort)) break;
      }
      if (!done) {
        *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        flag(kp, OSCAR_FLAG_TIMEOUT);
      }
    }
    __syncwarp();
    return done;
  };
  auto wait = [&](uint64_t& bar, uint32_t index) -> int {
    int done = 1;
    if (lane == 0) {
      const uint32_t a = smem_u32(&bar);
      done = mbar_try_wait(a, index & 1u);
      for (uint32_t i = 0; i < kWaitPolls && !done; ++i) {
        done = mbar_try_wait_for(a, index & 1u, 1000000u);
        if (!done && *reinterpret_cast<volatile int*>(&ctl->abort)) break;
      }
      if (!done) {
        *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        flag(kp, OSCAR_FLAG_TIMEOUT);
      }
    }
    __syncwarp();
    return done;
  };

  auto all = [](int done) -> bool { return __all_sync(0xffffffffu, done); };

  if (warp == 0) {
    // ---------------------------------------------------------------- pages
    uint32_t cnt = 0, nk = 0, nv = 0;  // pages; copies of keys and of values issued
    bool ok = true;
    for (int ix = blockIdx.x; ok && ix < n_items; ix += gridDim.x) {
      const Work w = load_work(ix);
      const int slot = reqs[order[w.it.lo]].slot;  // every member maps the same pages
      const bool slot_ok = slot >= 0 && slot < kp.max_requests;
      if (!slot_ok && lane == 0) flag(kp, OSCAR_FLAG_BAD_SLOT);
      const int* ptab = reinterpret_cast<const int*>(kp.base + kp.lay.page_table) +
                        size_t(slot_ok ? slot : 0) * kp.max_pages_per_request;
      int next = w.it.begin < kp.max_pages_per_request ? ptab[w.it.begin] : -1;
      for (int p = 0; p < w.pages; ++p, ++cnt) {
        const uint32_t st = cnt % kStages;
        int phys = next;
        next = p + 1 < w.pages && w.it.begin + p + 1 < kp.max_pages_per_request ? ptab[w.it.begin + p + 1] : -1;
        if (phys < 0 || phys >= kp.max_pages) {  // page 0 instead, and the flag
          if (lane == 0) flag(kp, OSCAR_FLAG_BAD_PAGE);
          phys = 0;
        }
        const int y = ((layer * kp.max_pages + phys) * kp.n_kv_heads + w.it.kvh) * (2 * kPage);
        const uint32_t dst = sst + st * kPageKv;
        int done = cnt >= kStages ? wait(ctl->k_empty[st], cnt / kStages - 1) : 1;
        if (lane == 0 && done) {  // (lane 0 polled: no copy into a stage that was not left)
          const uint32_t bar = smem_u32(&ctl->k_full[st]);
          mbar_expect_tx(bar, kPageKv / 2);
          tma_load(dst, &map, 0, y, bar);
          tma_load(dst + 8192, &map, 64, y, bar);
        }
        if (!(ok = all(done))) break;
        nk = cnt + 1;
        done = cnt >= kStages ? wait(ctl->v_empty[st], cnt / kStages - 1) : 1;
        if (lane == 0 && done) {
          const uint32_t bar = smem_u32(&ctl->v_full[st]);
          mbar_expect_tx(bar, kPageKv / 2);
          tma_load(dst + 16384, &map, 0, y + kPage, bar);
          tma_load(dst + 24576, &map, 64, y + kPage, bar);
        }
        if (!(ok = all(done))) break;
        nv = cnt + 1;
      }
    }
    // the last arrivals on the stages' barriers come before the CTA leaves
    for (uint32_t k = cnt > kStages ? cnt - kStages : 0; ok && k < cnt; ++k)
      ok = all(wait2(ctl->k_empty[k % kStages], k / kStages, ctl->v_empty[k % kStages], k / kStages));
    if (!ok) {  // copies still in flight land first, too
      for (uint32_t k = nk > kStages ? nk - kStages : 0; k < nk; ++k)
        mbar_wait(smem_u32(&ctl->k_full[k % kStages]), (k / kStages) & 1u);
      for (uint32_t k = nv > kStages ? nv - kStages : 0; k < nv; ++k)
        mbar_wait(smem_u32(&ctl->v_full[k % kStages]), (k / kStages) & 1u);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S = Q K^T
    constexpr uint32_t kIdS = tmem::idesc_bf16(kBlockRows, kPage, false);
    const uint64_t qd = tmem::sdesc_sw128(sq, 16, 1024), kd = tmem::sdesc_sw128(sst, 16, 1024);
    uint32_t st = 0, lap = 0;                      // stage, and laps of the stages
    uint32_t q0 = 0, q1 = 0, n0 = 0, n1 = 0;       // items and pages of each block
    bool ok = true;
    for (int ix = blockIdx.x; ok && ix < n_items; ix += gridDim.x) {
      const Work w = load_work(ix);
      ok = all(wait(ctl->q_full[0], q0++));
      if (ok && w.blocks > 1 && w.pages_of(1) > 0) ok = all(wait(ctl->q_full[1], q1++));
      for (int i = 0; ok && i < w.pages; ++i) {
        const int b0 = w.it.split ? i & 1 : 0, b1 = w.it.split ? b0 + 1 : w.blocks;
        for (int b = b0; ok && b < b1; ++b) {
          const uint32_t n = b ? n1++ : n0++;
          int done = 1;
          if (b == b0) done = n ? wait2(ctl->k_full[st], lap, ctl->s_empty[b], n - 1) : wait(ctl->k_full[st], lap);
          else if (n) done = wait(ctl->s_empty[b], n - 1);
          tmem::fence_after();
          if (elect_one()) {
            const uint32_t d = tm + b * kBlockCols;
            const uint64_t qb = qd + b * (kQBlock >> 4), kb = kd + st * (kPageKv >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tmem::mma_ss(d, qb + ((k >> 2) * (kQBlock / 2) + (k & 3) * 32) / 16, kb + ((k >> 2) * 8192 + (k & 3) * 32) / 16,
                           kIdS, k > 0);
            tmem::commit(smem_u32(&ctl->s_full[b]));
            if (b == b1 - 1) tmem::commit(smem_u32(&ctl->k_empty[st]));
          }
          ok = all(done);
        }
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    if (!ok) {  // MMAs in flight end before the tensor memory is freed
      if (elect_one()) tmem::commit(smem_u32(&ctl->drain[0]));
      __syncwarp();
      mbar_wait(smem_u32(&ctl->drain[0]), 0);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- O += P V
    constexpr uint32_t kIdO = tmem::idesc_bf16(kBlockRows, kHeadDim, true);
    const uint64_t vd = tmem::sdesc_sw128(sst + 16384, 8192, 1024);
    uint32_t st = 0, lap = 0, n0 = 0, n1 = 0;
    bool ok = true;
    for (int ix = blockIdx.x; ok && ix < n_items; ix += gridDim.x) {
      const Work w = load_work(ix);
      int l0 = 0, l1 = 0;
      for (int i = 0; ok && i < w.pages; ++i) {
        const int b0 = w.it.split ? i & 1 : 0, b1 = w.it.split ? b0 + 1 : w.blocks;
        for (int b = b0; ok && b < b1; ++b) {
          const uint32_t n = b ? n1++ : n0++;
          const bool first = (b ? l1++ : l0++) == 0;
          const int done = b == b0 ? wait2(ctl->v_full[st], lap, ctl->p_full[b], n) : wait(ctl->p_full[b], n);
          tmem::fence_after();
          if (elect_one()) {
            const uint32_t d = tm + b * kBlockCols + kColO, a = tm + b * kBlockCols + kColP;
            const uint64_t vb = vd + st * (kPageKv >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // hi then lo
              tmem::mma_ts(d, a + 8 * k, vb + (k & 3) * (2048 / 16), kIdO, !first || k > 0);
            tmem::commit(smem_u32(&ctl->o_done[b]));
            if (b == b1 - 1) tmem::commit(smem_u32(&ctl->v_empty[st]));
          }
          ok = all(done);
        }
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    if (!ok) {
      if (elect_one()) tmem::commit(smem_u32(&ctl->drain[1]));
      __syncwarp();
      mbar_wait(smem_u32(&ctl->drain[1]), 0);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax of block b
    const int b = (warp - 4) >> 2, wq = warp & 3, r = (wq << 5) | lane;
    const float scale = kLog2e * rsqrtf(float(kHeadDim));
    const uint32_t tl = tm + b * kBlockCols + (uint32_t(32 * wq) << 16);
    const int G = kp.gqa;
    uint32_t n = 0;  // pages of this block so far
    bool ok = true;
    for (int ix = blockIdx.x; ok && ix < n_items; ix += gridDim.x) {
      const Work w = load_work(ix);
      if (b >= w.blocks) continue;
      const int pages = w.pages_of(b);
      // the partial slot of row m's member
      auto slot_of = [&](int m) {
        const DecodeReq& dr = reqs[order[w.it.lo + m / G]];
        return partials + (size_t(dr.first_item) + size_t(w.it.kvh) * dr.items_per_head + w.it.seg + (w.it.split ? b : 0)) *
                              size_t(G) * (8 + 4 * kHeadDim);
      };
      if (pages == 0) {  // nothing attended: the merge reads no more than this of the slot
        const int m = w.row0(b) + r;
        if (m < w.rows) reinterpret_cast<float2*>(slot_of(m))[m % G] = make_float2(-INFINITY, 0.f);
        continue;
      }
      // ---- Q: rows 32 wq .. 32 wq + 31 of the block, two rows of 16 chunks at a time
      {
        // lane: the member of its row; then all loads before the first store
        const int m = w.row0(b) + r;
        const int req = m < w.rows ? order[w.it.lo + m / G] : -1;
        const int head = w.it.kvh * G + m % G;
        const int row_of_q = req >= 0 ? req * kp.n_q_heads + head : -1;
        uint4 v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int src = __shfl_sync(0xffffffffu, row_of_q, 2 * k + (lane >> 4));
          v[k] = src >= 0 ? reinterpret_cast<const uint4*>(q + size_t(src) * kHeadDim)[lane & 15] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int row = 32 * wq + 2 * k + (lane >> 4), c = lane & 15;
          *reinterpret_cast<uint4*>(smem + b * kQBlock + (c >> 3) * (kQBlock / 2) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[k];
        }
      }
      fence_proxy_async();
      mbar_arrive(smem_u32(&ctl->q_full[b]));
      float m_ref = -INFINITY, l = 0.f;
      const bool idle = w.row0(b) + 32 * wq >= w.rows;  // no query in this warp's rows: P is not needed
      for (int i = 0; i < pages; ++i, ++n) {
        int done = wait(ctl->s_full[b], n);
        // P and O of the page before (the item's first page: of an earlier item, long done)
        auto last_done = [&] {
          if (i > 0) done &= wait(ctl->o_done[b], n - 1);
        };
        if (idle) {
          mbar_arrive(smem_u32(&ctl->s_empty[b]));
          last_done();
          mbar_arrive(smem_u32(&ctl->p_full[b]));
          if (!(ok = all(done))) break;
          continue;
        }
        tmem::fence_after();
        uint32_t s0[32], s1[32];
        tmem::ld_x32(tl, s0);
        tmem::ld_x32(tl + 32, s1);
        tmem::wait_ld();
        tmem::fence_before();
        mbar_arrive(smem_u32(&ctl->s_empty[b]));
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) mx = max3(mx, __uint_as_float(s0[j]), __uint_as_float(s1[j]));
        mx *= scale;
        const bool raise = mx > m_ref + kRaise;  // also from -inf
        bool waited = false;
        if (i == 0) {
          m_ref = mx;
        } else if (__any_sync(0xffffffffu, raise)) {
          last_done();
          waited = true;
          tmem::fence_after();
          const float f = raise ? ex2(m_ref - mx) : 1.f;
          if (raise) m_ref = mx;
          l *= f;
#pragma unroll
          for (int c = 0; c < kHeadDim; c += 32) {
            uint32_t o[32];
            tmem::ld_x32(tl + kColO + c, o);
            tmem::wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem::st_x32(tl + kColO + c, o);
          }
        }
        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t scale2 = pack2(scale, scale), minus_ref = pack2(-ref, -ref), minus_one = pack2(-1.f, -1.f);
        uint64_t l2 = pack2(0.f, 0.f);
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint32_t* s = j < 16 ? s0 + 2 * j : s1 + 2 * (j - 16);
          float pa, pb;
          unpack2(fma2(pack2(__uint_as_float(s[0]), __uint_as_float(s[1])), scale2, minus_ref), pa, pb);
          pa = ex2(pa);
          pb = ex2(pb);
          const uint64_t p = pack2(pa, pb);
          l2 = add2(l2, p);
          hi[j] = pack_bf16(pa, pb);
          unpack2(fma2(pack2(bf16_lo(hi[j]), bf16_hi(hi[j])), minus_one, p), pa, pb);
          lo[j] = pack_bf16(pa, pb);
        }
        float la, lb;
        unpack2(l2, la, lb);
        l += la + lb;
        if (!waited) {
          last_done();
          tmem::fence_after();
        }
        tmem::st_x32(tl + kColP, hi);
        tmem::st_x32(tl + kColP + 32, lo);
        tmem::wait_st();
        tmem::fence_before();
        mbar_arrive(smem_u32(&ctl->p_full[b]));
        if (!(ok = all(done))) break;
      }
      if (!ok) break;
      // ---- the rows' partials
      if (!(ok = all(wait(ctl->o_done[b], n - 1)))) break;
      tmem::fence_after();
      const int m = w.row0(b) + r;
      const bool mine = m < w.rows;
      uint8_t* slot = partials;
      const int h = m % G;
      if (mine) {
        slot = slot_of(m);
        reinterpret_cast<float2*>(slot)[h] = make_float2(l == 0.f ? -INFINITY : m_ref, l);
      }
      float4* dst = reinterpret_cast<float4*>(slot + G * 8) + h * (kHeadDim / 4);
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int c = 0; c < kHeadDim; c += 32) {
        uint32_t o[32];
        tmem::ld_x32(tl + kColO + c, o);
        tmem::wait_ld();
        if (mine)
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            dst[(c + j) / 4] = make_float4(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv,
                                           __uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
      }
      tmem::fence_before();  // O is read before the next item's first MMA writes it
    }
  }
  __syncwarp();
  tmem::fence_before();
  __syncthreads();
  tmem::fence_after();
  if (warp == 0) tmem::dealloc(tm, 512);
}

}  // namespace

int encode_page_map(const KernelParams& kp, void* map) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return int(e);
  if (!fn || found != cudaDriverEntryPointSuccess) return int(cudaErrorNotSupported);
  // the pool as rows of 128 channels: [layer][page][kv-head][K|V][64 tokens]
  const cuuint64_t rows = cuuint64_t(kp.n_layers) * kp.max_pages * kp.n_kv_heads * 2 * kPage;
  const cuuint64_t dims[2] = {kHeadDim, rows}, strides[1] = {kHeadDim * 2};
  const cuuint32_t box[2] = {64, kPage}, step[2] = {1, 1};
  const CUresult r = reinterpret_cast<Encode>(fn)(
      static_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kp.base + kp.lay.bf16_pages, dims, strides, box,
      step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : int(cudaErrorInvalidValue);
}

int launch_shared(const KernelParams& kp, int layer, const void* map, const void* q, uint8_t* partials, int n_sm,
                  void* stream, int* launches) {
  static PerDevice attr;
  const int ready = attr.get([] {
    const int e = int(cudaFuncSetAttribute(shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    return e ? -e : 1;
  });
  if (ready < 0) return -ready;
  const int e = launch_ex(shared_kernel, dim3(n_sm), dim3(kThreads), size_t(kSmemBytes), stream, kp, layer,
                          *static_cast<const CUtensorMap*>(map), static_cast<const uint16_t*>(q), partials);
  if (!e) *launches += 1;
  return e;
}

}  // namespace oscar
