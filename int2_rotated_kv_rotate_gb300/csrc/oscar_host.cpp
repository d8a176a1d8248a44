// Host side of the C ABI (include/oscar.h): configuration checks, the device-block layout,
// the page allocator with reference-counted prefix sharing, request state, append and
// split-K decode planning, uploads of plans and page-table rows, status readback.
//
// Paged KV with prefix caching, BF16 sinks / recent tokens and INT2 history follow the
// online-serving part of the OSCAR technical summary (gist.science), section 2.2-B.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "oscar_internal.h"

using namespace oscar;

constexpr int kUploadSlots = 6;  // pinned upload buffers (two uploads per step: reserve, plan)

namespace {

thread_local std::string g_error;
thread_local int g_launches = 0;

oscar_status fail(oscar_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
oscar_status fail(oscar_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_error = buf;
  return st;
}

#define CUDA_TRY(expr)                                                                        \
  do {                                                                                        \
    cudaError_t e_ = (expr);                                                                  \
    if (e_ != cudaSuccess) return fail(OSCAR_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
// offsets of the items inside a plan block (counts at 0, requests at 256)
size_t append_items_offset(size_t reqs) { return 256 + align256(reqs * sizeof(AppendReq)); }
size_t score_base_offset(size_t reqs) { return 256 + align256(reqs * sizeof(DecodeReq)); }
size_t decode_items_offset(size_t reqs) { return score_base_offset(reqs) + align256(reqs * 8); }
// offset of the items behind the order of a plan's shared runs
size_t shared_items_offset(size_t reqs) { return align256(reqs * 4); }
int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kAppendChunk = 16;     // tokens (or ring slots) per append work item
constexpr int kMaxAppendTokenItems = 65536;
constexpr int kSharedItemPages = 16;  // an item's fixed time in the shared launch, in pages
// A plan uses the shared launch where the reads that it saves take longer than what it adds, in
// bytes read: itself (8 MB), a merge's turns over the shared slots of a head (1 MB each), the
// rows of an item (40 MB for a block of 128), and the private tokens that wait for the SMs it
// holds (2.5 times their bytes, up to 30 MB of them).  Fitted to 634 plans of 6 to 260 MB saved,
// 4 to 64 query heads on 1 to 8 kv-heads, 2 to 128 requests, tails of 1 to 2000 tokens.  On 240
// others: 1.2 % over the better of the two on average, 23 over it by more than 5 % (4.2 % and 59
// with the saved bytes alone, from 32 MB on).
// With / without it, 32 query heads on 8 kv-heads, tails of 40 tokens: 8 requests on 8 pages
// (15 MB saved) 11.2 / 10.5 us, 4 on 32 (25 MB) 12.9 / 12.3, 2 on 128 (34 MB) 21.1 / 17.3, 4 on
// 64 (50 MB) 14.9 / 17.5, 32 on 8 (65 MB) 22.0 / 19.5, 8 on 64 (117 MB) 20.5 / 27.8, 32 on 32
// (260 MB) 25.3 / 54.0; tails of 2000 tokens, 5 on 96 (101 MB) 31.4 / 27.3.
constexpr double kSharedLaunchBytes = 8e6, kSharedSlotBytes = 1e6, kSharedRowBytes = 40e6 / 128;
constexpr double kSharedPrivateBytes = 30e6, kSharedPrivateWeight = 2.5;
constexpr int kSharedMinSaved = 4;  // a run that saves fewer pages is none by itself: its members attend them, or their own runs do
constexpr int kBf16ItemTokens = 128;  // sink+ring tokens per decode work item (at least; one chunk of the CTA)

bool config_ok(const oscar_config* c, std::string* why) {
  auto bad = [&](const char* m) {
    *why = m;
    return false;
  };
  if (!c) return bad("config is NULL");
  if (c->format != OSCAR_FORMAT_INT2 && c->format != OSCAR_FORMAT_BF16 && c->format != OSCAR_FORMAT_INT2_CM)
    return bad("format must be INT2, INT2_CM or BF16");
  if (c->head_dim != kHeadDim) return bad("head_dim must be 128");
  if (c->page != kPage) return bad("page must be 64");
  if (c->n_kv_heads <= 0 || c->n_q_heads <= 0 || c->n_q_heads % c->n_kv_heads) return bad("bad head counts");
  int g = c->n_q_heads / c->n_kv_heads;
  if (g != 4 && g != 8) return bad("H_q / H_kv must be 4 or 8");
  if (c->n_layers <= 0 || c->max_requests <= 0 || c->max_pages <= 0 || c->max_pages_per_request <= 0)
    return bad("layers, requests and pages must be positive");
  if (c->max_pages_per_request > (1 << 20)) return bad("max_pages_per_request too large");
  if (c->format == OSCAR_FORMAT_INT2 || c->format == OSCAR_FORMAT_INT2_CM) {
    if (c->group != 32 && c->group != 128) return bad("group must be 32 or 128");
    if (c->format == OSCAR_FORMAT_INT2_CM && c->group == 32 && g != 4)
      return bad("the INT2_CM format supports group 32 at GQA 4 only");
    if (c->n_sink < 0 || c->n_sink > kPage) return bad("n_sink must be in [0, 64]");
    if (c->window < 0 || c->window > kMaxWindow || c->window % 16) return bad("window must be a multiple of 16 in [0, 1024]");
  }
  return true;
}

DeviceLayout compute_layout(const oscar_config& c) {
  DeviceLayout L;
  std::memset(&L, 0, sizeof L);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const size_t d = kHeadDim, Hkv = c.n_kv_heads, layers = c.n_layers, pages = c.max_pages;
  const size_t reqs = c.max_requests;
  if (c.format == OSCAR_FORMAT_INT2 || c.format == OSCAR_FORMAT_INT2_CM) {
    const size_t ng = d / c.group;
    L.codes_head_stride = 2 * kPage * kRowBytes;
    L.codes_page_stride = Hkv * L.codes_head_stride;
    L.codes_layer_stride = pages * L.codes_page_stride;
    L.codes = take(layers * L.codes_layer_stride);
    L.sz_head_stride = 2 * kPage * ng * 4;
    L.sz_page_stride = Hkv * L.sz_head_stride;
    L.sz_layer_stride = pages * L.sz_page_stride;
    L.sz = take(layers * L.sz_layer_stride);
    L.sink_head_stride = 2 * size_t(c.n_sink) * d * 2;
    L.sink_layer_stride = Hkv * L.sink_head_stride;
    L.sink_slot_stride = layers * L.sink_layer_stride;
    L.sink = take(reqs * L.sink_slot_stride);
    L.ring_head_stride = 2 * size_t(c.window) * d * 2;
    L.ring_layer_stride = Hkv * L.ring_head_stride;
    L.ring_slot_stride = layers * L.ring_layer_stride;
    L.ring = take(reqs * L.ring_slot_stride);
    L.R_K = take(layers * Hkv * d * d * 4);
    L.R_V = take(layers * Hkv * d * d * 4);
    L.R_Vt = take(layers * Hkv * d * d * 4);
    L.clip_K = take(layers * Hkv * 4);
    L.clip_V = take(layers * Hkv * 4);
  } else {
    L.bf16_head_stride = 2 * kPage * d * 2;
    L.bf16_page_stride = Hkv * L.bf16_head_stride;
    L.bf16_layer_stride = pages * L.bf16_page_stride;
    L.bf16_pages = take(layers * L.bf16_layer_stride);
    L.evict_plan = take(256 + reqs * sizeof(EvictReq));
    L.evict_pages = take(reqs * size_t(c.max_pages_per_request) * 4);
  }
  L.page_table = take(reqs * size_t(c.max_pages_per_request) * 4);
  L.status = take(256);
  L.counters = take(reqs * Hkv * 4);
  L.max_append_items = kMaxAppendTokenItems + reqs * (kMaxWindow / kAppendChunk + 1);  // + 1: a block-aligned split
  L.max_decode_items = reqs * Hkv * (2 + kMaxWindow / kBf16ItemTokens) + 16384;
  L.append_plan = take(append_items_offset(reqs) + L.max_append_items * sizeof(AppendItem));
  L.append_counts = L.append_plan;
  L.append_reqs = L.append_plan + 256;
  L.append_items = L.append_plan + append_items_offset(reqs);
  L.decode_plan = take(decode_items_offset(reqs) + L.max_decode_items * sizeof(DecodeItem));
  L.decode_counts = L.decode_plan;
  L.decode_reqs = L.decode_plan + 256;
  L.score_base = L.decode_plan + score_base_offset(reqs);
  L.decode_items = L.decode_plan + decode_items_offset(reqs);
  if (c.format == OSCAR_FORMAT_BF16) {
    L.max_shared_items = 16384;
    L.shared_order = take(shared_items_offset(reqs) + L.max_shared_items * sizeof(SharedItem));
    L.shared_items = L.shared_order + shared_items_offset(reqs);
  }
  L.sched = take(16);
  L.app_done = take(layers * reqs * Hkv * 8);
  L.total = off;
  return L;
}

struct Request {
  bool in_use = false;
  int L = 0, H = 0;
  std::vector<int> pages;
};

}  // namespace

struct oscar_cache {
  oscar_config cfg;
  DeviceLayout lay;
  uint8_t* base = nullptr;
  int n_sm = 148;
  std::vector<Request> reqs;
  std::vector<int> refcount;
  std::vector<int> free_pages;
  // host mirror of the page table, and a ring of pinned upload buffers: every upload copies
  // what it sends into the next buffer first, so the host never rewrites memory that an
  // enqueued copy still reads, and waits only when it runs kUploadSlots uploads ahead
  int32_t* h_page_table = nullptr;
  uint8_t* h_upload = nullptr;  // kUploadSlots x upload_bytes, pinned
  size_t upload_bytes = 0, staging_bytes = 0;
  cudaEvent_t upload_done[kUploadSlots] = {};
  bool upload_pending[kUploadSlots] = {};
  int upload_next = 0;
  uint32_t* h_status = nullptr;
  // pending append
  bool reserved = false;
  std::vector<AppendReq> app_reqs;
  std::vector<int> app_req_items;  // append items of each reservation request
  int app_items = 0, app_rows = 0;
  bool plan_covers_reservation = false;  // the plan lists every slot of the pending reservation
  bool dec_wide = false;                  // INT2: the plan is for 16-warp split-kernel CTAs; BF16: for the deep pipeline
  bool dec_folded = false;                // OSCAR_PLAN_FOLDED_ROTATIONS: q~ in, o~ out
  // pending eviction (BF16 format)
  bool evicting = false;
  std::vector<EvictReq> ev_reqs;
  std::vector<std::vector<int>> ev_pages;  // new pages of each request that gives tokens up
  int ev_max_pages = 0;
  // decode plan
  bool planned = false;
  bool planned_with_reservation = false;  // the plan already counts the reserved tokens
  bool dec_shared = false;  // OSCAR_PLAN_SHARED_PREFIX: the shared launch goes before the decode's
  int dec_shared_items = 0, dec_shared_pages = 0;
  bool map_ready = false;
  alignas(64) unsigned char page_map[128];  // tensor map of the BF16 page pool
  int dec_n_req = 0, dec_items = 0, dec_bf16_items = 0, dec_max_pages = 0;
  long long dec_tokens = 0;  // of all kv-heads
  DecodeWorkspace ws{};
  int device = 0;              // the device current at creation (the device of `base`)
  uint32_t counter_polls = 0;  // oscar_set_wait_limit (0 = kDefaultCounterPolls)
  uint32_t inject = 0;         // oscar_inject_fault: host-side faults armed for the next plan
};

namespace {

// One upload buffer: page-table rows (max_requests rows), then the image of a plan block.
struct Upload {
  int32_t* rows;
  uint8_t* staging;
  int slot;
};

KernelParams kernel_params(const oscar_cache* c) {
  KernelParams kp;
  kp.base = c->base;
  kp.n_q_heads = c->cfg.n_q_heads;
  kp.n_kv_heads = c->cfg.n_kv_heads;
  kp.gqa = c->cfg.n_q_heads / c->cfg.n_kv_heads;
  kp.group = c->cfg.group;
  kp.n_sink = c->cfg.n_sink;
  kp.window = c->cfg.window;
  kp.n_layers = c->cfg.n_layers;
  kp.max_requests = c->cfg.max_requests;
  kp.max_pages = c->cfg.max_pages;
  kp.max_pages_per_request = c->cfg.max_pages_per_request;
  kp.counter_polls = c->counter_polls ? c->counter_polls : kDefaultCounterPolls;
  kp.v_cm = c->cfg.format == OSCAR_FORMAT_INT2_CM;
  kp.weights_stride = oscar_weights_stride(c);
  kp.folded = c->dec_folded;
  kp.lay = c->lay;
  return kp;
}

// The next upload buffer of the ring, once the copies that last read it have run.
oscar_status begin_upload(oscar_cache* c, Upload* u) {
  const int i = c->upload_next;
  c->upload_next = (i + 1) % kUploadSlots;
  if (c->upload_pending[i]) {
    CUDA_TRY(cudaEventSynchronize(c->upload_done[i]));
    c->upload_pending[i] = false;
  }
  uint8_t* b = c->h_upload + size_t(i) * c->upload_bytes;
  u->rows = reinterpret_cast<int32_t*>(b);
  u->staging = b + align256(size_t(c->cfg.max_requests) * c->cfg.max_pages_per_request * 4);
  u->slot = i;
  return OSCAR_OK;
}

// Record that the copies enqueued on s so far read upload buffer u.
oscar_status end_upload(oscar_cache* c, const Upload& u, cudaStream_t s) {
  CUDA_TRY(cudaEventRecord(c->upload_done[u.slot], s));
  c->upload_pending[u.slot] = true;
  return OSCAR_OK;
}

// Every upload buffer is free again (teardown).
void drain_uploads(oscar_cache* c) {
  for (int i = 0; i < kUploadSlots; ++i)
    if (c->upload_pending[i]) {
      cudaEventSynchronize(c->upload_done[i]);
      c->upload_pending[i] = false;
    }
}

// Page-table rows of `slots` from the host mirror, through upload buffer u.
oscar_status upload_rows(oscar_cache* c, const Upload& u, const std::vector<int>& slots, cudaStream_t s) {
  const size_t n = size_t(c->cfg.max_pages_per_request);
  for (size_t k = 0; k < slots.size(); ++k) {
    int32_t* dst = u.rows + k * n;
    std::memcpy(dst, c->h_page_table + size_t(slots[k]) * n, n * 4);
    CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.page_table + size_t(slots[k]) * n * 4, dst, n * 4,
                             cudaMemcpyHostToDevice, s));
  }
  return OSCAR_OK;
}

bool is_int2(const oscar_cache* c) {
  return c->cfg.format == OSCAR_FORMAT_INT2 || c->cfg.format == OSCAR_FORMAT_INT2_CM;
}
// Channel-major value pages, decoded on the tcgen05 tensor cores; never a fused launch.
bool is_cm(const oscar_cache* c) { return c->cfg.format == OSCAR_FORMAT_INT2_CM; }

// Pages a request needs to hold its stored tokens: the INT2 format pages positions < H
// (sinks and recent tokens live elsewhere), the BF16 format pages all L positions.
int pages_needed(const oscar_cache* c, int L, int H) {
  if (is_int2(c)) return H > c->cfg.n_sink ? ceil_div(H, kPage) : 0;
  return ceil_div(L, kPage);
}

oscar_status check_slot(const oscar_cache* c, int slot) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (slot < 0 || slot >= c->cfg.max_requests) return fail(OSCAR_ERR_INVALID_ARG, "slot %d out of range", slot);
  if (!c->reqs[slot].in_use) return fail(OSCAR_ERR_INVALID_ARG, "slot %d is not allocated", slot);
  return OSCAR_OK;
}

// The calls that look at device memory through the current device.
oscar_status check_device(const oscar_cache* c) {
  int dev = -1;
  CUDA_TRY(cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(OSCAR_ERR_INVALID_ARG, "current device %d is not the cache's device %d", dev, c->device);
  return OSCAR_OK;
}

// The runs of pages that several requests of a plan map, as work items of the shared launch.
struct SharedRuns {
  std::vector<int> order;          // plan indices; the members of every run are neighbours
  std::vector<int> first_private;  // per plan index: pages before it are in shared runs
  std::vector<int> n_segs;         // per plan index: partial slots per head of its shared runs
  std::vector<SharedItem> items;
  int pages = 0;                   // pages attended once for several requests
};

SharedRuns find_shared_runs(const oscar_cache* c, const int* slots, const std::vector<int>& Ls, bool always) {
  SharedRuns out;
  const int n = int(Ls.size()), Hkv = c->cfg.n_kv_heads, G = c->cfg.n_q_heads / Hkv;
  out.order.resize(n);
  for (int i = 0; i < n; ++i) out.order[i] = i;
  out.first_private.assign(n, 0);
  out.n_segs.assign(n, 0);
  // page p of plan index i, -1 past its whole pages (only whole pages are shared)
  auto page = [&](int i, int p) {
    const std::vector<int>& v = c->reqs[slots[i]].pages;
    return p < Ls[i] / kPage && p < int(v.size()) ? v[p] : -1;
  };
  // Runs form a forest: the members of one that part ways in ever smaller sets.
  struct Run {
    int lo, hi, begin, end, parent;
  };
  struct Group {
    int lo, hi, begin, parent;
  };
  std::vector<Run> runs;
  std::vector<Group> todo{{0, n, 0, -1}};
  while (!todo.empty()) {
    const Group g = todo.back();
    todo.pop_back();
    if (g.hi - g.lo < 2) continue;
    int end = g.begin, parent = g.parent, begin = g.begin;
    for (int first; (first = page(out.order[g.lo], end)) >= 0; ++end) {
      bool same = true;
      for (int k = g.lo + 1; same && k < g.hi; ++k) same = page(out.order[k], end) == first;
      if (!same) break;
    }
    if (end > g.begin && (always || (end - g.begin) * (long long)(g.hi - g.lo - 1) >= kSharedMinSaved)) {
      runs.push_back({g.lo, g.hi, g.begin, end, g.parent});
      parent = int(runs.size()) - 1;
      begin = end;
      for (int k = g.lo; k < g.hi; ++k) out.first_private[out.order[k]] = end;
    }
    // (a run too short to pay by itself goes with those of its members that share on)
    std::stable_sort(out.order.begin() + g.lo, out.order.begin() + g.hi,
                     [&](int a, int b) { return page(a, end) < page(b, end); });
    for (int lo = g.lo; lo < g.hi;) {
      const int p = page(out.order[lo], end);
      int hi = lo + 1;
      while (hi < g.hi && page(out.order[hi], end) == p) ++hi;
      if (p >= 0 && hi - lo > 1) todo.push_back({lo, hi, begin, parent});
      lo = hi;
    }
  }
  // Pages of an item: the CTAs, one an SM, take the items in turn, so the launch lasts as
  // long as its rounds of items, each about kSharedItemPages pages' time longer than its
  // pages (the queries, the pipeline's fill, the partials); and every partial slot of a head
  // is merged, an eighth of a page's time each.  The row blocks of a run's pages are items of
  // their own.
  const int per_item = kSharedRows / G;  // members of an item at most
  long long best = -1, best_items = 0, best_slots = 0;
  int chunk = 0, longest = 0;
  for (const Run& r : runs) longest = std::max(longest, r.end - r.begin);
  for (int parts = 1; parts <= std::min(longest, 64); ++parts) {
    const int ch = ceil_div(longest, parts);
    long long items = 0, n_slots = 0;
    for (const Run& r : runs) {
      const long long segs = (long long)Hkv * ceil_div(r.end - r.begin, ch);
      items += segs * ceil_div(r.hi - r.lo, per_item);
      n_slots += segs * (r.hi - r.lo) * ((r.hi - r.lo) * G <= kSharedRows / 2 ? 2 : 1);
    }
    // (the other half of the partial slots is the private items')
    if (items > (long long)c->lay.max_shared_items || n_slots > (long long)c->lay.max_decode_items / 2) continue;
    const long long cost = 8 * ((items + c->n_sm - 1) / c->n_sm) * (ch + kSharedItemPages) + 2 * parts;
    if (best < 0 || cost < best) {
      best = cost;
      best_items = items;
      best_slots = n_slots;
      chunk = ch;
    }
  }
  bool pays = chunk > 0;  // else nothing shared, or no room for the runs' partials
  if (pays && !always) {
    long long saved = 0, rows = 0, sharers = 0, tokens = 0;  // pages; query rows of all items; requests; private tokens
    for (const Run& r : runs) {
      saved += (long long)(r.end - r.begin) * (r.hi - r.lo - 1);
      rows += (long long)Hkv * ceil_div(r.end - r.begin, chunk) * (r.hi - r.lo) * G;
    }
    for (int i = 0; i < n; ++i) {
      sharers += out.first_private[i] > 0;
      tokens += Ls[i] - kPage * out.first_private[i];
    }
    const double token_bytes = double(Hkv) * (2 * kHeadDim * 2);
    pays = double(saved) * kPage * token_bytes >=
           kSharedLaunchBytes + kSharedSlotBytes * double(best_slots) / double(Hkv * sharers) +
               kSharedRowBytes * std::min(double(rows) / double(best_items), kSharedRows / 2.0) +
               kSharedPrivateWeight * std::min(double(tokens) * token_bytes, kSharedPrivateBytes);
  }
  if (!pays) {
    out.first_private.assign(n, 0);
    return out;
  }
  std::vector<int> seg_end(runs.size());
  for (size_t k = 0; k < runs.size(); ++k) {  // parents come before their children
    const Run& r = runs[k];
    const int segs = ceil_div(r.end - r.begin, chunk);
    const int split = (r.hi - r.lo) * G <= kSharedRows / 2;  // two slots a segment
    const int seg0 = r.parent < 0 ? 0 : seg_end[r.parent];
    seg_end[k] = seg0 + segs * (1 + split);
    out.pages += r.end - r.begin;
    for (int m = r.lo; m < r.hi; ++m) out.n_segs[out.order[m]] = seg_end[k];
    for (int s = 0; s < segs; ++s)
      for (int h = 0; h < Hkv; ++h)
        for (int lo = r.lo; lo < r.hi; lo += per_item)
          out.items.push_back({lo, std::min(r.hi, lo + per_item), r.begin + s * chunk,
                               std::min(r.end, r.begin + (s + 1) * chunk), h, seg0 + s * (1 + split), split});
  }
  return out;
}

// Workspace of a decode with weights over `tokens` tokens of all kv-heads.  Only the total
// depends on the plan: a captured launch keeps its offsets.
WeightsWorkspace weights_workspace(const oscar_cache* c, size_t tokens) {
  const size_t Hq = c->cfg.n_q_heads, G = Hq / c->cfg.n_kv_heads;
  WeightsWorkspace w;
  w.ml = 0;
  w.partials = align256(size_t(c->cfg.max_requests) * Hq * 8);
  w.scores = w.partials + align256(c->lay.max_decode_items * G * (8 + 4 * kHeadDim));
  w.total = w.scores + tokens * G * 4;
  return w;
}

}  // namespace

extern "C" {

const char* oscar_last_error(void) { return g_error.c_str(); }
int oscar_last_launch_count(void) { return g_launches; }

size_t oscar_cache_device_bytes(const oscar_config* cfg) {
  std::string why;
  if (!config_ok(cfg, &why)) {
    g_error = why;
    return 0;
  }
  return compute_layout(*cfg).total;
}

oscar_status oscar_cache_create(const oscar_config* cfg, void* device_mem, size_t bytes, oscar_cache** out) {
  std::string why;
  if (!out) return fail(OSCAR_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!config_ok(cfg, &why)) return fail(OSCAR_ERR_INVALID_ARG, "%s", why.c_str());
  if (!device_mem) return fail(OSCAR_ERR_INVALID_ARG, "device_mem is NULL");
  if (reinterpret_cast<uintptr_t>(device_mem) % 256) return fail(OSCAR_ERR_INVALID_ARG, "device_mem must be 256-byte aligned");
  DeviceLayout lay = compute_layout(*cfg);
  if (bytes < lay.total) return fail(OSCAR_ERR_INVALID_ARG, "device block of %zu bytes < %zu needed", bytes, lay.total);
  oscar_cache* c = new (std::nothrow) oscar_cache();
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "host allocation failed");
  c->cfg = *cfg;
  c->lay = lay;
  c->base = static_cast<uint8_t*>(device_mem);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  c->device = dev;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->n_sm, cudaDevAttrMultiProcessorCount, dev);
  c->reqs.resize(cfg->max_requests);
  c->refcount.assign(cfg->max_pages, 0);
  c->free_pages.reserve(cfg->max_pages);
  for (int p = cfg->max_pages - 1; p >= 0; --p) c->free_pages.push_back(p);
  const size_t pt_bytes = size_t(cfg->max_requests) * cfg->max_pages_per_request * 4;
  // a plan block's image (the larger of the two)
  c->staging_bytes = std::max(append_items_offset(cfg->max_requests) + lay.max_append_items * sizeof(AppendItem),
                              decode_items_offset(cfg->max_requests) + lay.max_decode_items * sizeof(DecodeItem));
  if (cfg->format == OSCAR_FORMAT_BF16)  // a plan's shared runs go up behind its items
    c->staging_bytes += 256 + shared_items_offset(cfg->max_requests) + lay.max_shared_items * sizeof(SharedItem);
  c->upload_bytes = align256(pt_bytes) + align256(c->staging_bytes);
  if (e == cudaSuccess) e = cudaMallocHost(reinterpret_cast<void**>(&c->h_page_table), pt_bytes);
  if (e == cudaSuccess) e = cudaMallocHost(reinterpret_cast<void**>(&c->h_upload), kUploadSlots * c->upload_bytes);
  if (e == cudaSuccess) e = cudaMallocHost(reinterpret_cast<void**>(&c->h_status), 256);
  if (e == cudaSuccess) e = cudaMemset(c->base + lay.append_counts, 0, 16);
  if (e == cudaSuccess) e = cudaMemset(c->base + lay.decode_counts, 0, 16);
  for (int i = 0; i < kUploadSlots && e == cudaSuccess; ++i)
    e = cudaEventCreateWithFlags(&c->upload_done[i], cudaEventDisableTiming);
  if (e == cudaSuccess) {
    std::memset(c->h_page_table, 0xff, pt_bytes);  // -1 = unmapped
    e = cudaMemcpy(c->base + lay.page_table, c->h_page_table, pt_bytes, cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) e = cudaMemset(c->base + lay.status, 0, 256);
  if (e == cudaSuccess) e = cudaMemset(c->base + lay.counters, 0, size_t(cfg->max_requests) * cfg->n_kv_heads * 4);
  if (e == cudaSuccess) e = cudaMemset(c->base + lay.sched, 0, 16);
  // scale/zero words of rows no append has written yet (sink positions, the tail of a
  // page) are read with p = 0 by the decode: they must be finite, so the pool starts at 0
  if (e == cudaSuccess && is_int2(c)) e = cudaMemset(c->base + lay.sz, 0, size_t(cfg->n_layers) * lay.sz_layer_stride);
  if (e == cudaSuccess)
    e = cudaMemset(c->base + lay.app_done, 0, size_t(cfg->n_layers) * cfg->max_requests * cfg->n_kv_heads * 8);
  if (e == cudaSuccess && is_int2(c)) {
    // layer params start as zeros until oscar_set_layer_params
    e = cudaMemset(c->base + lay.R_K, 0, lay.clip_K - lay.R_K);
  }
  if (e != cudaSuccess) {
    fail(OSCAR_ERR_CUDA, "cache_create: %s", cudaGetErrorString(e));
    oscar_cache_destroy(c);
    return OSCAR_ERR_CUDA;
  }
  *out = c;
  return OSCAR_OK;
}

void oscar_cache_destroy(oscar_cache* c) {
  if (!c) return;
  drain_uploads(c);
  for (int i = 0; i < kUploadSlots; ++i)
    if (c->upload_done[i]) cudaEventDestroy(c->upload_done[i]);
  if (c->h_page_table) cudaFreeHost(c->h_page_table);
  if (c->h_upload) cudaFreeHost(c->h_upload);
  if (c->h_status) cudaFreeHost(c->h_status);
  delete c;
}

oscar_status oscar_cache_layout(const oscar_cache* c, oscar_layout* out) {
  if (!c || !out) return fail(OSCAR_ERR_INVALID_ARG, "NULL argument");
  const DeviceLayout& L = c->lay;
  out->codes = L.codes;
  out->sz = L.sz;
  out->sink = L.sink;
  out->ring = L.ring;
  out->bf16_pages = L.bf16_pages;
  out->codes_page_bytes = L.codes_head_stride;
  out->sz_page_bytes = L.sz_head_stride;
  out->bf16_page_bytes = L.bf16_head_stride;
  out->sink_bytes_per_head = L.sink_head_stride;
  out->ring_bytes_per_head = L.ring_head_stride;
  out->page_table = L.page_table;
  out->total = L.total;
  return OSCAR_OK;
}

oscar_status oscar_set_layer_params(oscar_cache* c, int layer, const float* R_K, const float* R_V, const float* clip_K,
                                    const float* clip_V, void* stream) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!is_int2(c)) return fail(OSCAR_ERR_STATE, "layer params apply to the INT2 format only");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (!R_K || !R_V || !clip_K || !clip_V) return fail(OSCAR_ERR_INVALID_ARG, "NULL parameter array");
  const int H = c->cfg.n_kv_heads, d = kHeadDim;
  for (int h = 0; h < H; ++h) {
    if (!(clip_K[h] > 0.f) || !(clip_V[h] > 0.f)) return fail(OSCAR_ERR_INVALID_ARG, "clip thresholds must be > 0");
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t mat = size_t(d) * d;
  std::vector<float> Vt(size_t(H) * mat);
  for (int h = 0; h < H; ++h)
    for (int i = 0; i < d; ++i)
      for (int j = 0; j < d; ++j) Vt[h * mat + size_t(j) * d + i] = R_V[h * mat + size_t(i) * d + j];
  const size_t lmat = size_t(layer) * H * mat * 4;
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.R_K + lmat, R_K, H * mat * 4, cudaMemcpyHostToDevice, s));
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.R_V + lmat, R_V, H * mat * 4, cudaMemcpyHostToDevice, s));
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.R_Vt + lmat, Vt.data(), H * mat * 4, cudaMemcpyHostToDevice, s));
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.clip_K + size_t(layer) * H * 4, clip_K, H * 4, cudaMemcpyHostToDevice, s));
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.clip_V + size_t(layer) * H * 4, clip_V, H * 4, cudaMemcpyHostToDevice, s));
  CUDA_TRY(cudaStreamSynchronize(s));  // Vt is a temporary
  return OSCAR_OK;
}

oscar_status oscar_request_alloc(oscar_cache* c, int* slot) {
  if (!c || !slot) return fail(OSCAR_ERR_INVALID_ARG, "NULL argument");
  for (int i = 0; i < c->cfg.max_requests; ++i) {
    if (!c->reqs[i].in_use) {
      c->reqs[i] = Request();
      c->reqs[i].in_use = true;
      c->reqs[i].H = is_int2(c) ? c->cfg.n_sink : 0;
      *slot = i;
      return OSCAR_OK;
    }
  }
  return fail(OSCAR_ERR_OUT_OF_PAGES, "no free request slot");
}

oscar_status oscar_request_free(oscar_cache* c, int slot) {
  oscar_status st = check_slot(c, slot);
  if (st) return st;
  if (c->evicting) return fail(OSCAR_ERR_STATE, "an eviction is pending");
  if (c->reserved)
    for (const AppendReq& r : c->app_reqs)
      if (r.slot == slot) return fail(OSCAR_ERR_STATE, "slot %d has a pending reservation", slot);
  Request& r = c->reqs[slot];
  for (int p : r.pages)
    if (--c->refcount[p] == 0) c->free_pages.push_back(p);
  // the device row keeps stale ids; it is rewritten before the slot is used again
  std::fill(c->h_page_table + size_t(slot) * c->cfg.max_pages_per_request,
            c->h_page_table + size_t(slot + 1) * c->cfg.max_pages_per_request, -1);
  r = Request();
  c->planned = false;
  return OSCAR_OK;
}

oscar_status oscar_cache_stats(const oscar_cache* c, int* free_pages, int* free_slots) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (free_pages) *free_pages = int(c->free_pages.size());
  if (free_slots) {
    int n = 0;
    for (const Request& r : c->reqs) n += !r.in_use;
    *free_slots = n;
  }
  return OSCAR_OK;
}

oscar_status oscar_request_info(const oscar_cache* c, int slot, int* length, int* history_end, int* n_pages) {
  oscar_status st = check_slot(c, slot);
  if (st) return st;
  const Request& r = c->reqs[slot];
  if (length) *length = r.L;
  if (history_end) *history_end = r.H;
  if (n_pages) *n_pages = int(r.pages.size());
  return OSCAR_OK;
}

oscar_status oscar_request_pages(const oscar_cache* c, int slot, int* pages, int n) {
  oscar_status st = check_slot(c, slot);
  if (st) return st;
  const Request& r = c->reqs[slot];
  if (!pages || n < 0 || n > int(r.pages.size())) return fail(OSCAR_ERR_INVALID_ARG, "bad page buffer");
  std::copy(r.pages.begin(), r.pages.begin() + n, pages);
  return OSCAR_OK;
}

oscar_status oscar_request_share_prefix(oscar_cache* c, int dst, int src, int n_tokens, void* stream) {
  oscar_status st = check_slot(c, dst);
  if (st) return st;
  st = check_slot(c, src);
  if (st) return st;
  if (dst == src) return fail(OSCAR_ERR_INVALID_ARG, "dst == src");
  if (c->reserved) return fail(OSCAR_ERR_STATE, "a reservation is pending");
  if (c->evicting) return fail(OSCAR_ERR_STATE, "an eviction is pending");
  Request& d = c->reqs[dst];
  const Request& s = c->reqs[src];
  if (d.L != 0 || !d.pages.empty()) return fail(OSCAR_ERR_INVALID_ARG, "dst must be empty");
  if (n_tokens <= 0 || n_tokens % kPage) return fail(OSCAR_ERR_INVALID_ARG, "n_tokens must be a positive multiple of 64");
  const int limit = is_int2(c) ? s.H : s.L / kPage * kPage;
  if (n_tokens > limit)
    return fail(OSCAR_ERR_INVALID_ARG, "n_tokens %d exceeds the shareable prefix %d of src", n_tokens, limit);
  if (n_tokens / kPage > c->cfg.max_pages_per_request) return fail(OSCAR_ERR_INVALID_ARG, "prefix too long");
  Upload u;
  st = begin_upload(c, &u);
  if (st) return st;
  cudaStream_t strm = static_cast<cudaStream_t>(stream);
  const int n = n_tokens / kPage;
  d.pages.assign(s.pages.begin(), s.pages.begin() + n);
  for (int p : d.pages) ++c->refcount[p];
  int32_t* row = c->h_page_table + size_t(dst) * c->cfg.max_pages_per_request;
  std::fill(row, row + c->cfg.max_pages_per_request, -1);
  std::copy(d.pages.begin(), d.pages.end(), row);
  d.L = n_tokens;
  d.H = is_int2(c) ? n_tokens : n_tokens;
  st = upload_rows(c, u, {dst}, strm);
  if (st) return st;
  if (is_int2(c) && c->lay.sink_slot_stride > 0) {
    CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.sink + size_t(dst) * c->lay.sink_slot_stride,
                             c->base + c->lay.sink + size_t(src) * c->lay.sink_slot_stride, c->lay.sink_slot_stride,
                             cudaMemcpyDeviceToDevice, strm));
  }
  st = end_upload(c, u, strm);
  if (st) return st;
  c->planned = false;
  return OSCAR_OK;
}

oscar_status oscar_reserve(oscar_cache* c, const int* slots, const int* n_new, int n_req, void* stream) {
  if (!c || !slots || !n_new || n_req <= 0 || n_req > c->cfg.max_requests)
    return fail(OSCAR_ERR_INVALID_ARG, "bad reserve arguments");
  if (c->reserved) return fail(OSCAR_ERR_STATE, "previous reservation not committed");
  if (c->evicting) return fail(OSCAR_ERR_STATE, "an eviction is pending");
  std::vector<char> seen(c->cfg.max_requests, 0);
  long long rows = 0;
  int new_pages = 0;
  const int S = is_int2(c) ? c->cfg.n_sink : 0, W = c->cfg.window;
  std::vector<AppendReq> reqs(n_req);
  for (int i = 0; i < n_req; ++i) {
    oscar_status st = check_slot(c, slots[i]);
    if (st) return st;
    if (seen[slots[i]]) return fail(OSCAR_ERR_INVALID_ARG, "slot %d listed twice", slots[i]);
    seen[slots[i]] = 1;
    if (n_new[i] < 0) return fail(OSCAR_ERR_INVALID_ARG, "negative n_new");
    const Request& r = c->reqs[slots[i]];
    AppendReq& a = reqs[i];
    a.slot = slots[i];
    a.L0 = r.L;
    a.H0 = r.H;
    long long L1 = (long long)r.L + n_new[i];
    if (L1 > (long long)kPage * c->cfg.max_pages_per_request)
      return fail(OSCAR_ERR_INVALID_ARG, "request %d would exceed its page-table row", slots[i]);
    a.L1 = int(L1);
    a.H1 = is_int2(c) ? std::max(r.H, a.L1 - W) : a.L1;
    a.x_offset = int(rows);
    rows += n_new[i];
    new_pages += std::max(0, pages_needed(c, a.L1, a.H1) - int(r.pages.size()));
  }
  if (rows > (1 << 30)) return fail(OSCAR_ERR_INVALID_ARG, "too many rows");
  if (new_pages > int(c->free_pages.size()))
    return fail(OSCAR_ERR_OUT_OF_PAGES, "need %d pages, %zu free", new_pages, c->free_pages.size());
  // work items
  std::vector<AppendItem> items;
  for (int i = 0; i < n_req; ++i) {
    const AppendReq& a = reqs[i];
    if (is_int2(c) && W > 0) {
      std::vector<char> touched(W, 0);
      for (int p = a.H0; p < std::min(a.L0, a.H1); ++p) touched[p % W] = 1;   // evicted
      for (int p = std::max(a.L0, a.H1); p < a.L1; ++p) touched[p % W] = 1;  // new ring tokens
      for (int s0 = 0; s0 < W; s0 += kAppendChunk) {
        bool any = false;
        for (int s = s0; s < s0 + kAppendChunk; ++s) any |= touched[s] != 0;
        if (any) items.push_back({i, 0, s0, kAppendChunk});
      }
    }
    const int d0 = a.L0, d1 = is_int2(c) ? std::min(a.L1, a.H1) : a.L1;
    // channel-major value pages: an item's positions stay inside one 16-position block,
    // whose code words (one per channel) the append kernel writes whole
    for (int p = d0; p < d1;) {
      const int e = is_cm(c) ? std::min(d1, (p / kAppendChunk + 1) * kAppendChunk) : std::min(d1, p + kAppendChunk);
      items.push_back({i, 1, p, e - p});
      p = e;
    }
  }
  if (items.size() > c->lay.max_append_items)
    return fail(OSCAR_ERR_INVALID_ARG, "append of %lld tokens is too large for one reservation; split it", rows);
  Upload u;
  oscar_status st = begin_upload(c, &u);
  if (st) return st;
  // allocate pages and update the host mirror
  std::vector<int> changed;
  for (const AppendReq& a : reqs) {
    Request& r = c->reqs[a.slot];
    int need = pages_needed(c, a.L1, a.H1);
    if (need > int(r.pages.size())) {
      int32_t* row = c->h_page_table + size_t(a.slot) * c->cfg.max_pages_per_request;
      while (int(r.pages.size()) < need) {
        int p = c->free_pages.back();
        c->free_pages.pop_back();
        c->refcount[p] = 1;
        row[r.pages.size()] = p;
        r.pages.push_back(p);
      }
      changed.push_back(a.slot);
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = upload_rows(c, u, changed, s);
  if (st) return st;
  // the append plan block, one copy
  const size_t items_off = append_items_offset(c->cfg.max_requests);
  int32_t* counts = reinterpret_cast<int32_t*>(u.staging);
  counts[0] = int(items.size());
  counts[1] = counts[2] = counts[3] = 0;
  std::memcpy(u.staging + 256, reqs.data(), reqs.size() * sizeof(AppendReq));
  std::memcpy(u.staging + items_off, items.data(), items.size() * sizeof(AppendItem));
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.append_plan, u.staging, items_off + items.size() * sizeof(AppendItem),
                           cudaMemcpyHostToDevice, s));
  st = end_upload(c, u, s);
  if (st) return st;
  c->app_reqs = reqs;
  c->app_req_items.assign(reqs.size(), 0);
  for (const AppendItem& it : items) ++c->app_req_items[it.req];
  c->app_items = int(items.size());
  c->app_rows = int(rows);
  c->reserved = true;
  c->planned = false;  // lengths change: plan again (a plan made now counts the new tokens)
  c->planned_with_reservation = false;
  return OSCAR_OK;
}

oscar_status oscar_commit_append(oscar_cache* c) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->reserved) return fail(OSCAR_ERR_STATE, "no reservation to commit");
  for (const AppendReq& a : c->app_reqs) {
    c->reqs[a.slot].L = a.L1;
    c->reqs[a.slot].H = a.H1;
  }
  c->reserved = false;
  if (!c->planned_with_reservation) c->planned = false;
  c->planned_with_reservation = false;
  c->plan_covers_reservation = false;
  return OSCAR_OK;
}

oscar_status oscar_quantize_append(oscar_cache* c, int layer, const void* k_new, const void* v_new, void* stream) {
  g_launches = 0;
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_quantize_append needs the INT2 format");
  if (!c->reserved) return fail(OSCAR_ERR_STATE, "no reservation");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (c->app_rows > 0 && (!k_new || !v_new)) return fail(OSCAR_ERR_INVALID_ARG, "NULL token arrays");
  if (c->app_items == 0) return OSCAR_OK;
  int e = launch_append(kernel_params(c), layer, k_new, v_new, c->app_items, c->n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "append launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_bf16_append(oscar_cache* c, int layer, const void* k_new, const void* v_new, void* stream) {
  g_launches = 0;
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_bf16_append needs the BF16 format");
  if (!c->reserved) return fail(OSCAR_ERR_STATE, "no reservation");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (c->app_rows > 0 && (!k_new || !v_new)) return fail(OSCAR_ERR_INVALID_ARG, "NULL token arrays");
  if (c->app_items == 0) return OSCAR_OK;
  int e = launch_bf16_append(kernel_params(c), layer, k_new, v_new, std::min(c->app_items, 4 * c->n_sm), stream,
                             &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "bf16 append launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_plan_decode(oscar_cache* c, const int* slots, int n_req, int max_split_pages, void* stream) {
  return oscar_plan_decode_ex(c, slots, n_req, max_split_pages, 0u, stream);
}

oscar_status oscar_plan_decode_ex(oscar_cache* c, const int* slots, int n_req, int max_split_pages, uint32_t flags,
                                  void* stream) try {
  if (!c || !slots || n_req <= 0 || n_req > c->cfg.max_requests)
    return fail(OSCAR_ERR_INVALID_ARG, "bad plan arguments");
  if (flags & ~(OSCAR_PLAN_NARROW | OSCAR_PLAN_FOLDED_ROTATIONS | OSCAR_PLAN_SHARED_PREFIX |
                OSCAR_PLAN_SHARED_ALWAYS))
    return fail(OSCAR_ERR_INVALID_ARG, "unknown plan flags %#x", flags);
  if ((flags & OSCAR_PLAN_FOLDED_ROTATIONS) && !is_int2(c))
    return fail(OSCAR_ERR_INVALID_ARG, "OSCAR_PLAN_FOLDED_ROTATIONS applies to the INT2 formats");
  const bool shared = (flags & OSCAR_PLAN_SHARED_PREFIX) != 0;
  if ((flags & OSCAR_PLAN_SHARED_ALWAYS) && !shared)
    return fail(OSCAR_ERR_INVALID_ARG, "OSCAR_PLAN_SHARED_ALWAYS goes with OSCAR_PLAN_SHARED_PREFIX");
  if (shared && is_int2(c))
    return fail(OSCAR_ERR_INVALID_ARG, "OSCAR_PLAN_SHARED_PREFIX applies to the BF16 format");
  if (max_split_pages < 0) return fail(OSCAR_ERR_INVALID_ARG, "max_split_pages < 0");
  std::vector<char> seen(c->cfg.max_requests, 0);
  const int Hkv = c->cfg.n_kv_heads, S = is_int2(c) ? c->cfg.n_sink : 0;
  // lengths the decode will see: a pending reservation's tokens count (append before decode)
  std::vector<int> Ls(n_req), Hs(n_req), Hpre(n_req), Lpre(n_req), app_items(n_req, 0), app_expect(n_req, 0);
  int n_reserved_planned = 0;
  long long total_pages = 0;
  for (int i = 0; i < n_req; ++i) {
    oscar_status st = check_slot(c, slots[i]);
    if (st) return st;
    if (seen[slots[i]]) return fail(OSCAR_ERR_INVALID_ARG, "slot %d listed twice", slots[i]);
    seen[slots[i]] = 1;
    const Request& r = c->reqs[slots[i]];
    Ls[i] = r.L;
    Hs[i] = r.H;
    Hpre[i] = r.H;
    Lpre[i] = r.L;
    if (c->reserved)
      for (size_t k = 0; k < c->app_reqs.size(); ++k) {
        const AppendReq& a = c->app_reqs[k];
        if (a.slot == slots[i]) {
          Ls[i] = a.L1;
          Hs[i] = a.H1;
          Hpre[i] = std::min(r.H, a.H0);
          Lpre[i] = std::min(r.L, a.L0);
          app_items[i] = c->app_req_items[k];
          ++n_reserved_planned;
        }
      }
  }
  SharedRuns runs;
  if (shared) {
    if (!c->map_ready) {
      const unsigned long long rows = 2ull * kPage * c->cfg.n_layers * c->cfg.max_pages * Hkv;
      if (rows > 0x7fffffffull)
        return fail(OSCAR_ERR_UNSUPPORTED, "OSCAR_PLAN_SHARED_PREFIX: a pool of %llu rows is too large", rows);
      const int e = encode_page_map(kernel_params(c), c->page_map);
      if (e) return fail(OSCAR_ERR_CUDA, "tensor map of the page pool: %s", cudaGetErrorString(cudaError_t(e)));
      c->map_ready = true;
    }
    runs = find_shared_runs(c, slots, Ls, (flags & OSCAR_PLAN_SHARED_ALWAYS) != 0);
  } else {
    runs.first_private.assign(n_req, 0);
    runs.n_segs.assign(n_req, 0);
  }
  for (int i = 0; i < n_req; ++i) total_pages += (long long)Hkv * (pages_needed(c, Ls[i], Hs[i]) - runs.first_private[i]);
  // Work items: per (request, kv-head) the BF16 sink+ring items and page ranges of
  // `chunk` pages.  Automatic chunk, from the bytes each resident CTA would stream:
  //  - small steps (latency-bound): the smallest chunk that lets one wave of resident CTAs
  //    hold every item (a second, partial wave would add a whole item's latency);
  //  - large steps: about kWaves items per resident CTA (at least kItemBytes each), taken
  //    dynamically by the CTAs, largest first, so the ragged tail stays short while the
  //    per-item costs (pipeline fill, partial store and merge) stay small.
  // Per request: INT2 pages np, BF16 sink+ring tokens n_bf, and the split points of the
  // items that do not (before) and may (after) read rows of this step's append: bf_new in
  // the BF16 list, pg_new in the pages.
  // Pages before p0_of, attended by the shared launch, are not counted.
  const std::vector<int>& p0_of = runs.first_private;
  std::vector<int> np_of(n_req), nbf_of(n_req), bfnew_of(n_req), pgnew_of(n_req);
  int max_np = 1;
  const int ng = kHeadDim / (is_int2(c) ? c->cfg.group : kHeadDim);
  const long long page_bytes = is_int2(c) ? 2LL * kPage * (kRowBytes + 4 * ng) : 2LL * kPage * kHeadDim * 2;
  long long total_bytes = 0;
  for (int i = 0; i < n_req; ++i) {
    np_of[i] = pages_needed(c, Ls[i], Hs[i]);
    nbf_of[i] = is_int2(c) ? std::min(Ls[i], S) + std::max(0, Ls[i] - Hs[i]) : 0;
    bfnew_of[i] = nbf_of[i];
    pgnew_of[i] = np_of[i];
    // A fused launch's BF16 items of an appending request wait for its rows as a whole (the
    // new rows are a small part of the list); its INT2 items are not split: the append's
    // eviction rows are signalled before the launch's wait, and the one warp whose page
    // holds them waits for that signal before copying it.
    if (app_items[i] > 0) bfnew_of[i] = 0;
    max_np = std::max(max_np, np_of[i] - p0_of[i]);
    total_bytes += (long long)Hkv * ((np_of[i] - p0_of[i]) * page_bytes + nbf_of[i] * 2LL * kHeadDim * 2);
  }
  // CTA shape: at GQA 4 a step that one wave of 16-warp CTAs holds (one per SM) is planned
  // for them ("wide"); larger steps for 8-warp CTAs, two per SM.
  constexpr long long kItemBytes = 512 << 10;
  constexpr long long kWaves = 2;
  const int G = c->cfg.n_q_heads / Hkv;
  bool wide = false;
  if (is_int2(c) && G == 4 && !(flags & OSCAR_PLAN_NARROW)) {
    const int r_wide = decode_resident_ctas(G, c->cfg.group, true, is_cm(c), c->n_sm);
    wide = r_wide > 0 && total_bytes <= kItemBytes * r_wide;
  }
  if (!is_int2(c)) {  // BF16: the deeper row pipeline for steps that one wave holds
    const int r_deep = bf16_decode_resident_ctas(G, true, c->n_sm);
    wide = r_deep > 0 && total_bytes <= kItemBytes * r_deep;
  }
  const int nw = decode_warps(G, wide);
  for (int i = 0; i < n_req; ++i) app_expect[i] = 2 * append_task_split(nw) * app_items[i];  // per kv-head
  if ((c->inject & OSCAR_FAULT_LOST_APPEND_SIGNAL) && c->reserved)
    for (int i = 0; i < n_req; ++i)
      if (app_expect[i] > 0) {  // one signal more than the append tasks send: it never arrives
        ++app_expect[i];
        c->inject &= ~OSCAR_FAULT_LOST_APPEND_SIGNAL;
        break;
      }
  auto split_count = [](int a, int b, int step) { return (a > 0 ? ceil_div(a, step) : 0) + (b > a ? ceil_div(b - a, step) : 0); };
  long long n_bf_items = 0, n_shared_slots = 0;
  for (int i = 0; i < n_req; ++i) n_shared_slots += (long long)Hkv * runs.n_segs[i];
  // BF16 items of one CTA chunk: 16 tokens per warp
  const int bf_item = is_int2(c) ? 16 * nw : kBf16ItemTokens;
  for (int i = 0; i < n_req; ++i) n_bf_items += (long long)Hkv * split_count(bfnew_of[i], nbf_of[i], bf_item);
  auto count_items = [&](int ch) {
    long long n = n_bf_items;
    for (int i = 0; i < n_req; ++i) {
      const int pg = split_count(pgnew_of[i] - p0_of[i], np_of[i] - p0_of[i], ch);
      const int bf = split_count(bfnew_of[i], nbf_of[i], bf_item);
      n += (long long)Hkv * (pg + bf > 0 ? pg : 1);
    }
    return n;
  };
  int chunk = max_split_pages;
  if (chunk == 0) {
    int resident =
        is_int2(c) ? decode_resident_ctas(G, c->cfg.group, wide, is_cm(c), c->n_sm) : bf16_decode_resident_ctas(G, wide, c->n_sm);
    if (resident <= 0) resident = 2 * c->n_sm;
    if (total_bytes <= kItemBytes * resident) {
      // a fused append + decode launch runs the reservation's append tasks in the same wave
      const long long n_app_tasks =
          c->reserved && !is_cm(c) ? (long long)c->app_items * Hkv * 2 * append_task_split(nw) : 0;
      const long long slots = std::max<long long>(1, resident - n_bf_items - n_app_tasks);
      chunk = int(std::max<long long>(4, (total_pages + slots - 1) / slots));
      while (chunk < max_np && count_items(chunk) + n_app_tasks > resident) ++chunk;
    } else {
      const long long item_bytes = std::max(kItemBytes, total_bytes / (kWaves * resident));
      chunk = int(std::max<long long>(4, item_bytes / page_bytes));
    }
    // the plan must fit the item buffers
    while (chunk < max_np && count_items(chunk) + n_shared_slots > (long long)c->lay.max_decode_items)
      chunk = std::min(max_np, chunk + chunk / 4 + 1);
  }
  std::vector<DecodeReq> reqs(n_req);
  std::vector<DecodeItem> items;
  int n_bf16 = 0, max_pages = 0, n_slots = 0;
  long long tokens = 0;  // of all kv-heads
  std::vector<long long> score_base(n_req);
  for (int i = 0; i < n_req; ++i) {
    DecodeReq& q = reqs[i];
    q.slot = slots[i];
    q.L = Ls[i];
    q.H = is_int2(c) ? Hs[i] : Ls[i];
    q.H_pre = is_int2(c) ? Hpre[i] : Lpre[i];
    q.app_expect = is_int2(c) ? app_expect[i] : 0;
    const int np = np_of[i], n_bf = nbf_of[i], bf_new = bfnew_of[i], pg_new = pgnew_of[i], page0 = p0_of[i];
    // BF16 list index of this step's first new row (index < min(L, S): sink, else ring
    // position H + index - min(L, S)); rows before it are final before the launch's wait
    int u_new = n_bf;
    if (is_int2(c) && Lpre[i] < Ls[i]) {
      const int n_s = std::min(q.L, S);
      u_new = std::min(n_bf, Lpre[i] < n_s ? Lpre[i] : n_s + std::max(0, Lpre[i] - q.H));
    }
    score_base[i] = tokens;
    tokens += (long long)Hkv * q.L;
    q.first_item = n_slots;
    q.n_shared = runs.n_segs[i];
    for (int h = 0; h < Hkv; ++h) {
      const size_t first = items.size();
      const int first_slot = n_slots;
      n_slots += q.n_shared;
      auto add = [&](int kind, int b, int e, int dep) {
        items.push_back({i, h, kind, b, e, first_slot, 0, dep, kind == 1 ? std::min(e, std::max(b, u_new)) : e, n_slots++});
      };
      // no private tokens: one empty item, which merges (an empty request's writes zeros)
      if (n_bf == 0 && np == page0) add(1, 0, 0, kDepNone);
      // BF16 sink+ring list, split where this step's new tokens start (those items wait for
      // a fused launch's append tasks; the others do not)
      for (int part = 0; part < 2; ++part) {
        const int b0 = part == 0 ? 0 : bf_new, b1 = part == 0 ? bf_new : n_bf;
        for (int t = b0; t < b1; t += bf_item) {
          add(1, t, std::min(b1, t + bf_item), part == 0 ? kDepNone : kDepRing);
          ++n_bf16;
        }
      }
      // INT2 pages, split where pages that this step's append writes begin
      for (int part = 0; part < 2; ++part) {
        const int p0 = part == 0 ? page0 : pg_new, p1 = part == 0 ? pg_new : np;
        for (int p = p0; p < p1; p += chunk) {
          add(0, p, std::min(p1, p + chunk), part == 0 ? kDepNone : kDepPages);
          max_pages = std::max(max_pages, std::min(p1, p + chunk) - p);
        }
      }
      for (size_t k = first; k < items.size(); ++k) items[k].head_count = n_slots - first_slot;
    }
    q.items_per_head = (n_slots - q.first_item) / Hkv;
  }
  if (size_t(n_slots) > c->lay.max_decode_items)
    return fail(OSCAR_ERR_INVALID_ARG, "plan of %d items exceeds %zu; raise max_split_pages", n_slots,
                c->lay.max_decode_items);
  // the order CTAs take items in (when they are more than one wave): the items that wait
  // on no append task first, then those that may wait; largest first within each (stable)
  std::vector<int> order(items.size());
  for (size_t k = 0; k < items.size(); ++k) order[k] = int(k);
  auto cost = [&](const DecodeItem& d) {
    return d.kind == 0 ? (long long)(d.end - d.begin) * page_bytes : (long long)(d.end - d.begin) * 2LL * kHeadDim * 2;
  };
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) {
    const bool wa = items[a].dep != kDepNone, wb = items[b].dep != kDepNone;
    if (wa != wb) return wb;
    return cost(items[a]) > cost(items[b]);
  });
  int n_front = 0;
  while (n_front < int(order.size()) && items[order[n_front]].dep == kDepNone) ++n_front;
  Upload u;
  oscar_status st = begin_upload(c, &u);
  if (st) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the decode plan block, one copy: the items in the order CTAs take them, each with its
  // partial slot (its index above)
  const size_t items_off = decode_items_offset(c->cfg.max_requests);
  int32_t* counts = reinterpret_cast<int32_t*>(u.staging);
  counts[0] = int(items.size());
  counts[1] = n_req;
  counts[2] = n_front;
  counts[3] = int(runs.items.size());
  std::memcpy(u.staging + 256, reqs.data(), reqs.size() * sizeof(DecodeReq));
  std::memcpy(u.staging + score_base_offset(c->cfg.max_requests), score_base.data(), score_base.size() * 8);
  DecodeItem* staged = reinterpret_cast<DecodeItem*>(u.staging + items_off);
  for (size_t k = 0; k < order.size(); ++k) staged[k] = items[order[k]];
  if (!runs.items.empty()) {
    const size_t at = shared_items_offset(c->cfg.max_requests);
    uint8_t* to = u.staging + align256(items_off + items.size() * sizeof(DecodeItem));
    std::memcpy(to, runs.order.data(), runs.order.size() * 4);
    std::memcpy(to + at, runs.items.data(), runs.items.size() * sizeof(SharedItem));
    CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.shared_order, to, at + runs.items.size() * sizeof(SharedItem),
                             cudaMemcpyHostToDevice, s));
  }
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.decode_plan, u.staging, items_off + items.size() * sizeof(DecodeItem),
                           cudaMemcpyHostToDevice, s));
  st = end_upload(c, u, s);
  if (st) return st;
  DecodeWorkspace w;
  size_t off = 0;
  w.partials = off;
  off = align256(off + size_t(n_slots) * size_t(G) * (8 + 4 * kHeadDim));  // partial slots
  w.total = off;
  c->ws = w;
  c->dec_n_req = n_req;
  c->dec_tokens = tokens;
  c->dec_items = int(items.size());
  c->dec_bf16_items = n_bf16;
  c->dec_max_pages = max_pages;
  c->planned = true;
  c->planned_with_reservation = c->reserved;
  c->dec_wide = wide;
  c->dec_folded = (flags & OSCAR_PLAN_FOLDED_ROTATIONS) != 0;
  c->dec_shared = shared;
  c->dec_shared_items = int(runs.items.size());
  c->dec_shared_pages = runs.pages;
  c->plan_covers_reservation = c->reserved && n_reserved_planned == int(c->app_reqs.size());
  return OSCAR_OK;
} catch (const std::bad_alloc&) {
  return fail(OSCAR_ERR_INVALID_ARG, "host allocation failed");
}

size_t oscar_decode_workspace_bytes(const oscar_cache* c) { return (c && c->planned) ? c->ws.total : 0; }

size_t oscar_decode_workspace_max_bytes(const oscar_cache* c) {
  if (!c) return 0;
  const size_t G = size_t(c->cfg.n_q_heads / c->cfg.n_kv_heads);
  return align256(c->lay.max_decode_items * G * (8 + 4 * kHeadDim));
}

oscar_status oscar_plan_info(const oscar_cache* c, int* n_items, int* n_bf16_items, int* max_item_pages) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->planned) return fail(OSCAR_ERR_STATE, "no decode plan");
  if (n_items) *n_items = c->dec_items;
  if (n_bf16_items) *n_bf16_items = c->dec_bf16_items;
  if (max_item_pages) *max_item_pages = c->dec_max_pages;
  return OSCAR_OK;
}

oscar_status oscar_plan_shared_info(const oscar_cache* c, int* n_items, int* n_pages) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->planned) return fail(OSCAR_ERR_STATE, "no decode plan");
  if (n_items) *n_items = c->dec_shared_items;
  if (n_pages) *n_pages = c->dec_shared_pages;
  return OSCAR_OK;
}

static oscar_status check_decode(oscar_cache* c, int layer, const void* q, void* out, void* ws, size_t ws_bytes) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->planned) return fail(OSCAR_ERR_STATE, "no decode plan (plan after every append commit)");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (!q || !out || !ws) return fail(OSCAR_ERR_INVALID_ARG, "NULL q, out or workspace");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(OSCAR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (ws_bytes < c->ws.total) return fail(OSCAR_ERR_INVALID_ARG, "workspace %zu < %zu bytes", ws_bytes, c->ws.total);
  return OSCAR_OK;
}

oscar_status oscar_decode_attention(oscar_cache* c, int layer, const void* q, void* out, void* workspace, size_t ws_bytes,
                                    float* out_f32, void* stream) {
  g_launches = 0;
  oscar_status st = check_decode(c, layer, q, out, workspace, ws_bytes);
  if (st) return st;
  if (!is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_decode_attention needs the INT2 format");
  int e = launch_decode(kernel_params(c), layer, q, out, out_f32, static_cast<uint8_t*>(workspace), c->ws, c->dec_wide,
                        c->n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "decode launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_append_decode_attention(oscar_cache* c, int layer, const void* k_new, const void* v_new,
                                           const void* q, void* out, void* workspace, size_t ws_bytes, float* out_f32,
                                           void* stream) {
  g_launches = 0;
  oscar_status st = check_decode(c, layer, q, out, workspace, ws_bytes);
  if (st) return st;
  if (!is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_append_decode_attention needs the INT2 format");
  if (!c->reserved) return fail(OSCAR_ERR_STATE, "no reservation");
  if (!c->plan_covers_reservation)
    return fail(OSCAR_ERR_STATE, "plan the decode after the reservation, over every reserved slot");
  if (c->app_rows > 0 && (!k_new || !v_new)) return fail(OSCAR_ERR_INVALID_ARG, "NULL token arrays");
  // The append tasks run in the same wave as the decode when they fit in it; more of them
  // (long chunks, many requests) would hold back the decode, so those go to the append
  // kernel, which is launched first.
  const int G = c->cfg.n_q_heads / c->cfg.n_kv_heads;
  const int resident = decode_resident_ctas(G, c->cfg.group, c->dec_wide, is_cm(c), c->n_sm);
  const long long n_tasks =
      (long long)c->app_items * c->cfg.n_kv_heads * 2 * append_task_split(decode_warps(G, c->dec_wide));
  const bool fused = !is_cm(c) && n_tasks <= (long long)resident;
  if (!fused && c->app_items > 0) {
    int e = launch_append(kernel_params(c), layer, k_new, v_new, c->app_items, c->n_sm, stream, &g_launches);
    if (e) return fail(OSCAR_ERR_CUDA, "append launch: %s", cudaGetErrorString(cudaError_t(e)));
  }
  int e = launch_decode(kernel_params(c), layer, q, out, out_f32, static_cast<uint8_t*>(workspace), c->ws, c->dec_wide,
                        c->n_sm, stream, &g_launches, k_new, v_new, fused);
  if (e) return fail(OSCAR_ERR_CUDA, "append + decode launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_bf16_decode_attention(oscar_cache* c, int layer, const void* q, void* out, void* workspace,
                                         size_t ws_bytes, float* out_f32, void* stream) {
  g_launches = 0;
  oscar_status st = check_decode(c, layer, q, out, workspace, ws_bytes);
  if (st) return st;
  if (is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_bf16_decode_attention needs the BF16 format");
  int e = 0;
  // A captured decode is replayed under later plans, which may share.
  bool with_shared = c->dec_shared && c->dec_shared_items > 0;
  if (c->dec_shared && !with_shared) {
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    CUDA_TRY(cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &capturing));
    with_shared = capturing != cudaStreamCaptureStatusNone;
  }
  if (with_shared) {
    st = check_device(c);
    if (st) return st;
    e = launch_shared(kernel_params(c), layer, c->page_map, q, static_cast<uint8_t*>(workspace) + c->ws.partials, c->n_sm,
                      stream, &g_launches);
  }
  if (!e)
    e = launch_bf16_decode(kernel_params(c), layer, q, out, out_f32, static_cast<uint8_t*>(workspace), c->ws, c->dec_wide,
                           with_shared, c->n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "bf16 decode launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

int oscar_weights_stride(const oscar_cache* c) {
  if (!c || is_int2(c)) return 0;
  return kPage * std::min(c->cfg.max_pages_per_request, c->cfg.max_pages);
}

size_t oscar_decode_weights_workspace_bytes(const oscar_cache* c) {
  return c && c->planned && !is_int2(c) ? weights_workspace(c, size_t(c->dec_tokens)).total : 0;
}

size_t oscar_decode_weights_workspace_max_bytes(const oscar_cache* c) {
  if (!c || is_int2(c)) return 0;
  return weights_workspace(c, size_t(c->cfg.max_requests) * c->cfg.n_kv_heads * size_t(oscar_weights_stride(c))).total;
}

oscar_status oscar_bf16_decode_weights(oscar_cache* c, int layer, const void* q, void* out, const float* weights_in,
                                       float* weights_out, void* workspace, size_t ws_bytes, float* out_f32,
                                       void* stream) {
  g_launches = 0;
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_bf16_decode_weights needs the BF16 format");
  if (!c->planned) return fail(OSCAR_ERR_STATE, "no decode plan (plan after every append commit)");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (c->dec_shared)
    return fail(OSCAR_ERR_STATE, "oscar_bf16_decode_weights needs a plan without OSCAR_PLAN_SHARED_PREFIX");
  if (!q || !out || !weights_out || !workspace)
    return fail(OSCAR_ERR_INVALID_ARG, "NULL q, out, weights_out or workspace");
  if ((reinterpret_cast<uintptr_t>(weights_in) | reinterpret_cast<uintptr_t>(weights_out)) % 4)
    return fail(OSCAR_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  const uintptr_t wi = reinterpret_cast<uintptr_t>(weights_in), wo = reinterpret_cast<uintptr_t>(weights_out);
  const uintptr_t w_bytes = uintptr_t(c->cfg.max_requests) * c->cfg.n_kv_heads * uintptr_t(oscar_weights_stride(c)) * 4;
  if (wi && wi != wo && wi < wo + w_bytes && wo < wi + w_bytes)
    return fail(OSCAR_ERR_INVALID_ARG, "weights_in and weights_out overlap");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(OSCAR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const WeightsWorkspace w = weights_workspace(c, size_t(c->dec_tokens));
  if (ws_bytes < w.total) return fail(OSCAR_ERR_INVALID_ARG, "workspace %zu < %zu bytes", ws_bytes, w.total);
  oscar_status st = check_device(c);
  if (st) return st;
  const int e = launch_bf16_decode_weights(kernel_params(c), layer, q, out, out_f32, weights_in, weights_out,
                                           static_cast<uint8_t*>(workspace), w, c->dec_wide, c->n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "decode with weights launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_evict_begin(oscar_cache* c, const int* slots, const int* keep, int n_req, int n_sink, int n_recent,
                               void* stream) try {
  if (!c || !slots || !keep || n_req <= 0 || n_req > c->cfg.max_requests)
    return fail(OSCAR_ERR_INVALID_ARG, "bad evict arguments");
  if (is_int2(c)) return fail(OSCAR_ERR_STATE, "eviction needs the BF16 format");
  if (c->reserved) return fail(OSCAR_ERR_STATE, "a reservation is pending");
  if (c->evicting) return fail(OSCAR_ERR_STATE, "an eviction is pending");
  if (n_sink < 0 || n_recent < 0) return fail(OSCAR_ERR_INVALID_ARG, "negative n_sink or n_recent");
  std::vector<char> seen(c->cfg.max_requests, 0);
  std::vector<EvictReq> reqs(n_req);
  int new_pages = 0, max_pages = 0;
  for (int i = 0; i < n_req; ++i) {
    oscar_status st = check_slot(c, slots[i]);
    if (st) return st;
    if (seen[slots[i]]) return fail(OSCAR_ERR_INVALID_ARG, "slot %d listed twice", slots[i]);
    seen[slots[i]] = 1;
    if (keep[i] < 0) return fail(OSCAR_ERR_INVALID_ARG, "negative keep");
    EvictReq& r = reqs[i];
    r.slot = slots[i];
    r.L = c->reqs[slots[i]].L;
    r.keep = std::min(keep[i], r.L);
    r.n_sink = std::min(n_sink, r.L);
    r.n_recent = std::min(n_recent, r.L - r.n_sink);
    if (r.keep < r.L && r.n_sink + r.n_recent > r.keep)
      return fail(OSCAR_ERR_INVALID_ARG, "slot %d: keep %d < %d protected tokens", slots[i], r.keep, r.n_sink + r.n_recent);
    if (r.keep < r.L) {
      new_pages += ceil_div(r.keep, kPage);
      max_pages = std::max(max_pages, ceil_div(r.keep, kPage));
    }
  }
  if (new_pages > int(c->free_pages.size()))
    return fail(OSCAR_ERR_OUT_OF_PAGES, "need %d pages, %zu free", new_pages, c->free_pages.size());
  Upload u;
  oscar_status st = begin_upload(c, &u);
  if (st) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t row = size_t(c->cfg.max_pages_per_request);
  int32_t* counts = reinterpret_cast<int32_t*>(u.staging);
  counts[0] = n_req;
  counts[1] = counts[2] = counts[3] = 0;
  std::memcpy(u.staging + 256, reqs.data(), reqs.size() * sizeof(EvictReq));
  std::vector<std::vector<int>> pages(n_req);
  size_t at = c->free_pages.size();  // taken from the end; given out once the uploads are enqueued
  for (int i = 0; i < n_req; ++i) {
    if (reqs[i].keep >= reqs[i].L) continue;
    for (int k = 0; k < ceil_div(reqs[i].keep, kPage); ++k) pages[i].push_back(c->free_pages[--at]);
    if (pages[i].empty()) continue;
    int32_t* src = u.rows + size_t(i) * row;
    std::copy(pages[i].begin(), pages[i].end(), src);
    CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.evict_pages + size_t(i) * row * 4, src, pages[i].size() * 4,
                             cudaMemcpyHostToDevice, s));
  }
  CUDA_TRY(cudaMemcpyAsync(c->base + c->lay.evict_plan, u.staging, 256 + reqs.size() * sizeof(EvictReq),
                           cudaMemcpyHostToDevice, s));
  st = end_upload(c, u, s);
  if (st) return st;
  c->free_pages.resize(at);
  for (const auto& v : pages)
    for (int p : v) c->refcount[p] = 1;
  c->ev_reqs = std::move(reqs);
  c->ev_pages = std::move(pages);
  c->ev_max_pages = max_pages;
  c->evicting = true;
  return OSCAR_OK;
} catch (const std::bad_alloc&) {
  return fail(OSCAR_ERR_INVALID_ARG, "host allocation failed");
}

oscar_status oscar_evict(oscar_cache* c, int layer, const float* weights, float* weights_out, int* kept, void* stream) {
  g_launches = 0;
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->evicting) return fail(OSCAR_ERR_STATE, "no eviction begun");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (!weights || !weights_out || !kept) return fail(OSCAR_ERR_INVALID_ARG, "NULL weights, weights_out or kept");
  if (reinterpret_cast<uintptr_t>(weights) % 16) return fail(OSCAR_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(weights_out) | reinterpret_cast<uintptr_t>(kept)) % 4)
    return fail(OSCAR_ERR_INVALID_ARG, "weights_out and kept must be 4-byte aligned");
  const uintptr_t bytes = uintptr_t(c->cfg.max_requests) * c->cfg.n_kv_heads * uintptr_t(oscar_weights_stride(c)) * 4;
  const uintptr_t at[3] = {reinterpret_cast<uintptr_t>(weights), reinterpret_cast<uintptr_t>(weights_out),
                           reinterpret_cast<uintptr_t>(kept)};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (at[i] < at[j] + bytes && at[j] < at[i] + bytes)
        return fail(OSCAR_ERR_INVALID_ARG, "weights, weights_out and kept must not overlap");
  oscar_status st = check_device(c);
  if (st) return st;
  int max_len = 0;
  for (const EvictReq& r : c->ev_reqs) max_len = std::max(max_len, r.L);
  const int e = launch_evict(kernel_params(c), layer, weights, weights_out, kept, int(c->ev_reqs.size()), max_len, c->ev_max_pages,
                             c->n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "evict launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_evict_pages(const oscar_cache* c, int slot, int* pages, int n, int* n_pages) {
  oscar_status st = check_slot(c, slot);
  if (st) return st;
  if (!c->evicting) return fail(OSCAR_ERR_STATE, "no eviction begun");
  const std::vector<int>* v = &c->reqs[slot].pages;  // a request that gives nothing up keeps its pages
  for (size_t i = 0; i < c->ev_reqs.size(); ++i)
    if (c->ev_reqs[i].slot == slot && c->ev_reqs[i].keep < c->ev_reqs[i].L) v = &c->ev_pages[i];
  if (n_pages) *n_pages = int(v->size());
  if (n < 0 || (n > 0 && !pages)) return fail(OSCAR_ERR_INVALID_ARG, "bad page buffer");
  std::copy(v->begin(), v->begin() + std::min<size_t>(size_t(n), v->size()), pages);
  return OSCAR_OK;
}

oscar_status oscar_evict_commit(oscar_cache* c, void* stream) try {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->evicting) return fail(OSCAR_ERR_STATE, "no eviction begun");
  Upload u;
  oscar_status st = begin_upload(c, &u);
  if (st) return st;
  std::vector<int> changed;
  changed.reserve(c->ev_reqs.size());  // nothing below allocates
  for (size_t i = 0; i < c->ev_reqs.size(); ++i) {
    const EvictReq& e = c->ev_reqs[i];
    if (e.keep >= e.L) continue;
    Request& r = c->reqs[e.slot];
    for (int p : r.pages)
      if (--c->refcount[p] == 0) c->free_pages.push_back(p);
    r.pages.swap(c->ev_pages[i]);
    r.L = r.H = e.keep;
    int32_t* row = c->h_page_table + size_t(e.slot) * c->cfg.max_pages_per_request;
    std::fill(row, row + c->cfg.max_pages_per_request, -1);
    std::copy(r.pages.begin(), r.pages.end(), row);
    changed.push_back(e.slot);
  }
  c->evicting = false;
  c->ev_reqs.clear();
  c->ev_pages.clear();
  if (!changed.empty()) c->planned = false;  // lengths changed: plan again
  st = upload_rows(c, u, changed, static_cast<cudaStream_t>(stream));
  if (st) return st;
  return end_upload(c, u, static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return fail(OSCAR_ERR_INVALID_ARG, "host allocation failed");
}

oscar_status oscar_evict_cancel(oscar_cache* c) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!c->evicting) return fail(OSCAR_ERR_STATE, "no eviction begun");
  for (size_t i = c->ev_pages.size(); i-- > 0;)
    for (size_t k = c->ev_pages[i].size(); k-- > 0;) {
      c->refcount[c->ev_pages[i][k]] = 0;
      c->free_pages.push_back(c->ev_pages[i][k]);
    }
  c->evicting = false;
  c->ev_reqs.clear();
  c->ev_pages.clear();
  return OSCAR_OK;
}

oscar_status oscar_decode_attention_noalloc(oscar_cache* c, int layer, const void* q, void* out, float* out_f32,
                                            void* stream) {
  g_launches = 0;
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (!is_int2(c)) return fail(OSCAR_ERR_STATE, "oscar_decode_attention_noalloc needs the INT2 format");
  if (!c->planned) return fail(OSCAR_ERR_STATE, "no decode plan (plan after every append commit)");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(OSCAR_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (!q || !out) return fail(OSCAR_ERR_INVALID_ARG, "NULL q or out");
  int dev = -1;
  cudaError_t de = cudaGetDevice(&dev);
  if (de != cudaSuccess) return fail(OSCAR_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(de));
  if (dev != c->device)
    return fail(OSCAR_ERR_INVALID_ARG, "current device %d is not the cache's device %d (the library scratch is looked "
                "up on the current device)", dev, c->device);
  bool too_big = false;
  int e = launch_decode_static_scratch(kernel_params(c), layer, q, out, out_f32, c->ws, c->dec_wide,
                                       c->n_sm, stream, &g_launches, &too_big);
  if (too_big)
    return fail(OSCAR_ERR_INVALID_ARG,
                "decode plan needs %zu bytes of scratch, more than the library's fixed %zu; use "
                "oscar_decode_attention with a caller workspace or plan fewer requests / larger splits",
                c->ws.total, static_scratch_bytes());
  if (e) return fail(OSCAR_ERR_CUDA, "decode launch (library scratch): %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

size_t oscar_calibration_workspace_bytes(int n_tokens, int n_q_heads, int n_kv_heads) {
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads) return 0;
  return calib_workspace(n_tokens, n_q_heads, n_kv_heads).total;
}

oscar_status oscar_calibrate_layer(const void* q, const void* k, const void* v, int n_tokens, int n_q_heads,
                                   int n_kv_heads, long long clip_rank, int rotation, float* R_K, float* R_V,
                                   float* clip_K, float* clip_V, double* covariances, void* workspace,
                                   size_t ws_bytes, void* stream) {
  g_launches = 0;
  if (!q || !k || !v || !R_K || !R_V || !clip_K || !clip_V || !workspace)
    return fail(OSCAR_ERR_INVALID_ARG, "NULL input, output or workspace");
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads)
    return fail(OSCAR_ERR_INVALID_ARG, "bad shape: %d tokens, %d query heads, %d kv-heads", n_tokens, n_q_heads,
                n_kv_heads);
  if (rotation != OSCAR_ROTATION_OSCAR && rotation != OSCAR_ROTATION_HADAMARD)
    return fail(OSCAR_ERR_INVALID_ARG, "unknown rotation %d", rotation);
  if (clip_rank < 1 || clip_rank > (long long)n_tokens * kHeadDim)
    return fail(OSCAR_ERR_INVALID_ARG, "clip_rank %lld outside [1, %lld]", clip_rank, (long long)n_tokens * kHeadDim);
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(OSCAR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const size_t need = calib_workspace(n_tokens, n_q_heads, n_kv_heads).total;
  if (ws_bytes < need) return fail(OSCAR_ERR_INVALID_ARG, "calibration workspace of %zu bytes < %zu needed", ws_bytes, need);
  const int e = launch_calibrate(q, k, v, n_tokens, n_q_heads, n_kv_heads, long(clip_rank),
                                 rotation == OSCAR_ROTATION_HADAMARD, R_K, R_V, clip_K, clip_V, covariances,
                                 static_cast<uint8_t*>(workspace), stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "calibration launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_rope_steps(const oscar_rope_config* cfg, uint64_t* steps, float* magnitude) {
  if (!cfg || !steps || !magnitude) return fail(OSCAR_ERR_INVALID_ARG, "NULL argument");
  const int R = cfg->rotary_dim;
  if (R < 2 || R > 512 || R % 2) return fail(OSCAR_ERR_INVALID_ARG, "rotary_dim %d must be even and in [2, 512]", R);
  if (!(cfg->base > 1.0) || !std::isfinite(cfg->base)) return fail(OSCAR_ERR_INVALID_ARG, "base must be > 1");
  if (cfg->scaling < OSCAR_ROPE_UNSCALED || cfg->scaling > OSCAR_ROPE_YARN)
    return fail(OSCAR_ERR_INVALID_ARG, "unknown scaling %d", cfg->scaling);
  const bool banded = cfg->scaling == OSCAR_ROPE_BANDS || cfg->scaling == OSCAR_ROPE_YARN;
  if (cfg->scaling != OSCAR_ROPE_UNSCALED &&
      (!(cfg->factor > 0.0) || !std::isfinite(cfg->factor) || (cfg->scaling == OSCAR_ROPE_YARN && cfg->factor < 1.0)))
    return fail(OSCAR_ERR_INVALID_ARG, "factor %g out of range", cfg->factor);
  if (banded && (!(cfg->low > 0.0) || !(cfg->high > cfg->low) || !std::isfinite(cfg->high) ||
                 !(cfg->original_context > 0.0) || !std::isfinite(cfg->original_context)))
    return fail(OSCAR_ERR_INVALID_ARG, "scaling needs 0 < low < high and original_context > 0");
  const double two_pi = 6.283185307179586476925;
  double x0 = 0.0, x1 = 0.0;
  if (cfg->scaling == OSCAR_ROPE_YARN) {
    auto index = [&](double n) {
      return R * std::log(cfg->original_context / (two_pi * n)) / (2.0 * std::log(cfg->base));
    };
    x0 = std::min(std::max(std::floor(index(cfg->high)), 0.0), R - 1.0);
    x1 = std::min(std::max(std::ceil(index(cfg->low)), 0.0), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(cfg->base, -2.0 * i / R);
    double keep = 1.0;  // share of the unscaled frequency
    if (cfg->scaling == OSCAR_ROPE_LINEAR) keep = 0.0;
    if (cfg->scaling == OSCAR_ROPE_BANDS) {
      const double n = cfg->original_context * f / two_pi;
      keep = std::min(std::max((n - cfg->low) / (cfg->high - cfg->low), 0.0), 1.0);
    }
    if (cfg->scaling == OSCAR_ROPE_YARN)
      keep = 1.0 - std::min(std::max((i - x0) / std::max(x1 - x0, 0.001), 0.0), 1.0);
    if (cfg->scaling != OSCAR_ROPE_UNSCALED) f = f / cfg->factor * (1.0 - keep) + f * keep;
    double turns = f / two_pi;
    turns -= std::floor(turns);  // positions are whole numbers: whole turns a position are none
    steps[i] = uint64_t(std::ldexp(turns, 64));
  }
  *magnitude = cfg->scaling == OSCAR_ROPE_YARN ? float(0.1 * std::log(cfg->factor) + 1.0) : 1.0f;
  return OSCAR_OK;
}

oscar_status oscar_rope(const oscar_rope_tensor* tensors, int n_tensors, const uint64_t* steps, int head_dim,
                        int rotary_dim, float magnitude, int dtype, uint32_t flags, const void* positions,
                        long long n_rows, void* stream) {
  g_launches = 0;
  if (!tensors || n_tensors < 1 || n_tensors > 2) return fail(OSCAR_ERR_INVALID_ARG, "one or two tensors");
  if (rotary_dim < 2 || rotary_dim % 2 || head_dim < rotary_dim || head_dim > 512)
    return fail(OSCAR_ERR_INVALID_ARG, "rotary_dim %d must be even, head_dim %d in [rotary_dim, 512]", rotary_dim, head_dim);
  if (dtype != OSCAR_DTYPE_BF16 && dtype != OSCAR_DTYPE_F16 && dtype != OSCAR_DTYPE_F32)
    return fail(OSCAR_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
  if (flags & ~(OSCAR_ROPE_INTERLEAVED | OSCAR_ROPE_TRANSPOSE | OSCAR_ROPE_POSITIONS64))
    return fail(OSCAR_ERR_INVALID_ARG, "unknown rope flags %#x", flags);
  if (n_rows < 0 || n_rows > 0x7fffffffLL) return fail(OSCAR_ERR_INVALID_ARG, "n_rows %lld out of range", n_rows);
  const size_t size = dtype == OSCAR_DTYPE_F32 ? 4 : 2;
  const size_t pos_size = flags & OSCAR_ROPE_POSITIONS64 ? 8 : 4;
  RopeParams p = {};
  bool aligned = true;
  for (int i = 0; i < n_tensors; ++i) {
    const oscar_rope_tensor& t = tensors[i];
    if (t.n_heads < 1 || t.n_heads > 65536) return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: %d heads", i, t.n_heads);
    if (n_rows > 0 && (!t.in || !t.out)) return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: NULL in or out", i);
    if (t.in_row < 0 || t.in_head < 0 || t.out_row < 0 || t.out_head < 0)
      return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: negative stride", i);
    // outputs: heads inside their row, or rows inside their head
    const bool rows_out = (t.n_heads == 1 || t.out_head >= head_dim) &&
                          (n_rows <= 1 || t.out_row >= (t.n_heads - 1) * t.out_head + head_dim);
    const bool heads_out = (n_rows <= 1 || t.out_row >= head_dim) &&
                           (t.n_heads == 1 || t.out_head >= (n_rows - 1) * t.out_row + head_dim);
    if (!rows_out && !heads_out) return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: output rows or heads overlap", i);
    if (t.in == t.out && ((n_rows > 1 && t.in_row != t.out_row) || (t.n_heads > 1 && t.in_head != t.out_head)))
      return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: in place with other strides", i);
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
    if (a % size) return fail(OSCAR_ERR_INVALID_ARG, "tensor %d: not aligned to its dtype", i);
    if (a % 16 || (t.in_row * size) % 16 || (t.in_head * size) % 16 || (t.out_row * size) % 16 || (t.out_head * size) % 16)
      aligned = false;
    p.x[i] = {t.in, t.out, t.n_heads, t.in_row, t.in_head, t.out_row, t.out_head};
  }
  if (n_rows == 0) return OSCAR_OK;
  if (!steps || !positions) return fail(OSCAR_ERR_INVALID_ARG, "NULL steps or positions");
  if (reinterpret_cast<uintptr_t>(steps) % 8 || reinterpret_cast<uintptr_t>(positions) % pos_size)
    return fail(OSCAR_ERR_INVALID_ARG, "steps or positions are not aligned to their type");
  p.steps = steps;
  p.positions = positions;
  p.n_rows = n_rows;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.magnitude = magnitude;
  p.interleaved = (flags & OSCAR_ROPE_INTERLEAVED) != 0;
  p.transpose = (flags & OSCAR_ROPE_TRANSPOSE) != 0;
  p.positions64 = (flags & OSCAR_ROPE_POSITIONS64) != 0;
  int dev = 0, n_sm = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev));
  const int e = launch_rope(p, dtype, aligned, n_sm, stream, &g_launches);
  if (e) return fail(OSCAR_ERR_CUDA, "rope launch: %s", cudaGetErrorString(cudaError_t(e)));
  return OSCAR_OK;
}

oscar_status oscar_set_wait_limit(oscar_cache* c, uint32_t counter_polls) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  c->counter_polls = counter_polls;
  return OSCAR_OK;
}

oscar_status oscar_inject_fault(oscar_cache* c, uint32_t faults) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  if (faults & ~uint32_t(OSCAR_FAULT_LOST_APPEND_SIGNAL)) return fail(OSCAR_ERR_INVALID_ARG, "unknown faults %#x", faults);
  c->inject |= faults;
  return OSCAR_OK;
}

oscar_status oscar_get_status(oscar_cache* c, void* stream, uint32_t* flags) {
  if (!c) return fail(OSCAR_ERR_INVALID_ARG, "cache is NULL");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUDA_TRY(cudaMemcpyAsync(c->h_status, c->base + c->lay.status, 4, cudaMemcpyDeviceToHost, s));
  CUDA_TRY(cudaStreamSynchronize(s));
  uint32_t f = c->h_status[0];
  if (flags) *flags = f;
  if (f) {
    CUDA_TRY(cudaMemsetAsync(c->base + c->lay.status, 0, 4, s));
    if (f & OSCAR_FLAG_TIMEOUT) {
      // a wait gave up: the append-dependency counters may be off by the signals that never
      // came (or came late), so they restart from zero (no launch of this cache is in flight:
      // the stream is synchronised and a cache has one launch at a time)
      CUDA_TRY(cudaMemsetAsync(c->base + c->lay.app_done, 0,
                               size_t(c->cfg.n_layers) * c->cfg.max_requests * c->cfg.n_kv_heads * 8, s));
      CUDA_TRY(cudaMemsetAsync(c->base + c->lay.counters, 0, size_t(c->cfg.max_requests) * c->cfg.n_kv_heads * 4, s));
    }
    CUDA_TRY(cudaStreamSynchronize(s));
    if (f & OSCAR_FLAG_TIMEOUT) return fail(OSCAR_ERR_TIMEOUT, "device flags 0x%x: a bounded wait gave up", f);
    return fail(OSCAR_ERR_BAD_PAGE, "device flags 0x%x: an out-of-range page or slot was skipped", f);
  }
  return OSCAR_OK;
}

}  // extern "C"
