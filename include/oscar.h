/*
 * oscar.h -- C ABI of a GB300 (sm_103a) library for the hot path of OSCAR-style 2-bit
 * KV-cache serving: quantize-on-append into a mixed-precision paged cache, and fused
 * split-K decode attention over it, plus an uncompressed BF16 paged cache used as the
 * comparison.
 *
 * The method: "기술 요약: OSCAR - 2 비트 KV 캐시 양자화를 위한 오프라인 스펙트럴 공분산
 * 인지 회전" (gist.science technical summary of OSCAR), referred to below as [OSCAR].
 *   [OSCAR] §2.2-A.3  composite rotations R_K = U_Q H_Had P_br, R_V = U_S H_Had P_br;
 *   [OSCAR] §2.2-A.4  per-layer clip thresholds on rotated activations;
 *   [OSCAR] §2.2-B    paged KV cache: sink (initial) and recent tokens in BF16, the
 *                     history in INT2 after the fixed rotation and clipping; a fused
 *                     kernel that unpacks, dequantises, inverse-rotates and attends over
 *                     the INT2 history, compatible with paged attention and prefix caching.
 * The tilnote.io note on OSCAR restates the same layout (sink and recent tokens BF16,
 * long history INT2, paged KV).
 *
 * Conventions (every call):
 *   - Plain C types only.  `stream` is a cudaStream_t passed as void* (NULL = legacy
 *     default stream).  Device pointers are marked [dev], host pointers [host].
 *   - The caller owns all memory.  The cache lives in one caller-allocated device block;
 *     the library sub-allocates it and never calls cudaMalloc after creation.  Decode
 *     scratch is a caller-provided device workspace.
 *   - Launching calls are asynchronous on `stream`.  Host-side validation happens before
 *     any launch and returns a status; nothing is launched on error.
 *   - Device-side faults never trap: a kernel that meets a page id or slot out of range
 *     skips that access and sets a bit in a device status word (oscar_get_status).
 *   - No C++ exception crosses this ABI.  oscar_last_error() gives a thread-local text.
 *   - A cache is not thread-safe; at most one append or decode of a cache may be in
 *     flight on the GPU at a time (they share plan buffers and merge counters).
 *
 * Stored format (bit-exact contract, identical for every layer):
 *   head_dim d = 128.  Rotated value of a token x: r = bf16_rne(R^T x), where
 *   r_j = bf16(acc_j) with acc_j = +0 then acc_j = fmaf(R[i][j], x_i, acc_j) for
 *   i = 0..127 ascending (fp32, no contraction changes).  R is row-major R[i][j].
 *   Per request and layer: positions [0, min(L, S)) are BF16 sinks (r); positions
 *   [S, H) are INT2 history; positions [H, L) are BF16 recent tokens (r) in ring slot
 *   p % W.  H starts at S; after an append that brings L to L', H' = max(H, L' - W).
 *   INT2 of a token: x = fmaxf(fminf(r, c), -c) with the (layer, kv-head, K|V) clip c;
 *   per group of `group` consecutive channels s = bf16((max x - min x) / 3.0f),
 *   z = bf16(min x); code = 0 if s == 0 else fminf(fmaxf(rintf((x - z) / s), 0), 3);
 *   dequantised value fmaf(code, s, z).  A 32-byte token row holds channel
 *   c = 16 f + 2 w + h at bit 32 w + 16 h + 2 f (word w little-endian, half h, field f).
 *
 * Device pools (byte offsets are exposed through oscar_cache_layout for tests):
 *   codes : [layer][phys_page][kv_head][K|V][64 tokens][32 B]   (token-major rows)
 *           format OSCAR_FORMAT_INT2_CM: the K block as above; the V block (2048 B) is
 *           channel-major: 32-bit word 128 b + c holds channel c of the page's tokens
 *           16 b .. 16 b + 15, token 16 b + 8 h + f at bit 16 h + 2 f (b 0..3, h 0..1,
 *           f 0..7).  Codes, scale and zero are the same numbers as in OSCAR_FORMAT_INT2.
 *   sz    : [layer][phys_page][kv_head][K|V][64 tokens][d/group][scale, zero] bf16
 *   sink  : [request_slot][layer][kv_head][K|V][S][d] bf16
 *   ring  : [request_slot][layer][kv_head][K|V][W][d] bf16
 *   bf16 pages (format OSCAR_FORMAT_BF16): [layer][phys_page][kv_head][K|V][64][d] bf16
 *   A logical page p of a request holds positions [64 p, 64 p + 64); physical page ids
 *   come from the request's page table and are shared by all layers, K and V.  INT2
 *   slots of positions outside [S, H) are never read and hold unspecified bytes.
 */
#ifndef OSCAR_H_
#define OSCAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  OSCAR_OK = 0,
  OSCAR_ERR_INVALID_ARG = 1,  /* a size, index or pointer is out of the documented range */
  OSCAR_ERR_UNSUPPORTED = 2,  /* a shape the library has no kernel for */
  OSCAR_ERR_OUT_OF_PAGES = 3, /* the page pool cannot hold the reservation; nothing changed */
  OSCAR_ERR_BAD_PAGE = 4,     /* device: a page-table entry or slot out of range was skipped */
  OSCAR_ERR_CUDA = 5,         /* a CUDA runtime call failed (text in oscar_last_error) */
  OSCAR_ERR_TIMEOUT = 6,      /* device: a bounded wait on a copy gave up */
  OSCAR_ERR_STATE = 7         /* call order violated (e.g. append without a reservation) */
} oscar_status;

/* Device status word bits (oscar_get_status). */
#define OSCAR_FLAG_BAD_PAGE 0x1u
#define OSCAR_FLAG_TIMEOUT 0x2u
#define OSCAR_FLAG_BAD_SLOT 0x4u

/* OSCAR_FORMAT_INT2: INT2 history, token-major pages, decoded with warp-level MMAs; the
 * step's append can run inside the decode launch.  OSCAR_FORMAT_INT2_CM: the same stored
 * numbers with channel-major value pages, decoded on the tcgen05 tensor cores with the
 * code operands in tensor memory (GQA 4 or 8 at group 128, GQA 4 at group 32); the append
 * always runs as its own launch.  OSCAR_FORMAT_BF16: the uncompressed comparison cache.
 * OSCAR_FORMAT_INT4: every token in 4-bit pages, with no rotation, sinks or recent window
 * (oscar_int4_append below has its rows). */
typedef enum {
  OSCAR_FORMAT_INT2 = 0,
  OSCAR_FORMAT_BF16 = 1,
  OSCAR_FORMAT_INT2_CM = 2,
  OSCAR_FORMAT_INT4 = 4
} oscar_format;

typedef struct {
  int format;                /* oscar_format */
  int head_dim;              /* must be 128 */
  int n_q_heads;             /* H_q */
  int n_kv_heads;            /* H_kv; H_q / H_kv must be 4 or 8 */
  int group;                 /* INT2 and INT4 quantisation group along head_dim: 32 or 128 */
  int page;                  /* tokens per page: must be 64 */
  int n_sink;                /* S, 0..64 (INT2 format; BF16 and INT4 ignore it) */
  int window;                /* W, 0..1024 and a multiple of 16 (INT2 format) */
  int n_layers;              /* >= 1 */
  int max_requests;          /* request slots */
  int max_pages;             /* physical pages in the pool (shared by all layers) */
  int max_pages_per_request; /* page-table row length: max context = 64 * this */
} oscar_config;

typedef struct oscar_cache oscar_cache;

/* Byte offsets of the pools inside the device block, and their strides (for tests and
 * debugging dumps).  All offsets are multiples of 256. */
typedef struct {
  size_t codes, sz, sink, ring, bf16_pages;          /* pool offsets (0 if absent) */
  size_t codes_page_bytes, sz_page_bytes;            /* per (layer, page, kv-head), K then V */
  size_t bf16_page_bytes;                            /* per (layer, page, kv-head), K then V */
  size_t sink_bytes_per_head, ring_bytes_per_head;   /* per (slot, layer, kv-head), K then V */
  size_t page_table;                                 /* int32 [max_requests][max_pages_per_request] */
  size_t total;
} oscar_layout;

/* Device bytes a cache of this configuration needs (0 if the configuration is invalid). */
size_t oscar_cache_device_bytes(const oscar_config* cfg);

/* Create a cache inside `device_mem` [dev] of `bytes` (>= oscar_cache_device_bytes).
 * Zeroes the control words with cudaMemset (synchronous).  *out receives the handle. */
oscar_status oscar_cache_create(const oscar_config* cfg, void* device_mem, size_t bytes, oscar_cache** out);
void oscar_cache_destroy(oscar_cache* cache);
oscar_status oscar_cache_layout(const oscar_cache* cache, oscar_layout* out);

/* Rotation and clip inputs of one layer ([OSCAR] §2.2-A.3, A.4), produced offline:
 * R_K, R_V [host] fp32 [H_kv][d][d] row-major (orthogonal), clip_K, clip_V [host] fp32
 * [H_kv] (> 0, +inf allowed).  Copied to the device on `stream` before return.
 * Only the INT2 format uses them. */
oscar_status oscar_set_layer_params(oscar_cache* cache, int layer, const float* R_K, const float* R_V,
                                    const float* clip_K, const float* clip_V, void* stream);

/* Request slots.  alloc gives an empty request (L = 0).  free drops its page references. */
oscar_status oscar_request_alloc(oscar_cache* cache, int* slot);
oscar_status oscar_request_free(oscar_cache* cache, int slot);
/* Free physical pages of the pool and free request slots (host view; a page shared by
 * several requests is free once the last of them is freed).  Either pointer may be NULL. */
oscar_status oscar_cache_stats(const oscar_cache* cache, int* free_pages, int* free_slots);
/* Host view of a request: length L, history end H (INT2 format), pages mapped. */
oscar_status oscar_request_info(const oscar_cache* cache, int slot, int* length, int* history_end, int* n_pages);
/* Host copy of a request's page-table row (n entries). */
oscar_status oscar_request_pages(const oscar_cache* cache, int slot, int* pages, int n);

/* Prefix caching ([OSCAR] §2.2-B): the empty request `dst` takes the first `n_tokens`
 * tokens of `src` by sharing src's physical pages (reference counted), and copies src's
 * sink tokens for every layer on `stream`.  n_tokens must be a positive multiple of 64
 * and, in the INT2 format, at most src's history end H (those pages are never rewritten,
 * so no copy-on-write is needed); in the BF16 format at most 64 * floor(L_src / 64).
 * Afterwards dst has L = H = n_tokens. */
oscar_status oscar_request_share_prefix(oscar_cache* cache, int dst, int src, int n_tokens, void* stream);

/* Append, step 1 (host): reserve pages for `n_new[i]` more tokens of request `slots[i]`
 * [host arrays of n_req distinct slots], upload the changed page-table rows and the append
 * plan on `stream`.  The plan serves every layer until oscar_commit_append.  On
 * OSCAR_ERR_OUT_OF_PAGES nothing is reserved. */
oscar_status oscar_reserve(oscar_cache* cache, const int* slots, const int* n_new, int n_req, void* stream);

/* Append, step 2 (device, per layer): quantize-on-append of the reserved tokens of one
 * layer.  k_new, v_new [dev] bf16 [sum n_new][H_kv][d], requests in reservation order.
 * Rotates by R^T, routes each position to its sink, ring slot or INT2 row, evicts ring
 * tokens that leave the recent window into INT2, clips, quantises and packs. */
oscar_status oscar_quantize_append(oscar_cache* cache, int layer, const void* k_new, const void* v_new, void* stream);

/* Append, step 3 (host): the reserved tokens count as held (L, H advance). */
oscar_status oscar_commit_append(oscar_cache* cache);

/* Decode, step 1 (host): plan split-K decode of requests `slots` [host, n_req distinct]
 * at their current lengths, upload on `stream`.  The plan serves every layer until the
 * next plan or append commit.  max_split_pages > 0 caps the INT2 pages per work item
 * (0 = automatic, balanced over the SMs). */
oscar_status oscar_plan_decode(oscar_cache* cache, const int* slots, int n_req, int max_split_pages, void* stream);

/* oscar_plan_decode with plan flags (OSCAR_PLAN_*, or-ed).  OSCAR_PLAN_NARROW plans for
 * the 8-warp CTA shape (two CTAs per SM at GQA 4), which the automatic choice takes only
 * for steps larger than one wave of 16-warp CTAs; results are the same either way. */
#define OSCAR_PLAN_NARROW 0x1u
/* OSCAR_PLAN_FOLDED_ROTATIONS (INT2 formats): the model folds the rotations into its
 * projections ([OSCAR] §2.2-A.3 and B: R_K into the query projection, R_V into the output
 * projection), so the decode calls of this plan take q already rotated, q~ = R_K^T q (bf16,
 * same layout as q), and write o~, the output in the rotated basis (o = R_V o~ is left to
 * the model).  The stored cache is the same; only the two matrix-vector products at the
 * ends of the decode are skipped. */
#define OSCAR_PLAN_FOLDED_ROTATIONS 0x2u
/* OSCAR_PLAN_SHARED_PREFIX (format OSCAR_FORMAT_BF16): requests of the plan whose page-table
 * rows begin with the same pages (oscar_request_share_prefix, at any depth: a prefix under
 * several longer ones) have those pages attended once for all of them, as one more launch
 * of oscar_bf16_decode_attention before the decode's own; each request's further pages and
 * the merge are as without the flag.  Results are those of the plan without it, up to the
 * rounding of the sums (and values below 2^78: the shared sums carry factors up to 2^32).  Where sharing would save too few reads to pay for the launch, the
 * plan goes without it; with OSCAR_PLAN_SHARED_ALWAYS (only together with it) it never does.
 * A decode captured under a plan with the flag may be replayed under any later plan; one
 * captured without it may not be replayed under a plan with shared runs. */
#define OSCAR_PLAN_SHARED_PREFIX 0x4u
#define OSCAR_PLAN_SHARED_ALWAYS 0x8u
oscar_status oscar_plan_decode_ex(oscar_cache* cache, const int* slots, int n_req, int max_split_pages, uint32_t flags,
                                  void* stream);

/* Decode workspace bytes for the current plan (0 without a plan). */
size_t oscar_decode_workspace_bytes(const oscar_cache* cache);

/* Decode workspace bytes that cover every plan of this cache (0 for NULL).  A launch
 * captured into a CUDA graph keeps the workspace pointer it was given, and a replay after
 * a later plan writes that plan's partial results through it: a workspace of this size
 * keeps such replays in bounds whatever the later plans are. */
size_t oscar_decode_workspace_max_bytes(const oscar_cache* cache);

/* Number of split-K work items of the current plan, and of them BF16 (sink/ring) items. */
oscar_status oscar_plan_info(const oscar_cache* cache, int* n_items, int* n_bf16_items, int* max_item_pages);

/* Of a plan with OSCAR_PLAN_SHARED_PREFIX: the shared launch's work items, and the pages of
 * a kv-head that it attends once for several requests (0 and 0 where it goes without). */
oscar_status oscar_plan_shared_info(const oscar_cache* cache, int* n_items, int* n_pages);

/* Decode, step 2 (device, per layer): fused decode attention over the mixed-precision
 * cache ([OSCAR] §2.2-B): q~ = R_K^T q per query head; scores q~.k / sqrt(d) in the
 * rotated basis over BF16 sinks, the BF16 recent window and the INT2 history (2-bit codes
 * unpacked and dequantised in registers); online softmax merged across splits;
 * out = R_V o~ (inverse rotation, once per head).
 * q [dev] bf16 [n_req][H_q][d] in plan order; out [dev] bf16 same shape; out_f32 [dev]
 * nullable fp32 copy of the output before bf16 rounding; workspace [dev] of ws_bytes.
 * A request with L = 0 gets zeros. */
oscar_status oscar_decode_attention(oscar_cache* cache, int layer, const void* q, void* out, void* workspace,
                                    size_t ws_bytes, float* out_f32, void* stream);

/* Quantize-append and decode in one launch (device, per layer): oscar_quantize_append of
 * the pending reservation's tokens for `layer` (same k_new / v_new layout) followed by
 * oscar_decode_attention of q over the cache that includes them, as a single kernel: the
 * append tasks run first and each decode work item waits only for the append tasks of
 * its own (request, kv-head) before it reads a ring or sink row or an INT2 page that the
 * append writes ([OSCAR] §2.2-B: quantize on append, then fused decode over the
 * mixed-precision cache; one launch per layer is this library's scheduling, not the
 * paper's).  When the reservation has more append work than one wave of decode CTAs
 * holds (long chunks, many requests), the call launches the append kernel and then the
 * decode kernel instead (oscar_last_launch_count tells which).  Requires a reservation
 * and a plan made after it that lists every reserved slot (OSCAR_ERR_STATE otherwise);
 * oscar_commit_append afterwards as usual.  Results are those of the two separate calls.
 * Waits are bounded: a wait that runs out sets OSCAR_FLAG_TIMEOUT. */
oscar_status oscar_append_decode_attention(oscar_cache* cache, int layer, const void* k_new, const void* v_new,
                                           const void* q, void* out, void* workspace, size_t ws_bytes,
                                           float* out_f32, void* stream);

/* Uncompressed comparison path (format OSCAR_FORMAT_BF16, same page tables and calls
 * for requests, reserve, commit and plan): append writes plain bf16 K and V rows into
 * pages; decode is softmax(q K^T / sqrt(d)) V over all L tokens, with no rotation. */
oscar_status oscar_bf16_append(oscar_cache* cache, int layer, const void* k_new, const void* v_new, void* stream);
oscar_status oscar_bf16_decode_attention(oscar_cache* cache, int layer, const void* q, void* out, void* workspace,
                                         size_t ws_bytes, float* out_f32, void* stream);

/* Appends with rotary positions (formats OSCAR_FORMAT_BF16 and OSCAR_FORMAT_INT4), in the place
 * of oscar_rope and the format's append: the reservation's new keys are turned by their
 * positions on the way into the pages, its values go in as they are, and the queries of the same
 * tokens, if given, are turned into q->out; one launch.  What the cache holds and q->out are
 * those of oscar_rope (keys rounded to bf16) and the append after it, bit for bit.
 * k, v: the rows of the reservation [sum n_new][H_kv][d] bf16, any row and head strides >= 0 in
 * elements, channels contiguous (a fused projection's slices go in as they are).  q NULL, or
 * the queries of the same rows in bf16, as a tensor of oscar_rope (q->out may be q->in; any other
 * overlap of q->out with q->in, k, v or positions is refused).  steps, rotary_dim (<= 128), magnitude: as for
 * oscar_rope (steps may be read before the kernel in front of this one has ended); flags: OSCAR_ROPE_INTERLEAVED, OSCAR_ROPE_POSITIONS64.  positions [dev]: int32
 * (int64 with the flag), one a row, or NULL: a token's place in its request.  The current device
 * must be the cache's. */
typedef struct {
  const void* in;
  long long row, head;
} oscar_rows;
struct oscar_rope_tensor_s;
oscar_status oscar_append_rotated(oscar_cache* cache, int layer, const uint64_t* steps, int rotary_dim, float magnitude,
                                  uint32_t flags, const void* positions, const struct oscar_rope_tensor_s* q,
                                  const oscar_rows* k, const oscar_rows* v, void* stream);

/* 4-bit pages (format OSCAR_FORMAT_INT4): every token of a request, quantised as it is appended.
 * Per token, K or V, and group of `group` consecutive channels, all in fp32: s = bf16((max x -
 * min x) / 15), z = bf16(min x); code = 0 if s == 0 else fminf(fmaxf(rintf((x - z) / s), 0), 15);
 * value fmaf(code, s, z).  Values past +-2^126 and infinities count as +-2^126, NaN as 2^126.
 * Pool (at oscar_layout.codes; codes_page_bytes a kv-head): [layer][phys_page][kv_head][2 halves of
 * 32 tokens], a half page being K codes [32][64 B], V codes [32][64 B], K [32][d/group][scale,
 * zero] bf16, V the same.  Channel c of a half page's token t is bits 4 (c % 8) .. + 3 of the
 * little-endian word at byte 64 t + 16 ((c / 8 % 4) ^ (t / 2 % 4)) + 4 (c / 32) of its codes.
 * Requests, reservations, plans and prefix sharing are as for the BF16 format.
 * oscar_int4_append: step 2 of an append, arguments as oscar_quantize_append.
 * oscar_int4_read: the values of tokens [begin, end) of a request (a pending reservation's among
 * them once they are appended) into k_out, v_out [dev] [end - begin][H_kv][d], contiguous, in
 * dtype OSCAR_DTYPE_BF16 (one more rounding) or OSCAR_DTYPE_F32, 16-byte aligned, not overlapping.
 * oscar_int4_decode_attention: softmax(q K^T / sqrt(d)) V over the values of all L tokens, as
 * oscar_bf16_decode_attention takes it (values below 2^100).  Weights enter the product with the
 * codes times their scale, each rounded to 11 bits, or by 2^-31 of a head's largest such product
 * in the item where it is far below it.  The current device must be the cache's. */
oscar_status oscar_int4_append(oscar_cache* cache, int layer, const void* k_new, const void* v_new, void* stream);
oscar_status oscar_int4_read(oscar_cache* cache, int layer, int slot, int begin, int end, void* k_out, void* v_out,
                             int dtype, void* stream);
oscar_status oscar_int4_decode_attention(oscar_cache* cache, int layer, const void* q, void* out, void* workspace,
                                         size_t ws_bytes, float* out_f32, void* stream);

/* Attention within a sliding window and over the first tokens (format OSCAR_FORMAT_BF16), for one
 * or many of each request's last tokens: decode steps, prompts and chunks of them, drafted tokens.
 * The query at position p (its token's place in the request) attends the tokens t <= p with
 * t < n_sink or t > p - window; window 0: all t <= p.
 *
 * oscar_plan_window (host): the queries are the last n_queries[i] tokens (0 .. L; NULL: one each)
 * of request slots[i] [host, n_req distinct], a pending reservation's tokens counted; uploads the
 * plan on `stream`.  It stands beside the decode plan, so that layers with and without a window
 * take turns, serves every layer, and ends as that one does (the next window plan, reservation
 * or append commit).  oscar_plan_window_info: work items of the single queries, those of the others
 * (tiles of 256 / G queries and a kv-head, or parts of them), and how many tiles were cut.
 * oscar_window_attention (device, per layer): out = softmax(q K^T / sqrt(d)) V over what each query
 * attends.  q, out [dev] bf16 [sum n_queries][H_q][d], requests in plan order, out_f32 nullable
 * (before the rounding); all 16-byte aligned.  workspace [dev], 256-byte aligned, of
 * oscar_window_workspace_bytes for the current plan, _max_bytes for every plan (as captured
 * launches need it, which may be replayed under any later plan; q and out must then hold that
 * plan's queries; a captured call holds the kernels of single and of several queries, whatever its
 * own plan).  Values of tokens that no
 * query attends are not used, and infinities and NaN reach only queries that attend them: a query
 * or key of NaN, or a score of +inf, makes the whole output NaN, a value its channel NaN or
 * infinite (as in every decode of this library).  With
 * several queries a request, weights enter the product with the values as bf16; values below 2^78.
 * The current device must be the cache's. */
oscar_status oscar_plan_window(oscar_cache* cache, const int* slots, const int* n_queries, int n_req, int n_sink,
                               int window, void* stream);
oscar_status oscar_plan_window_info(const oscar_cache* cache, int* n_row_items, int* n_tiles, int* n_cut);
size_t oscar_window_workspace_bytes(const oscar_cache* cache);
size_t oscar_window_workspace_max_bytes(const oscar_cache* cache);
oscar_status oscar_window_attention(oscar_cache* cache, int layer, const void* q, void* out, void* workspace,
                                    size_t ws_bytes, float* out_f32, void* stream);

/* Accumulated attention weights (format OSCAR_FORMAT_BF16).  A row of weights is
 * oscar_weights_stride tokens, 64 * min(max_pages_per_request, max_pages); a buffer of one
 * layer is fp32 [max_requests][H_kv][stride] [dev], indexed by request slot and position and
 * owned by the caller, who zeroes a slot's rows when a request starts in it.
 *
 * oscar_bf16_decode_weights is oscar_bf16_decode_attention (same plan, q, out and out_f32)
 * that also writes weights_out[slot][kv-head][t] = weights_in[slot][kv-head][t] + sum over
 * the kv-head's query heads of softmax(q K^T / sqrt(d))[t] for every token t < L of the
 * planned requests; weights_in NULL counts as zeros and may be weights_out (it must not
 * overlap it otherwise).  Other entries of weights_out stay as they are.  The workspace
 * (oscar_decode_weights_workspace_bytes for the current plan, _max_bytes for every plan, as a
 * captured launch needs it) also holds the scores, 4 bytes a query head and token of the
 * plan's requests.  Two launches.  Not with a plan of OSCAR_PLAN_SHARED_PREFIX
 * (OSCAR_ERR_STATE). */
int oscar_weights_stride(const oscar_cache* cache);
size_t oscar_decode_weights_workspace_bytes(const oscar_cache* cache);
size_t oscar_decode_weights_workspace_max_bytes(const oscar_cache* cache);
oscar_status oscar_bf16_decode_weights(oscar_cache* cache, int layer, const void* q, void* out, const float* weights_in,
                                       float* weights_out, void* workspace, size_t ws_bytes, float* out_f32,
                                       void* stream);

/* Eviction by accumulated attention weight (format OSCAR_FORMAT_BF16): of a request's L
 * tokens `keep` stay, per layer and kv-head: the first n_sink, the last n_recent, and of the
 * others those with the greatest weight (equal weights: the lowest positions; -0 equals 0;
 * NaN comes last).  They move, in the order of their positions, into new pages (pages shared
 * with other requests are never rewritten), and the request's length becomes keep.  A
 * request with L <= keep keeps everything where it is.
 *
 * Step 1 (host): oscar_evict_begin takes the new pages for `keep[i]` tokens of request
 * `slots[i]` [host arrays of n_req distinct slots] and uploads the plan on `stream`, which
 * serves every layer until the commit.  keep[i] >= n_sink + n_recent where tokens go.  On
 * OSCAR_ERR_OUT_OF_PAGES nothing is taken.  Until the commit (or cancel), reserving, freeing
 * requests and sharing prefixes is refused; decodes still see the old pages.
 * Step 2 (device, per layer): oscar_evict copies the layer's kept rows.  weights as above,
 * 16-byte aligned; weights_out, same shape: the rows of the listed slots become the kept
 * tokens' weights, then zeros to the end of the row; kept int32, same shape: the positions
 * (before the eviction) of the kept tokens, entries from keep on stay as they are.  The
 * three must not overlap.  Every layer goes before the commit, in any order.
 * Step 3 (host): oscar_evict_commit makes the new pages the requests' (uploads their
 * page-table rows on `stream`) and frees the old ones; plan again before decoding.
 * oscar_evict_cancel gives the new pages back instead.
 * oscar_evict_pages: between begin and commit, host copy of up to n of the pages that slot
 * will have, their number in *n_pages (nullable). */
oscar_status oscar_evict_begin(oscar_cache* cache, const int* slots, const int* keep, int n_req, int n_sink,
                               int n_recent, void* stream);
oscar_status oscar_evict(oscar_cache* cache, int layer, const float* weights, float* weights_out, int* kept,
                         void* stream);
oscar_status oscar_evict_pages(const oscar_cache* cache, int slot, int* pages, int n, int* n_pages);
oscar_status oscar_evict_commit(oscar_cache* cache, void* stream);
oscar_status oscar_evict_cancel(oscar_cache* cache);

/* oscar_decode_attention without a caller workspace.  The paper has no counterpart:
 * this exists for callers that cannot allocate device memory themselves, for example a
 * plugin whose host framework owns every device allocation and gives it none, or a
 * serving loop that must not allocate once it is running, and so cannot supply the
 * decode workspace.  The scratch is instead a fixed 8 MiB array inside the library
 * (static device memory, held on every GPU that loads the library until exit).
 *   - Same semantics, inputs and outputs as oscar_decode_attention (q, out, out_f32).
 *   - Returns OSCAR_ERR_INVALID_ARG, launching nothing, when the current plan needs more
 *     than 8 MiB (oscar_decode_workspace_bytes tells the need).
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *   - The current device must be the cache's device (the one current at
 *     oscar_cache_create): the array's address is looked up on the current device, on
 *     every call; OSCAR_ERR_INVALID_ARG otherwise.  The first call on a device also loads
 *     the library's device code there if nothing has yet; make that first call before any
 *     stream capture.
 *   - Every call, on every cache and stream, shares the one array and leaves its
 *     contents behind; nothing in it needs to start at zero.  Calls that overlap on the
 *     GPU race on it: order them on one stream or serialise them. */
oscar_status oscar_decode_attention_noalloc(oscar_cache* cache, int layer, const void* q, void* out, float* out_f32,
                                            void* stream);

/* Offline calibration of one layer on the GPU ([OSCAR] §2.2-A.1 to A.4), in fp64:
 *   A.1  C_Q = (1/(G N)) sum over tokens and the G query heads of each kv-head of q^T q;
 *        C_S = (1/(G N)) sum_h O_h^T O_h, O_h = causal softmax(Q_h K^T / sqrt(d)) V
 *        (the score-aware value target V^T S^T S V / N);
 *   A.2  eigenbases by cyclic Jacobi: eigenvalues descending, each eigenvector's first
 *        largest-magnitude entry positive;
 *   A.3  R_K = U_Q H_Had P_br, R_V = U_S H_Had P_br (H_Had the Sylvester matrix / sqrt(d),
 *        P_br sending e_j to e_rev(j)), rounded to fp32;
 *   A.4  clip = the clip_rank-th smallest of |x R| over the N tokens x d channels of each
 *        kv-head's keys (values), with R as rounded; a nearest-rank percentile p is
 *        clip_rank = ceil(p / 100 * N * d).
 * rotation OSCAR_ROTATION_HADAMARD skips A.1 and A.2 (U = I: the Hadamard-only rotation).
 * q [dev] bf16 [N][H_q][d], k and v [dev] bf16 [N][H_kv][d] (d = 128); outputs [dev]:
 * R_K, R_V fp32 [H_kv][d][d] row-major (the inputs of oscar_set_layer_params), clip_K,
 * clip_V fp32 [H_kv]; covariances [dev] nullable fp64 [2 H_kv][d][d] (C_Q of every
 * kv-head, then C_S; untouched in the Hadamard-only mode).  workspace [dev], 256-byte
 * aligned, of oscar_calibration_workspace_bytes (0 for a bad shape).  Asynchronous on
 * `stream`. */
#define OSCAR_ROTATION_OSCAR 0
#define OSCAR_ROTATION_HADAMARD 1
size_t oscar_calibration_workspace_bytes(int n_tokens, int n_q_heads, int n_kv_heads);
oscar_status oscar_calibrate_layer(const void* q, const void* k, const void* v, int n_tokens, int n_q_heads,
                                   int n_kv_heads, long long clip_rank, int rotation, float* R_K, float* R_V,
                                   float* clip_K, float* clip_V, double* covariances, void* workspace,
                                   size_t ws_bytes, void* stream);

/* Rotary positions (RoPE) on queries and keys, before the append and the decode.  Pair i of
 * a row at position p turns by the angle p f_i, (a, b) -> magnitude (a cos - b sin, b cos +
 * a sin); channels from rotary_dim on pass through.  The pairs are channels (i, i +
 * rotary_dim / 2), or (2 i, 2 i + 1) with OSCAR_ROPE_INTERLEAVED.  With
 * OSCAR_ROPE_TRANSPOSE the angles are negated: the transposed map, which takes the
 * gradient of the outputs to that of the inputs.
 *
 * oscar_rope_steps computes the table of a configuration [host]: steps [rotary_dim / 2],
 * entry i = f_i / (2 pi) turns a position as a 64-bit fixed-point fraction of a turn
 * (p * steps[i] modulo 2^64 is the phase: every 64-bit position keeps its precision), and
 * *magnitude.  f_i = base^(-2 i / rotary_dim), scaled for contexts longer than the model's
 * original_context by
 *   OSCAR_ROPE_LINEAR  f_i / factor;
 *   OSCAR_ROPE_BANDS   by the turns n_i = original_context f_i / (2 pi): f_i where n_i >= high,
 *                      f_i / factor where n_i <= low, linear in n_i between (low < high);
 *   OSCAR_ROPE_YARN    by the pair's index (YaRN): with x(n) = rotary_dim ln(original_context /
 *                      (2 pi n)) / (2 ln base), f_i up to floor(x(high)), f_i / factor from
 *                      ceil(x(low)), linear in i between (both held to [0, rotary_dim - 1]);
 *                      magnitude = 0.1 ln(factor) + 1.
 * rotary_dim even in [2, 512], base > 1, factor > 0 (>= 1 for YARN), 0 < low < high. */
#define OSCAR_ROPE_UNSCALED 0
#define OSCAR_ROPE_LINEAR 1
#define OSCAR_ROPE_BANDS 2
#define OSCAR_ROPE_YARN 3
typedef struct {
  int rotary_dim;
  int scaling; /* OSCAR_ROPE_UNSCALED, _LINEAR, _BANDS or _YARN; the fields below as it needs them */
  double base, factor, low, high, original_context;
} oscar_rope_config;
oscar_status oscar_rope_steps(const oscar_rope_config* cfg, uint64_t* steps, float* magnitude);

/* One tensor of a call: rows x n_heads x head_dim channels [dev], channels contiguous, the
 * strides in elements (inputs: any >= 0; outputs: rows and heads that do not overlap).
 * Elementwise: out may be in, with the same strides; any other overlap of a call's outputs
 * with its inputs or outputs is not allowed. */
typedef struct oscar_rope_tensor_s {
  const void* in;
  void* out;
  int n_heads;
  long long in_row, in_head, out_row, out_head;
} oscar_rope_tensor;

/* Turn tensors[0 .. n_tensors - 1] (1 or 2: queries and keys of the same rows and dtype) by
 * the table `steps` [dev] uint64 [rotary_dim / 2] and `magnitude`.  positions [dev]: int32
 * [n_rows], or int64 with OSCAR_ROPE_POSITIONS64; any values, in any order.  head_dim in
 * [rotary_dim, 512].  Products and sums in fp32, one rounding to dtype.  n_rows = 0 launches
 * nothing.  Everything must belong to the current device. */
#define OSCAR_DTYPE_BF16 0
#define OSCAR_DTYPE_F16 1
#define OSCAR_DTYPE_F32 2
#define OSCAR_ROPE_INTERLEAVED 0x1u
#define OSCAR_ROPE_TRANSPOSE 0x2u
#define OSCAR_ROPE_POSITIONS64 0x4u
oscar_status oscar_rope(const oscar_rope_tensor* tensors, int n_tensors, const uint64_t* steps, int head_dim,
                        int rotary_dim, float magnitude, int dtype, uint32_t flags, const void* positions,
                        long long n_rows, void* stream);

/* Bounded waits: a work item of oscar_append_decode_attention that waits for the append
 * tasks it depends on gives up after `counter_polls` polls of their counter (each poll
 * sleeps about 0.1 us; 0 restores the default of 2^22 polls, about a second), sets
 * OSCAR_FLAG_TIMEOUT and carries on.  Applies to launches made after the call. */
oscar_status oscar_set_wait_limit(oscar_cache* cache, uint32_t counter_polls);

/* Host-side fault injection, for tests of the failure paths (nothing faults on the GPU).
 * OSCAR_FAULT_LOST_APPEND_SIGNAL: the next decode plan made while a reservation is pending
 * expects one more append signal for its first appending request than the append tasks
 * send, so that request's waits in oscar_append_decode_attention run out (a signal that
 * never arrives); the kernel returns with OSCAR_FLAG_TIMEOUT set.  One-shot. */
#define OSCAR_FAULT_LOST_APPEND_SIGNAL 0x1u
oscar_status oscar_inject_fault(oscar_cache* cache, uint32_t faults);

/* Synchronises `stream`, returns the device status word in *flags (OSCAR_FLAG_*) and
 * clears it.  Returns OSCAR_ERR_BAD_PAGE / OSCAR_ERR_TIMEOUT if a flag was set.  After a
 * timeout it also resets the cache's append-dependency and merge counters, so the next
 * step starts from a consistent state. */
oscar_status oscar_get_status(oscar_cache* cache, void* stream, uint32_t* flags);

/* Text of the last error on this thread ("" if none). */
const char* oscar_last_error(void);

/* Number of kernels the last launching call on this thread put on its stream. */
int oscar_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* OSCAR_H_ */
