"""Throughput-mode serving over one cache: continuous batching at a fixed HBM budget.

The OSCAR technical summary (gist.science) reports, for large batches, up to 7x the
throughput of BF16 under the same memory budget (section 4), and runs the INT2 kernel
inside a serving framework with paged KV and prefix caching (section 2.2-B).  This module
is the analogue for this library: one loop that admits requests while the pool's pages
allow, prefills their prompts (mapping a group's shared prefix from a prefix holder
instead of recomputing it: a prefix-cache hit), decodes one token per running request per
step through the library's calls, and frees a request's pages when it finishes.  The same
loop runs the INT2 cache, the 4-bit cache and the uncompressed BF16 cache, each sized to the
same byte budget; the number of requests that fit at once is what differs.

Around the attention the loop can run what a model's serving step runs: rotary positions on
the queries and the new keys (`rotary`; on the BF16 and 4-bit caches the keys are turned as they
are appended); the BF16 cache's decode with shared prefixes attended once (`share_decode`) or
within a sliding window and the first tokens (`window`, `window_sinks`); and, on the BF16 cache, eviction of the tokens with the least
accumulated attention weight once a request holds more than `evict_above` of them, down to
`evict_to`, so that a long request stays within a bounded number of pages (the weights that
this keeps count against the budget: a row of the longest request for every slot and layer,
so `max_requests` and `max_len` decide what they take).

Scheduling: first come, first served.  A request is admitted when a slot is free and the
free pages cover its final length on top of what the running requests will still need
(so a running request never runs out of pages).  A prefix holder is a slot that holds
one group's prefix tokens and stays resident once made.

Tokens: K, V and q rows come from seeded pools on the device, indexed by (layer, stream,
position), where the stream is the group's prefix below the prefix length and the
request's own beyond it, so shared prefixes really are the same tokens and any token can
be rebuilt on the host (the tests' oracle does).  The model that would produce them is
out of scope: these are the cache's inputs.
"""
from __future__ import annotations

import dataclasses
import time
from typing import Callable, Optional

import torch

from . import _native as N

_INT2 = (N.OSCAR_FORMAT_INT2, N.OSCAR_FORMAT_INT2_CM)  # both INT2 page formats
from . import workloads as wl
from .cache import KVCache


@dataclasses.dataclass
class Request:
    rid: int
    prompt: int  # context tokens before generation
    gen: int  # tokens generated (decode steps)
    group: int = -1  # shared-prefix group, -1 = none
    slot: int = -1
    length: int = 0  # tokens held in the cache
    position: int = 0  # tokens seen: the next token's position (= length unless some were evicted)
    generated: int = 0
    shared: int = 0  # prompt tokens mapped from the group's prefix holder


def make_requests(n: int, prompt_range, gen_range, n_groups: int, seed: int):
    """n seeded requests: prompt and generation lengths uniform in the given ranges, every
    request in one of n_groups shared-prefix groups (round robin)."""
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(prompt_range[0], prompt_range[1] + 1, (n,), generator=g).tolist()
    o = torch.randint(gen_range[0], gen_range[1] + 1, (n,), generator=g).tolist()
    return [Request(rid=i, prompt=int(p[i]), gen=int(o[i]), group=(i % n_groups) if n_groups else -1)
            for i in range(n)]


class TokenSource:
    """K, V (bf16 [P, H_kv, d]) and q (bf16 [P, H_q, d]) pools; the row of (layer, stream,
    position) is pool[(A * stream + B * layer + position) mod P]."""

    A, B = 7919, 104729

    def __init__(self, w: wl.Workload, seed: int, pool_tokens: int = 8192, device="cuda"):
        self.P = pool_tokens
        self.K, self.V = wl.gen_kv(wl.scaled(w, prefix_tokens=0), seed, 0, 0, 0, pool_tokens, device=device)
        self.Q = wl.gen_q(w, seed, 0, 0, pool_tokens, device=device)
        self.device = torch.device(device)

    @staticmethod
    def stream(req: Request, position: int, prefix_tokens: int) -> int:
        if req.group >= 0 and position < prefix_tokens:
            return 1_000_000 + req.group
        return req.rid

    def rows(self, layer: int, stream: int, start: int, n: int) -> torch.Tensor:
        base = (self.A * stream + self.B * layer + start) % self.P
        return (torch.arange(n, device=self.device) + base) % self.P

    def index(self, layer: int, pieces) -> torch.Tensor:
        """Pool rows of the pieces [(stream, start, n)] concatenated."""
        parts = [self.rows(layer, s, a, n) for s, a, n in pieces if n > 0]
        if not parts:
            return torch.empty(0, dtype=torch.long, device=self.device)
        return torch.cat(parts)


def pages_needed(fmt: int, L: int, S: int, W: int) -> int:
    """Pages of a request of length L (the library's rule: INT2 pages hold history rows only)."""
    if fmt in _INT2:
        H = max(S, L - W)
        return -(-H // 64) if H > S else 0
    return -(-L // 64)


def eviction_bytes(w: wl.Workload, max_requests: int, pages: int, pages_per_request: int) -> int:
    """Device bytes that a loop with eviction keeps beside a cache of so many pages: the layers'
    weights, a layer's kept weights and positions, and the scores of the pool's tokens."""
    row = 64 * min(pages, pages_per_request)
    return 4 * ((w.n_layers + 2) * max_requests * w.n_kv_heads * row + 64 * pages * w.n_q_heads)


def cache_for_budget(w: wl.Workload, fmt: int, budget_bytes: int, max_requests: int, max_len: int, device,
                     evicts: bool = False):
    """The cache with the most pages whose device block, with what eviction keeps beside it, fits
    the budget."""
    ppr = -(-max_len // 64) + 2

    def cfg(pages):
        return N.oscar_config(fmt, w.head_dim, w.n_q_heads, w.n_kv_heads, w.group, 64, w.n_sink, w.window, w.n_layers,
                              max_requests, pages, ppr)

    def total(pages):
        return N.oscar_cache_device_bytes(cfg(pages)) + (eviction_bytes(w, max_requests, pages, ppr) if evicts else 0)

    lo, hi = 1, 1 << 24
    if total(lo) > budget_bytes:
        raise ValueError(f"a budget of {budget_bytes} bytes holds no page")
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if total(mid) <= budget_bytes:
            lo = mid
        else:
            hi = mid - 1
    return KVCache(fmt=fmt, n_q_heads=w.n_q_heads, n_kv_heads=w.n_kv_heads, group=w.group, n_sink=w.n_sink,
                   window=w.window, n_layers=w.n_layers, max_requests=max_requests, max_pages=lo,
                   max_pages_per_request=ppr, device=device)


class ServingLoop:
    """Continuous batching over one cache (INT2, INT4 or BF16) of workload shape w."""

    def __init__(self, w: wl.Workload, fmt: int, budget_bytes: int, tokens: TokenSource, layer_params=None,
                 max_requests: int = 128, max_len: int = 1 << 16, prefix_tokens: int = 0,
                 prefill_chunk: int = 16384, device="cuda", rotary=None, share_decode: bool = False,
                 evict_above: int = 0, evict_to: int = 0, n_sink: int = 4, n_recent: int = 64, window: int = 0,
                 window_sinks: int = 0):
        if (share_decode or evict_above or window) and fmt != N.OSCAR_FORMAT_BF16:
            raise ValueError("share_decode, eviction and a window need the BF16 format")
        if window < 0 or window_sinks < 0 or (window_sinks and not window):
            raise ValueError("window_sinks go with a window of at least one token")
        if window and (share_decode or evict_above):
            raise ValueError("a window excludes share_decode and eviction")
        if share_decode and evict_above:
            raise ValueError("share_decode and eviction exclude each other (the weights' decode does not share)")
        if evict_above and not (0 < evict_to <= evict_above and n_sink >= 0 and n_recent >= 0 and n_sink + n_recent <= evict_to):
            raise ValueError("eviction needs n_sink + n_recent <= evict_to <= evict_above")
        self.w, self.fmt, self.tokens = w, fmt, tokens
        self.S = w.n_sink if fmt in _INT2 else 0
        self.W = w.window if fmt in _INT2 else 0
        self.prefix = prefix_tokens
        self.prefill_chunk = prefill_chunk
        self.cache = cache_for_budget(w, fmt, budget_bytes, max_requests, max_len, device, evicts=evict_above > 0)
        if fmt in _INT2:
            RK, RV, cK, cV = layer_params
            for layer in range(w.n_layers):
                self.cache.set_layer_params(layer, RK[layer], RV[layer], cK[layer], cV[layer])
        self.rotary, self.share_decode = rotary, share_decode
        self.window, self.window_sinks = window, window_sinks
        self.evict_above, self.evict_to, self.protect = evict_above, evict_to, (n_sink, n_recent)
        if evict_above:
            self.weights = [self.cache.new_weights() for _ in range(w.n_layers)]
            self._weights_out, self._kept = self.cache.new_weights(), torch.empty(
                self.weights[0].shape, dtype=torch.int32, device=device)
        self.holders = {}  # group -> holder slot
        self.stats = dict(steps=0, generated=0, completed=0, prefill_tokens=0, shared_tokens=0, prefix_hits=0,
                          max_batch=0, batch_sum=0, decode_s=0.0, wall_s=0.0, max_pages_used=0, evictions=0)

    # ------------------------------------------------------------------ pages
    def _need(self, L: int) -> int:
        return pages_needed(self.fmt, L, self.S, self.W)

    def _shareable(self) -> int:
        """Prefix tokens a request maps from its group's holder (full pages the holder will
        never rewrite)."""
        if not self.prefix:
            return 0
        held = self.prefix if self.fmt not in _INT2 else max(self.S, self.prefix - self.W)
        return held // 64 * 64

    # ------------------------------------------------------------------ appends
    def _append(self, reqs, starts, counts):
        """Append tokens [start, start + count) of each request (as one reservation)."""
        c = self.cache
        slots = [r.slot for r in reqs]
        c.reserve(slots, counts)
        for layer in range(self.w.n_layers):
            pieces = []
            for r, a, n in zip(reqs, starts, counts):
                pieces += self._pieces(r, a, n)
            idx = self.tokens.index(layer, pieces)
            K = self.tokens.K.index_select(0, idx)
            V = self.tokens.V.index_select(0, idx)
            if self.rotary is not None:
                if layer == 0:
                    positions = torch.cat([torch.arange(a, a + n, dtype=torch.int32, device=K.device)
                                           for a, n in zip(starts, counts)])
                if self.fmt not in _INT2:
                    c.append_rotated(layer, self.rotary, K, V, positions=positions)
                    continue
                self.rotary.apply(positions, K, q_out=K)
            c.append(layer, K, V)
        c.commit()

    def _pieces(self, r: Request, a: int, n: int):
        """(stream, start, count) pieces of tokens [a, a + n) of request r."""
        out = []
        p = a
        while p < a + n:
            stop = a + n
            if r.group >= 0 and p < self.prefix:
                stop = min(stop, self.prefix)
            out.append((TokenSource.stream(r, p, self.prefix), p, stop - p))
            p = stop
        return out

    def _holder(self, group: int) -> Optional[int]:
        """The group's prefix holder slot (made on first use if the pool allows)."""
        if group in self.holders:
            return self.holders[group]
        free_pages, free_slots = self.cache.stats()
        if free_slots < 2 or free_pages - self._future_pages() < self._need(self.prefix):
            return None
        h = Request(rid=-1 - group, prompt=self.prefix, gen=0, group=group)
        h.slot = self.cache.alloc()
        self._append([h], [0], [self.prefix])
        self.holders[group] = h.slot
        return h.slot

    def _future_pages(self) -> int:
        """Pages the running requests will still take before they finish."""
        return sum(max(0, self._peak_pages(r, r.shared) - max(0, self._need(r.length) - r.shared // 64))
                   for r in self.running)

    def _peak_pages(self, r: Request, shared: int) -> int:
        """The most pages of its own a request will hold at once, with `shared` prefix tokens in its
        holder's.  An eviction needs those up to the step that crosses the limit and the new ones;
        what stays is all its own, also of a prefix that it shared before."""
        left, length = r.prompt + r.gen - r.position, r.length
        if r.position < r.prompt:  # not prefilled yet
            left, length = r.gen, r.prompt
        evicted = r.position > r.length
        if not self.evict_above:
            return self._need(length + left) - shared // 64
        peak = 0
        if not evicted:
            at = max(length, self.evict_above) + 1  # where the first eviction comes, if the request gets so far
            if length + left <= at:
                return self._need(length + left) - shared // 64
            peak = self._need(at) - shared // 64 + self._need(self.evict_to)
            length, left = self.evict_to, length + left - at
        at = self.evict_above + 1
        return max(peak, self._need(length + left) if length + left <= at else self._need(at) + self._need(self.evict_to))

    def _admit(self, waiting) -> list:
        admitted = []
        while waiting:
            r = waiting[0]
            free_pages, free_slots = self.cache.stats()
            if free_slots == 0:
                break
            sh = 0
            if r.group >= 0 and self.prefix and r.prompt >= self.prefix + self.W:
                sh = self._shareable()
            if sh and self._holder(r.group) is None:
                sh = 0
            free_pages, free_slots = self.cache.stats()
            own = self._peak_pages(r, sh)
            if free_slots == 0 or free_pages - self._future_pages() < own:
                break
            waiting.pop(0)
            r.slot = self.cache.alloc()
            if sh:
                self.cache.share_prefix(r.slot, self.holders[r.group], sh)
                r.shared = sh
                self.stats["shared_tokens"] += sh
                self.stats["prefix_hits"] += 1
            r.length = r.position = sh
            if self.evict_above:
                for wt in self.weights:
                    wt[r.slot].zero_()
            admitted.append(r)
            self.running.append(r)
        # prefill the admitted prompts, in chunks
        while admitted:
            batch, starts, counts, total = [], [], [], 0
            for r in admitted:
                n = min(r.prompt - r.length, self.prefill_chunk - total)
                if n <= 0:
                    continue
                batch.append(r)
                starts.append(r.length)
                counts.append(n)
                total += n
                if total >= self.prefill_chunk:
                    break
            if not batch:
                break
            self._append(batch, starts, counts)
            for r, n in zip(batch, counts):
                r.length += n
                r.position += n
                self.stats["prefill_tokens"] += n
            admitted = [r for r in admitted if r.length < r.prompt]
        return admitted

    # ------------------------------------------------------------------ decode
    def _decode_step(self, on_output: Optional[Callable]):
        c = self.cache
        reqs = self.running
        slots = [r.slot for r in reqs]
        c.reserve(slots, [1] * len(reqs))
        if self.window:
            c.plan_window(slots, n_sink=self.window_sinks, window=self.window)
        else:
            c.plan(slots, flags=N.OSCAR_PLAN_SHARED_PREFIX if self.share_decode else 0)
        # pool rows of every request's new token and query, all layers: row = (A * stream +
        # B * layer + position) mod P, one device tensor per step
        tk = self.tokens
        base = torch.tensor([[TokenSource.A * TokenSource.stream(r, r.position, self.prefix) + r.position,
                              TokenSource.A * (r.rid + 17) + r.position] for r in reqs], dtype=torch.long)
        if self.rotary is not None:
            positions = torch.tensor([r.position for r in reqs], dtype=torch.int32).to(tk.device)
        rows = ((base.to(tk.device)[None] + TokenSource.B * torch.arange(self.w.n_layers, device=tk.device)[:, None, None])
                % tk.P)  # [layer, request, (token, query)]
        for layer in range(self.w.n_layers):
            idx, qi = rows[layer, :, 0], rows[layer, :, 1]
            K = tk.K.index_select(0, idx)
            V = tk.V.index_select(0, idx)
            q = tk.Q.index_select(0, qi)
            turned = self.rotary is not None and self.fmt not in _INT2  # by the append
            if turned:
                c.append_rotated(layer, self.rotary, K, V, q, positions=positions, q_out=q)
            elif self.rotary is not None:
                self.rotary.apply(positions, q, K, q_out=q, k_out=K)
            o32 = torch.empty(q.shape, dtype=torch.float32, device=q.device) if on_output else None
            if self.fmt in _INT2:
                out = c.append_decode(layer, K, V, q, out_f32=o32)
            else:
                if not turned:
                    c.append(layer, K, V)
                if self.evict_above:
                    out, _ = c.decode_weights(layer, q, self.weights[layer], out_f32=o32)
                elif self.window:
                    out = c.attend_window(layer, q, out_f32=o32)
                else:
                    out = c.decode(layer, q, out_f32=o32)
            if on_output:
                if turned:  # (the rows as the cache has them)
                    self.rotary.apply(positions, K, q_out=K)
                on_output(self.stats["steps"], layer, list(reqs), K, V, q, out, o32)
        c.commit()
        for r in reqs:
            r.length += 1
            r.position += 1
            r.generated += 1

    def _evict_long(self, on_evict: Optional[Callable]):
        """Evict from the requests that hold more tokens than the limit and still generate."""
        reqs = [r for r in self.running if r.length > self.evict_above and r.generated < r.gen]
        if not reqs:
            return
        c, slots = self.cache, [r.slot for r in reqs]
        c.evict_begin(slots, [self.evict_to] * len(reqs), *self.protect)
        idx = torch.tensor(slots, dtype=torch.long).to(self.tokens.device)
        for layer in range(self.w.n_layers):
            c.evict(layer, self.weights[layer], self._weights_out, self._kept)
            if on_evict:
                on_evict(layer, reqs, self.weights[layer], self._kept)
            self.weights[layer].index_copy_(0, idx, self._weights_out.index_select(0, idx))
        c.evict_commit()
        for r in reqs:
            r.length, r.shared = self.evict_to, 0
        self.stats["evictions"] += len(reqs)

    def _warm_gathers(self, n_max: int) -> None:
        """Run the step's gathers once for every batch size (set-up, untimed): the first use
        of a torch gather of a given size can stall for seconds while its device code loads."""
        tk = self.tokens
        idx = torch.zeros((self.w.n_layers, n_max, 2), dtype=torch.long, device=tk.device)
        for n in range(1, n_max + 1):
            for t in (tk.K, tk.V, tk.Q):
                t.index_select(0, idx[0, :n, 0])
        base = torch.zeros((n_max, 2), dtype=torch.long)
        _ = ((base.to(tk.device)[None] + TokenSource.B * torch.arange(self.w.n_layers, device=tk.device)[:, None, None])
             % tk.P)
        torch.cuda.synchronize(tk.device)

    def run(self, requests, on_output: Optional[Callable] = None, on_step: Optional[Callable] = None,
            on_evict: Optional[Callable] = None):
        """Serve every request to completion; returns the statistics."""
        waiting = list(requests)
        self._warm_gathers(min(len(requests), self.cache.cfg.max_requests))
        self.running = []
        st = self.stats
        free0 = self.cache.stats()[0]
        dev = self.tokens.device
        ev = []
        torch.cuda.synchronize(dev)
        t0 = time.perf_counter()
        while waiting or self.running:
            self._admit(waiting)
            if not self.running:
                raise RuntimeError(f"request {waiting[0].rid} does not fit the budget even alone")
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            self._decode_step(on_output)
            e1.record()
            ev.append((e0, e1))
            n = len(self.running)
            st["steps"] += 1
            st["generated"] += n
            st["batch_sum"] += n
            st["max_batch"] = max(st["max_batch"], n)
            st["max_pages_used"] = max(st["max_pages_used"], free0 - self.cache.stats()[0])
            if self.evict_above:
                self._evict_long(on_evict)
            done = [r for r in self.running if r.generated >= r.gen]
            for r in done:
                self.cache.free(r.slot)
                r.slot = -1
                st["completed"] += 1
            self.running = [r for r in self.running if r.generated < r.gen]
            if on_step:
                on_step(st["steps"], done)
        torch.cuda.synchronize(dev)
        st["wall_s"] = time.perf_counter() - t0
        st["decode_s"] = sum(a.elapsed_time(b) for a, b in ev) / 1000.0
        st["mean_batch"] = st["batch_sum"] / max(1, st["steps"])
        st["tokens_per_s"] = st["generated"] / st["wall_s"]
        st["decode_tokens_per_s"] = st["generated"] / max(st["decode_s"], 1e-9)
        st["pool_pages"] = self.cache.cfg.max_pages
        return st

    def close(self):
        for slot in self.holders.values():
            self.cache.free(slot)
        self.holders = {}
        self.cache.close()
