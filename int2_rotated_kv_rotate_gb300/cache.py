"""A torch-facing handle on one cache of the C library (marshalling only).

torch allocates the device block and the decode workspace; every operation is one call
of the C ABI (see include/oscar.h for semantics and layouts).
"""
from __future__ import annotations

import torch

from . import _native as N


class KVCache:
    """One cache: INT2 mixed-precision (fmt=N.OSCAR_FORMAT_INT2, or N.OSCAR_FORMAT_INT2_CM with
    channel-major value pages) or plain BF16 pages (N.OSCAR_FORMAT_BF16)."""

    def __init__(self, *, fmt: int = N.OSCAR_FORMAT_INT2, n_q_heads: int, n_kv_heads: int, group: int = 128,
                 n_sink: int = 4, window: int = 128, n_layers: int = 1, max_requests: int = 1, max_pages: int,
                 max_pages_per_request: int, head_dim: int = 128, device="cuda"):
        self.cfg = N.oscar_config(fmt, head_dim, n_q_heads, n_kv_heads, group, 64, n_sink, window, n_layers,
                                  max_requests, max_pages, max_pages_per_request)
        self.nbytes = N.oscar_cache_device_bytes(self.cfg)
        self.device = torch.device(device)
        self.mem = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        self.handle = N.oscar_cache_create(self.cfg, self.mem, self.nbytes)
        self.layout = N.oscar_cache_layout(self.handle)
        self.workspace = None
        self.weights_workspace = None
        self._weights_full = N.oscar_decode_weights_workspace_max_bytes(self.handle)  # bytes of it for every plan
        self._weights_need = 0  # and for the current one
        self._weights_streams = []  # streams that launched on it, its own first
        self.weights_stride = N.oscar_weights_stride(self.handle)  # 0: no weights in this format
        self.fmt = fmt
        self.is_int2 = fmt in (N.OSCAR_FORMAT_INT2, N.OSCAR_FORMAT_INT2_CM)
        self._rows = None  # rows of k_new / v_new the pending reservation expects
        self._n_plan = None  # requests of the current decode plan

    # ------------------------------------------------------------------ lifecycle
    def close(self) -> None:
        if getattr(self, "handle", None):
            N.oscar_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ params / requests
    def set_layer_params(self, layer: int, R_K, R_V, clip_K, clip_V, stream=None) -> None:
        f = lambda t: torch.as_tensor(t, dtype=torch.float32).contiguous().cpu()  # noqa: E731
        N.oscar_set_layer_params(self.handle, layer, f(R_K), f(R_V), f(clip_K), f(clip_V), stream)

    def stats(self):
        """(free pages, free request slots)."""
        return N.oscar_cache_stats(self.handle)

    def alloc(self) -> int:
        return N.oscar_request_alloc(self.handle)

    def free(self, slot: int) -> None:
        N.oscar_request_free(self.handle, slot)

    def info(self, slot: int):
        return N.oscar_request_info(self.handle, slot)

    def pages(self, slot: int):
        return N.oscar_request_pages(self.handle, slot, self.info(slot)[2])

    def share_prefix(self, dst: int, src: int, n_tokens: int, stream=None) -> None:
        N.oscar_request_share_prefix(self.handle, dst, src, n_tokens, stream)

    # ------------------------------------------------------------------ append
    def reserve(self, slots, n_new, stream=None) -> None:
        N.oscar_reserve(self.handle, slots, n_new, stream)
        self._rows = int(sum(int(n) for n in n_new))

    def _check_tokens(self, k_new, v_new) -> None:
        shape = (self._rows, self.cfg.n_kv_heads, self.cfg.head_dim)
        for t in (k_new, v_new):
            if (tuple(t.shape) != shape or t.dtype != torch.bfloat16 or not t.is_contiguous()
                    or t.device != self.mem.device):
                raise ValueError(f"token tensors must be contiguous bf16 {shape} on {self.mem.device}")

    def quantize_append(self, layer: int, k_new, v_new, stream=None) -> None:
        self._check_tokens(k_new, v_new)
        N.oscar_quantize_append(self.handle, layer, k_new, v_new, stream)

    def bf16_append(self, layer: int, k_new, v_new, stream=None) -> None:
        self._check_tokens(k_new, v_new)
        N.oscar_bf16_append(self.handle, layer, k_new, v_new, stream)

    def append(self, layer: int, k_new, v_new, stream=None) -> None:
        if self.is_int2:
            self.quantize_append(layer, k_new, v_new, stream)
        else:
            self.bf16_append(layer, k_new, v_new, stream)

    def commit(self) -> None:
        N.oscar_commit_append(self.handle)
        self._rows = None
        self._n_plan = None

    # ------------------------------------------------------------------ decode
    def plan(self, slots, max_split_pages: int = 0, stream=None, flags: int = 0) -> int:
        N.oscar_plan_decode_ex(self.handle, slots, max_split_pages, flags, stream)
        self._n_plan = len(list(slots))
        need = N.oscar_decode_workspace_bytes(self.handle)
        if self.workspace is None or self.workspace.numel() < need:
            # sized for every plan of the cache, once: launches captured into a graph keep
            # this pointer across later plans
            full = N.oscar_decode_workspace_max_bytes(self.handle)
            with N.on_stream(stream):
                self.workspace = torch.empty(max(need, full, 256), dtype=torch.uint8, device=self.device)
        if not self.is_int2:
            self._weights_need = N.oscar_decode_weights_workspace_bytes(self.handle)
        return need

    def plan_info(self):
        return N.oscar_plan_info(self.handle)

    def shared_info(self):
        """(work items, pages) that the plan attends once for several requests."""
        return N.oscar_plan_shared_info(self.handle)

    def _check_decode(self, q, out, out_f32, stream):
        shape = (self._n_plan, self.cfg.n_q_heads, self.cfg.head_dim)
        if tuple(q.shape) != shape or q.dtype != torch.bfloat16 or not q.is_contiguous() or q.device != self.mem.device:
            raise ValueError(f"q must be contiguous bf16 {shape} on {self.mem.device}")
        if out is None:
            if stream is None:
                out = torch.empty_like(q)
            else:
                with N.on_stream(stream):
                    out = torch.empty_like(q)
        elif (tuple(out.shape) != shape or out.dtype != torch.bfloat16 or not out.is_contiguous()
                or out.device != self.mem.device):
            raise ValueError("out must be contiguous bf16 like q")
        if out_f32 is not None and (tuple(out_f32.shape) != shape or out_f32.dtype != torch.float32
                                    or not out_f32.is_contiguous() or out_f32.device != self.mem.device):
            raise ValueError("out_f32 must be contiguous fp32 like q")
        return out

    def decode(self, layer: int, q, out=None, out_f32=None, stream=None):
        out = self._check_decode(q, out, out_f32, stream)
        if self.is_int2:
            N.oscar_decode_attention(self.handle, layer, q, out, self.workspace, out_f32, stream)
        else:
            N.oscar_bf16_decode_attention(self.handle, layer, q, out, self.workspace, out_f32, stream)
        return out

    # ------------------------------------------------------------------ accumulated weights (BF16 format)
    def new_weights(self) -> torch.Tensor:
        """A layer's accumulated attention weights, zeros: fp32 [request slots, H_kv, weights_stride]."""
        return torch.zeros(self._weights_shape(), device=self.device)

    def _weights_shape(self):
        if not self.weights_stride:
            raise ValueError("accumulated weights need the BF16 format")
        return (self.cfg.max_requests, self.cfg.n_kv_heads, self.weights_stride)

    def _check_weights(self, name, t, dtype=torch.float32):
        shape = self._weights_shape()
        if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous() or t.device != self.mem.device:
            raise ValueError(f"{name} must be contiguous {dtype} {shape} on {self.mem.device}")

    def _score_space(self, stream):
        """The weights' workspace: the plan's size and some to grow, or every plan's size from the
        first captured launch on, since a graph keeps the pointer across later plans."""
        ws = self.weights_workspace
        full = self._weights_full
        if ws is not None and ws.numel() >= full:
            return ws
        with N.on_stream(stream):
            captured = torch.cuda.is_current_stream_capturing()
            if ws is None or ws.numel() < (full if captured else self._weights_need):
                for handle in self._weights_streams:  # launches of any of them may still use the old one
                    ws.record_stream(torch.cuda.ExternalStream(handle, device=self.mem.device))
                scores = self._weights_need - full + 4 * self.cfg.max_requests * self.cfg.n_q_heads * self.weights_stride
                size = full if captured else min(full, self._weights_need + scores // 4)
                self.weights_workspace = ws = torch.empty(max(size, 256), dtype=torch.uint8, device=self.device)
                self._weights_streams = []
            handle = N._stream(None)
        if handle not in self._weights_streams:
            self._weights_streams.append(handle)
        return ws

    def decode_weights(self, layer: int, q, weights, weights_out=None, out=None, out_f32=None, stream=None):
        """decode that also adds every attended token's softmax probability, summed over its
        kv-head's query heads, to `weights`: (out, weights_out).  In place without weights_out;
        rows of requests outside the plan and entries past a request's length stay as they are."""
        weights_out = weights if weights_out is None else weights_out
        self._check_weights("weights", weights)
        self._check_weights("weights_out", weights_out)
        out = self._check_decode(q, out, out_f32, stream)
        N.oscar_bf16_decode_weights(self.handle, layer, q, out, weights, weights_out, self._score_space(stream), out_f32,
                                    stream)
        return out, weights_out

    # ------------------------------------------------------------------ eviction (BF16 format)
    def evict_begin(self, slots, keep, n_sink: int = 0, n_recent: int = 0, stream=None) -> None:
        """Plan the eviction of all but keep[i] tokens of request slots[i], per layer and kv-head:
        the first n_sink and the last n_recent stay, of the others those with the greatest weight."""
        N.oscar_evict_begin(self.handle, slots, keep, n_sink, n_recent, stream)

    def evict(self, layer: int, weights, weights_out=None, kept=None, stream=None):
        """Copy one layer's kept tokens into their new pages: (weights_out, kept), the kept tokens'
        weights (zeros behind them) and their positions before the eviction, int32 (-1 behind
        them when this call makes the tensor).  Rows of other slots stay as they are (those of a
        weights_out that this call makes: as in weights)."""
        self._check_weights("weights", weights)
        with N.on_stream(stream):  # what this call makes is made in the launch's order
            if weights_out is None:
                weights_out = weights.clone()
            if kept is None:
                kept = torch.full(weights.shape, -1, dtype=torch.int32, device=self.device)
        self._check_weights("weights_out", weights_out)
        self._check_weights("kept", kept, torch.int32)
        N.oscar_evict(self.handle, layer, weights, weights_out, kept, stream)
        return weights_out, kept

    def evict_pages(self, slot: int):
        """Pages that slot will have after the commit of the pending eviction."""
        return N.oscar_evict_pages(self.handle, slot)

    def evict_commit(self, stream=None) -> None:
        N.oscar_evict_commit(self.handle, stream)
        self._n_plan = None

    def evict_cancel(self) -> None:
        N.oscar_evict_cancel(self.handle)

    def append_decode(self, layer: int, k_new, v_new, q, out=None, out_f32=None, stream=None):
        """quantize_append then decode of `layer` in one launch (INT2 format; plan made
        during the reservation over every reserved slot)."""
        self._check_tokens(k_new, v_new)
        out = self._check_decode(q, out, out_f32, stream)
        N.oscar_append_decode_attention(self.handle, layer, k_new, v_new, q, out, self.workspace, out_f32, stream)
        return out

    def status(self, stream=None):
        return N.oscar_get_status(self.handle, stream)

    # ------------------------------------------------------------------ raw reads (tests)
    def _bytes(self, offset: int, n: int) -> torch.Tensor:
        return self.mem[offset:offset + n]

    def bf16_pages(self, layer: int) -> torch.Tensor:
        """The BF16 format's pages of one layer, a view: [pages, H_kv, K|V, 64, 128]."""
        if self.is_int2:
            raise ValueError("BF16 pages need the BF16 format")
        n = self.cfg.max_pages * self.cfg.n_kv_heads * self.layout.bf16_page_bytes
        at = self.layout.bf16_pages + layer * n
        return self._bytes(at, n).view(torch.bfloat16).view(self.cfg.max_pages, self.cfg.n_kv_heads, 2, 64, 128)

    def int2_rows(self, layer: int, slot: int, kvh: int, kv: int, positions):
        """Device-stored 32-byte code rows and scale/zero words of INT2 positions (host)."""
        H = self.cfg.n_kv_heads
        ng = 128 // self.cfg.group
        pos = torch.as_tensor(list(positions) if not torch.is_tensor(positions) else positions, dtype=torch.long)
        if pos.numel() == 0:
            return torch.empty((0, 32), dtype=torch.uint8), torch.empty((0, ng * 2), dtype=torch.int16)
        pages = torch.tensor(self.pages(slot), dtype=torch.long)
        phys = pages[pos // 64]
        t = pos % 64
        code_head = self.layout.codes_page_bytes
        sz_head = self.layout.sz_page_bytes
        code_layer = self.cfg.max_pages * H * code_head
        sz_layer = self.cfg.max_pages * H * sz_head
        c0 = self.layout.codes + layer * code_layer + (phys * H + kvh) * code_head + kv * 64 * 32 + t * 32
        s0 = self.layout.sz + layer * sz_layer + (phys * H + kvh) * sz_head + kv * 64 * ng * 4 + t * ng * 4
        dev = self.mem.device
        is_ = (s0[:, None] + torch.arange(ng * 4)[None, :]).to(dev)
        sz = self.mem[is_].cpu().contiguous().view(torch.int16)
        if self.fmt == N.OSCAR_FORMAT_INT2_CM and kv == 1:
            return self._cm_rows(c0 - t * 32, t), sz
        ic = (c0[:, None] + torch.arange(32)[None, :]).to(dev)
        rows = self.mem[ic].cpu()
        return rows, sz

    def _cm_rows(self, vblock: torch.Tensor, t: torch.Tensor) -> torch.Tensor:
        """Token-major 32-byte rows of positions t (in their pages) rebuilt from channel-major
        value blocks at byte offsets vblock: word 128 b + c holds channel c of tokens
        16 b .. 16 b + 15, token 16 b + 8 h + f at bit 16 h + 2 f."""
        dev = self.mem.device
        c = torch.arange(128)
        word0 = vblock + 4 * (128 * (t // 16))
        iw = (word0[:, None, None] + 4 * c[None, :, None] + torch.arange(4)[None, None, :]).to(dev)
        words = self.mem[iw].cpu().to(torch.int64)
        words = words[..., 0] | (words[..., 1] << 8) | (words[..., 2] << 16) | (words[..., 3] << 24)  # [n, 128]
        sh = (16 * ((t // 8) % 2) + 2 * (t % 8))[:, None]
        codes = (words >> sh) & 3  # [n, 128] code of channel c
        f, w, h = c // 16, (c % 16) // 2, c % 2  # channel c = 16 f + 2 w + h: bit 32 w + 16 h + 2 f of the row
        row_words = torch.zeros((t.numel(), 8), dtype=torch.int64)
        row_words.scatter_add_(1, w[None, :].expand(t.numel(), 128), codes << (16 * h + 2 * f)[None, :])
        row_words = torch.where(row_words >= 2**31, row_words - 2**32, row_words)  # two's complement words
        return row_words.to(torch.int32).view(torch.uint8).reshape(t.numel(), 32)

    def _head_block(self, pool_off: int, per_head: int, slot: int, layer: int, kvh: int):
        H = self.cfg.n_kv_heads
        off = pool_off + ((slot * self.cfg.n_layers + layer) * H + kvh) * per_head
        return self.mem[off:off + per_head]

    def sink_tokens(self, layer: int, slot: int, kvh: int, kv: int) -> torch.Tensor:
        S = self.cfg.n_sink
        blk = self._head_block(self.layout.sink, self.layout.sink_bytes_per_head, slot, layer, kvh)
        return blk.view(torch.int16).view(2, S, 128)[kv].cpu()

    def ring_tokens(self, layer: int, slot: int, kvh: int, kv: int) -> torch.Tensor:
        W = self.cfg.window
        blk = self._head_block(self.layout.ring, self.layout.ring_bytes_per_head, slot, layer, kvh)
        return blk.view(torch.int16).view(2, W, 128)[kv].cpu()
