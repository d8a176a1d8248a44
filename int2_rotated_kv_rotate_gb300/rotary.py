"""Rotary positions on queries and keys (marshalling of oscar_rope, see include/oscar.h).

A model turns its queries and its new keys by their positions before the cache takes them:
RotaryEmbedding holds the table of one configuration on the device and applies it, in
either cache format's step, as one launch for both tensors.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _native as N

_DTYPES = {torch.bfloat16: N.OSCAR_DTYPE_BF16, torch.float16: N.OSCAR_DTYPE_F16, torch.float32: N.OSCAR_DTYPE_F32}
_SCALINGS = {"linear": N.OSCAR_ROPE_LINEAR, "bands": N.OSCAR_ROPE_BANDS, "yarn": N.OSCAR_ROPE_YARN}


_count_as_written = torch.autograd.graph.increment_version  # (a graph that saved the tensor is told)


class _Apply(torch.autograd.Function):
    """RotaryEmbedding.apply on inputs that need gradients: the transposed map on theirs."""

    @staticmethod
    def forward(ctx, rotary, transpose, positions, *tensors):
        ctx.rotary, ctx.transpose = rotary, transpose
        ctx.save_for_backward(positions)
        ctx.set_materialize_grads(False)
        return rotary.apply(positions, *tensors, transpose=transpose)

    @staticmethod
    def backward(ctx, *grads):
        out = [None] * len(grads)
        live = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[3 + i]]
        if live:
            (positions,) = ctx.saved_tensors
            rows = [grads[i] if grads[i].stride(-1) == 1 else grads[i].contiguous() for i in live]
            turned = ctx.rotary.apply(positions, *rows, transpose=not ctx.transpose)
            for i, g in zip(live, turned if len(live) > 1 else (turned,)):
                out[i] = g
        return (None, None, None, *out)


class RotaryEmbedding:
    """Rotary positions of one configuration.

    head_dim channels per head, the first rotary_dim of which turn (all of them by default);
    pairs are channels (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when interleaved.
    scaling, for contexts longer than the model's own: a dict with "type" ("linear", "bands"
    or "yarn"), "factor", and for the last two "original_context" and the turns within it that
    bound the mixed pairs, "low" and "high" (default 1 and 4 for bands, 1 and 32 for yarn).
    """

    def __init__(self, *, head_dim: int = 128, rotary_dim: Optional[int] = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: Optional[dict] = None, device="cuda"):
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.interleaved = bool(interleaved)
        if not 2 <= self.rotary_dim <= self.head_dim <= 512:
            raise ValueError("head_dim must be in [rotary_dim, 512] and rotary_dim at least 2")
        s = dict(scaling or {})
        kind = s.pop("type", None)
        if scaling is not None and kind not in _SCALINGS:
            raise ValueError(f"scaling type must be one of {sorted(_SCALINGS)}")
        code = _SCALINGS[kind] if kind else N.OSCAR_ROPE_UNSCALED
        factor = float(s.pop("factor", 1.0))
        low = float(s.pop("low", 1.0))
        high = float(s.pop("high", 32.0 if kind == "yarn" else 4.0))
        original = float(s.pop("original_context", 0.0))
        if s:
            raise ValueError(f"unknown scaling entries {sorted(s)}")
        cfg = N.oscar_rope_config(self.rotary_dim, code, float(base), factor, low, high, original)
        steps, self.magnitude = N.oscar_rope_steps(cfg)
        signed = [v - (1 << 64) if v >= 1 << 63 else v for v in steps]
        self.steps = torch.tensor(signed, dtype=torch.int64).to(device)
        self.device = self.steps.device

    def _check(self, name: str, x, rows: int, like=None):
        shape = x.shape
        if len(shape) != 3 or shape[2] != self.head_dim or x.stride()[2] != 1:
            raise ValueError(f"{name} must be [rows, heads, {self.head_dim}] with contiguous channels")
        if x.dtype not in _DTYPES or x.device != self.device:
            raise ValueError(f"{name} must be bf16, fp16 or fp32 on {self.device}")
        if shape[0] != rows:
            raise ValueError(f"{name} must have {rows} rows")
        if like is not None and (shape != like.shape or x.dtype != like.dtype):
            raise ValueError(f"{name} must have the shape and dtype of its input")

    @staticmethod
    def _new(x, stream):
        if stream is None:
            return torch.empty(x.shape, dtype=x.dtype, device=x.device)
        with N.on_stream(stream):  # in the launch's order
            return torch.empty(x.shape, dtype=x.dtype, device=x.device)

    def apply(self, positions, q, k=None, *, q_out=None, k_out=None, transpose: bool = False, stream=None):
        """(q', k') of rows at `positions` (int32 or int64 [rows], any order): q [rows, H_q,
        head_dim] and optionally k [rows, H_kv, head_dim], any row and head strides.  Outputs
        are new contiguous tensors unless given, made on the stream of the launch; q_out = q
        (k_out = k) works in place.
        transpose=True applies the transposed map: gradients of q', k' to those of q, k.  Inputs
        that require gradients get them through autograd, on new outputs only."""
        if (positions.dim() != 1 or positions.dtype not in (torch.int32, torch.int64)
                or positions.device != self.device or (positions.shape[0] > 1 and positions.stride(0) != 1)):
            raise ValueError(f"positions must be contiguous int32 or int64 [rows] on {self.device}")
        rows = positions.shape[0]
        if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)
                                        or (q_out is not None and q_out.requires_grad)
                                        or (k_out is not None and k_out.requires_grad)):
            if q_out is not None or k_out is not None:
                raise ValueError("tensors that require grad are turned into new outputs only")
            with N.on_stream(stream):
                return _Apply.apply(self, transpose, positions, q) if k is None else _Apply.apply(self, transpose, positions, q, k)
        self._check("q", q, rows)
        written = []
        if q_out is None:
            q_out = self._new(q, stream)
        else:
            if q_out is not q:
                self._check("q_out", q_out, rows, q)
            written.append(q_out)
        pairs = [(q, q_out)]
        if k is not None:
            self._check("k", k, rows)
            if k.dtype != q.dtype:
                raise ValueError("q and k must have one dtype")
            if k_out is None:
                k_out = self._new(k, stream)
            else:
                if k_out is not k:
                    self._check("k_out", k_out, rows, k)
                written.append(k_out)
            pairs.append((k, k_out))
        elif k_out is not None:
            raise ValueError("k_out without k")
        flags = ((N.OSCAR_ROPE_INTERLEAVED if self.interleaved else 0) | (N.OSCAR_ROPE_TRANSPOSE if transpose else 0)
                 | (N.OSCAR_ROPE_POSITIONS64 if positions.dtype == torch.int64 else 0))
        args = (pairs, self.steps, self.head_dim, self.rotary_dim, self.magnitude, _DTYPES[q.dtype], flags, positions,
                stream)
        if self.device.index == torch.cuda.current_device():
            N.oscar_rope(*args)
        else:
            with torch.cuda.device(self.device):
                N.oscar_rope(*args)
        if written:
            _count_as_written(written)
        return (q_out, k_out) if k is not None else q_out
