"""Prompts through a routed MoE layer: its experts as dense matrices, thousands of tokens at once.

The plane store serves decode steps and small batches, where an expert is hit by a few tokens at the
depths they need. A prompt hits every expert with many tokens; there the experts are held dense (q8: e4m3
codes with a power-of-two scale per 32 columns; or bf16), filled like a :class:`store.ResidentLayer` or
decoded from one, and a layer runs as

  ``residual_norm_q8`` -> (router logits) ``route`` -> ``group_pairs`` -> ``grouped_swiglu`` ->
  ``grouped_matmul`` -> ``combine_rows``

This module allocates (torch) and calls the C ABI; the only arithmetic of its own is the cast of filled
weights to bf16 and the decoding of stored ones, when a layer is built.
"""
from __future__ import annotations

import torch

from . import (BF16, Q8, _dense_ptr, combine_rows, extract_prefix, group_pairs, group_workspace_bytes, grouped_matmul,
               grouped_swiglu, make_dense, make_rows, quantize_q8, residual_norm_q8, route)
from .store import DOWN, GATE, UP, ResidentLayer


def _floats(name, t, n: int) -> None:
    """Refuses a tensor that is not float32 or has fewer than n elements: the library takes addresses and would read
    past its end (None, and what is no tensor, pass)."""
    if isinstance(t, torch.Tensor) and (t.dtype != torch.float32 or t.numel() < n):
        raise ValueError(f"{name}: float32 with at least {n} elements, not {t.dtype} with {t.numel()}")


class DenseExperts:
    """The experts of one layer: [E][gate rows | up rows][H] and [E][H][I] in q8 or bf16."""

    def __init__(self, E: int, H: int, I: int, fill, kind: int = Q8, device="cuda", stream=None):
        """fill(expert, mat, w) writes float32 weights of shape (rows*cols,) into device tensor w
        (gate/up: I x H, down: H x I), on the current stream. H and I: multiples of 128 (q8) or 8 (bf16)."""
        step = {Q8: 128, BF16: 8}.get(kind)
        if step is None or not 1 <= E <= 2048 or min(H, I) < 1 or H % step or I % step:
            raise ValueError(f"{E} experts of {H} x {I} in type {kind}: 1..2048 of multiples of 128 (q8) or 8 (bf16)")
        self.E, self.H, self.I, self.kind = E, H, I, kind
        dev = torch.device(device)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            dtype = torch.uint8 if kind == Q8 else torch.bfloat16
            self.up = torch.empty(E, 2 * I, H, dtype=dtype, device=dev)
            self.down = torch.empty(E, H, I, dtype=dtype, device=dev)
            self.up_scales = self.down_scales = None
            if kind == Q8:
                self.up_scales = torch.empty(E, 2 * I, H // 32, dtype=torch.uint8, device=dev)
                self.down_scales = torch.empty(E, H, I // 32, dtype=torch.uint8, device=dev)
            w = torch.empty(H * I, dtype=torch.float32, device=dev)
            for e in range(E):
                for m in (GATE, UP, DOWN):
                    rows, cols = (I, H) if m != DOWN else (H, I)
                    at = slice(0, I) if m == GATE else slice(I, 2 * I) if m == UP else slice(0, H)
                    fill(e, m, w)
                    to, scales = (self.up, self.up_scales) if m != DOWN else (self.down, self.down_scales)
                    if kind == Q8:
                        quantize_q8(w, False, rows, cols, to[e, at], scales[e, at], st)
                    else:
                        to[e, at].copy_(w.view(rows, cols))
        self.up_dense = make_dense(kind, self.up, self.up_scales, E, 2 * I, H)
        self.down_dense = make_dense(kind, self.down, self.down_scales, E, H, I)

    @classmethod
    def from_layer(cls, R: ResidentLayer, kind: int = Q8, depth: int = 8, stream=None) -> "DenseExperts":
        """A stored layer's experts at the given depth."""
        dev = R.pool.device
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):  # torch takes its memory back in the order of this stream
            idx = torch.empty(R.H * R.I, dtype=torch.uint8, device=dev)
        level = slice((1 << depth) - 2, (1 << (depth + 1)) - 2)

        def fill(e, m, w):
            rows, cols = (R.I, R.H) if m != DOWN else (R.H, R.I)
            planes = R.pool[e * 8 * R.slot_words + m * R.mat_words:]
            extract_prefix(planes, R.slot_words, rows, cols, depth, idx, st)
            table = R.codebooks[(3 * e + m) * 510:(3 * e + m + 1) * 510][level]
            v = table[idx.int()].view(rows, cols // R.G, R.G) * R.expert_scales(e, m)[:, :, None]
            w.copy_(v.reshape(-1))

        return cls(R.E, R.H, R.I, fill, kind, dev, st)


class PromptLayer:
    """Buffers for up to max_tokens tokens through one layer's experts, k of them each. Calls that overlap
    on the GPU need a PromptLayer each (they may share the experts). Calls run on the stream given, or on
    torch's current stream of the layer's device; keep the layer until what they enqueued has finished."""

    def __init__(self, experts: DenseExperts, k: int, max_tokens: int):
        self.experts, self.k, self.max_tokens = experts, k, max_tokens
        E, H, I, T, P = experts.E, experts.H, experts.I, max_tokens, max_tokens * k
        dev = experts.up.device
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        q8 = experts.kind == Q8
        self.x = new(T, H, dtype=torch.uint8 if q8 else torch.bfloat16)
        self.x_scales = new(T, H // 32, dtype=torch.uint8) if q8 else None
        self.ids, self.w = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        self.offsets = new(E + 1, dtype=torch.int32)
        self.row_of, self.token_of = new(P, dtype=torch.int32), new(P, dtype=torch.int32)
        # fewer tokens never need more: the count of blocks grows with the pairs
        self.ws = new(max(group_workspace_bytes(T, k, E), 16), dtype=torch.uint8)
        self.h = new(P, I, dtype=torch.uint8 if q8 else torch.bfloat16)
        self.h_scales = new(P, I // 32, dtype=torch.uint8) if q8 else None
        self.out = new(P, H, dtype=torch.bfloat16)
        self.y = new(T, H, dtype=torch.float32)
        self.errors = torch.zeros(2, dtype=torch.int32, device=dev)
        if dev.type == "cuda" and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()  # calls may come on any stream

    def _tokens(self, T: int) -> None:
        if not 0 <= T <= self.max_tokens:
            raise ValueError(f"{T} tokens in a layer of {self.max_tokens}")

    def _stream(self, stream):
        return stream if stream is not None else torch.cuda.current_stream(self.y.device)

    def norm(self, r, y, T: int, gain=None, eps: float = 0.0, stream=None) -> None:
        """The layer's input from the residual stream: r += y (y may be None), x = r / rms(r) * gain. All in float32:
        r and y [T, H], gain [H]."""
        self._tokens(T)
        H = self.experts.H
        for name, t, n in (("r", r, T * H), ("y", y, T * H), ("gain", gain, H)):
            _floats(name, t, n)
        x, stream = self.experts, self._stream(stream)
        if x.kind == Q8:
            residual_norm_q8(r, y, gain, eps, T, x.H, self.x, self.x_scales, None, stream)
        else:
            residual_norm_q8(r, y, gain, eps, T, x.H, None, None, self.x, stream)

    def route(self, logits, T: int, stream=None) -> None:
        """Experts and weights of the first T tokens from their router logits, float32 [T, E]."""
        self._tokens(T)
        _floats("logits", logits, T * self.experts.E)
        route(_dense_ptr(logits), T, self.experts.E, self.k, self.ids, self.w, self._stream(stream))

    def forward(self, T: int, stream=None) -> torch.Tensor:
        """The layer's output [T, H] for the first T rows of x, ids and w (an id outside 0..E-1 marks a
        slot that no expert takes). The tensor is the layer's own buffer. After a wait that ran out on the GPU
        it is not complete: see error()."""
        self._tokens(T)
        x, k, P, stream = self.experts, self.k, T * self.k, self._stream(stream)
        group_pairs(self.ids, T, k, x.E, self.offsets, self.row_of, self.token_of, self.ws, self.ws.numel(), stream)
        rows = make_rows(x.kind, self.x, self.x_scales, T, self.token_of, self.errors)
        grouped_swiglu(x.up_dense, rows, self.offsets, P, x.kind, self.h, self.h_scales, stream)
        rows = make_rows(x.kind, self.h, self.h_scales, P, None, self.errors)
        grouped_matmul(x.down_dense, rows, self.offsets, P, BF16, self.out, stream)
        combine_rows(self.out, True, self.row_of, self.w, T, k, x.H, self.y, stream)
        return self.y[:T]

    def error(self, stream=None):
        """(code, detail) of the first wait that ran out in this layer's products (code 3; 0: none) since the last
        such call, after what the stream holds (waits for it)."""
        st = self._stream(stream)
        with torch.cuda.stream(st if hasattr(st, "cuda_stream") else torch.cuda.ExternalStream(int(st), self.y.device)):
            code, detail = self.errors.tolist()
            self.errors.zero_()
        return code, detail
