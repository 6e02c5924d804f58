"""A gated feed-forward block on 8-bit weights with block scales, run through the C ABI.

The block is  y = x + (gate(g) * u) W_down^T,  [g u] = norm(x) W_gate_up^T.  A call enqueues, on the current stream and
without reading anything back:

    dlf_rms_norm            the norm, straight into e4m3 codes and a scale for each 128 values
    dlf_gemm_blocks_gated   gate and up projections in one product, gated in its epilogue
    dlf_quant_blocks        the activations into codes and scales
    dlf_gemm_blocks         the down projection with the residual

so that it can be captured in a graph.  The weights take half of what bf16 does; where there are few rows, as in a step
of decoding, their read is what a call takes.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (Buffers, dlf_gemm_blocks, dlf_gemm_blocks_gated, dlf_gemm_blocks_workspace_bytes, dlf_quant_blocks,
               dlf_quant_blocks_weights, dlf_rms_norm, gemm_blocks_desc, quant_blocks_desc, rms_norm_desc, scale_stride)

FP8 = torch.float8_e4m3fn


def pack_gate_up(w_gate, w_up, device="cuda"):
    """Codes and scales of gate and up weights [d_ff][d_model] (host, fp32), their rows interleaved, on the device."""
    gate, up = (np.asarray(w, np.float32) for w in (w_gate, w_up))
    if gate.shape != up.shape or gate.ndim != 2:
        raise ValueError("gate and up weights must have one shape [d_ff][d_model]")
    both = np.empty((2 * gate.shape[0], gate.shape[1]), np.float32)
    both[0::2], both[1::2] = gate, up
    return _to_device(dlf_quant_blocks_weights(both, gated=True), device)


def pack(w, device="cuda"):
    """Codes and scales of one weight [out][in] (host, fp32), on the device."""
    return _to_device(dlf_quant_blocks_weights(np.asarray(w, np.float32)), device)


def _to_device(packed, device):
    codes, scale = (torch.from_numpy(t).to(device) for t in packed)
    return codes.view(FP8), scale


def _packed(w, rows, cols, scale_rows, name):
    codes, scale = w
    if tuple(codes.shape) != (rows, cols) or codes.dtype != FP8:
        raise ValueError(f"{name} codes must be {FP8} [{rows}][{cols}], got {codes.dtype} {list(codes.shape)}")
    if tuple(scale.shape) != (scale_rows, scale_stride(cols)) or scale.dtype != torch.float32:
        raise ValueError(f"{name} scales must be fp32 [{scale_rows}][{scale_stride(cols)}], got {scale.dtype} {list(scale.shape)}")


class GatedFeedForward:
    """``gate_up`` and ``down``: what pack_gate_up and pack return.  ``norm``: fp32 [d_model] or None (= 1).
    ``rows``: rows of a call that may be captured: their buffers are made here and stay where they are.  Calls of other
    lengths share one set of buffers, which grows to the longest, and are refused under capture.  A set is one call's at a
    time: calls on streams that overlap need a block each (the weights may be the same tensors); calls on one stream after
    another, each waiting for the last, may share one."""

    def __init__(self, gate_up, down, norm=None, eps=1e-5, gate="silu", rows=0):
        self.gate_up, self.down, self.norm, self.eps, self.gate = gate_up, down, norm, eps, gate
        self.d_model, self.d_ff = down[0].shape
        _packed(gate_up, 2 * self.d_ff, self.d_model, 2 * -(-2 * self.d_ff // 256), "gate and up")
        _packed(down, self.d_model, self.d_ff, -(-self.d_model // 128), "down")
        if norm is not None and (tuple(norm.shape) != (self.d_model,) or norm.dtype != torch.float32):
            raise ValueError(f"norm must be fp32 [{self.d_model}]")
        device = down[0].device
        for t, name in ((gate_up[0], "gate and up codes"), (gate_up[1], "gate and up scales"), (down[1], "down scales"), (norm, "norm")):
            if t is not None and t.device != device:
                raise ValueError(f"{name} are on {t.device}, the down codes on {device}")
        self.rows = rows
        self._own_room = self._allocate(rows) if rows > 0 else None
        self._own = self._views(rows, self._own_room) if rows > 0 else None
        self._shared = None

    def _descs(self, m):
        return (gemm_blocks_desc(m, 2 * self.d_ff, self.d_model), gemm_blocks_desc(m, self.d_model, self.d_ff))

    def _allocate(self, m, ws=0):
        device = self.down[0].device
        f32 = dict(dtype=torch.float32, device=device)
        ws = max([ws] + [dlf_gemm_blocks_workspace_bytes(d) for d in self._descs(m)])
        return Buffers(x=torch.empty(m, self.d_model, dtype=FP8, device=device),
                       x_scale=torch.empty(m, scale_stride(self.d_model), **f32),
                       h=torch.empty(m, self.d_ff, dtype=torch.bfloat16, device=device),
                       q=torch.empty(m, self.d_ff, dtype=FP8, device=device),
                       q_scale=torch.empty(m, scale_stride(self.d_ff), **f32),
                       ws=torch.empty(ws, dtype=torch.uint8, device=device))

    def _views(self, m, room):
        got = {n: t if n == "ws" else t[:m] for n, t in room.items()}
        got["first"], got["second"] = self._descs(m)
        got["norm"] = rms_norm_desc(m, self.d_model, self.eps, "bf16", "fp8")
        got["quant"] = quant_blocks_desc(m, self.d_ff)
        return got

    def _buffers(self, m):
        if m == self.rows and self._own is not None:
            self._own_room.used()
            return self._own
        if torch.cuda.is_current_stream_capturing():
            raise ValueError(f"only calls of `rows` = {self.rows} rows may be captured, got {m}")
        need = max(dlf_gemm_blocks_workspace_bytes(d) for d in self._descs(m))
        if self._shared is None or self._shared["x"].shape[0] < m or self._shared["ws"].numel() < need:
            most, ws = (0, 0) if self._shared is None else (self._shared["x"].shape[0], self._shared["ws"].numel())
            self._shared = None             # before the next is made
            self._shared = self._allocate(max(m, most), max(ws, need))
        return self._views(m, self._shared.used())

    def __call__(self, x, y):
        """y = x + the block of x, both bf16 [rows][d_model] and contiguous; y is not x."""
        m = x.shape[0]
        for t, name in ((x, "x"), (y, "y")):
            if tuple(t.shape) != (m, self.d_model) or t.dtype != torch.bfloat16:
                raise ValueError(f"{name} must be bf16 [{m}][{self.d_model}], got {t.dtype} {list(t.shape)}")
        if m == 0:
            return
        b = self._buffers(m)
        dlf_rms_norm(b["norm"], x, None, self.norm, None, b["x"], b["x_scale"])
        dlf_gemm_blocks_gated(b["first"], b["x"], b["x_scale"], *self.gate_up, None, self.gate, b["h"], b["ws"], b["ws"].numel())
        dlf_quant_blocks(b["quant"], b["h"], b["q"], b["q_scale"])
        dlf_gemm_blocks(b["second"], b["q"], b["q_scale"], *self.down, None, x, y, b["ws"], b["ws"].numel())
