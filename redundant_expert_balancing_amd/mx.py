"""Serving layer whose experts are held in 4 bits (moonep.h, "Experts in 4 bits"), and its
hot path as a sequence of library calls (no computation here).

Set-up  : quantise_weights(w), once
Forward : plan -> prefetch -> quantise(x), one row per token -> grouped GEMM, which reads
          each position's token through src_index (nothing is permuted) -> combine
"""
from __future__ import annotations

import torch

from . import _lib as L


def buffers(rows: int, width: int, device="cuda"):
    """(q, scales) of `rows` token rows of `width` values."""
    qb, sb = L.mx_row_bytes(width)
    u8 = dict(dtype=torch.uint8, device=device)
    return torch.empty((max(rows, 1), qb), **u8), torch.empty((max(rows, 1), sb), **u8)


def weight_buffers(rows: int, H: int, Hp: int, device="cuda"):
    """(q, scales) of `rows` experts' weights [H, Hp]."""
    T, C = -(-H // 128), -(-H // 512)
    u8 = dict(dtype=torch.uint8, device=device)
    return (torch.empty((rows, Hp // 16, T, 64, 16), **u8),
            torch.empty((rows, Hp // 16, C, 64, 4), **u8))


class _MXBase:
    """Plan buffers and the workspace of a layer on `shapes` (the largest workspace first)."""

    def __init__(self, cfg, shapes, device):
        for sh in shapes:
            st = L.moonep_validate_shape(sh)
            if st != L.OK:
                raise L.MoonepError("moonep_validate_shape", st)
            if sh.H % 64 or sh.Hp % 64:
                raise L.MoonepError(f"{type(self).__name__} (H and H' must be multiples of 64)",
                                    L.EINVAL)
        c = self.cfg = cfg
        self.device = torch.device(device)
        self.dtype = torch.bfloat16 if c.dtype == "bf16" else torch.float32
        i32 = dict(dtype=torch.int32, device=self.device)
        NK = max(c.R * c.S * c.K, 1)
        self.cu_seqlens = torch.empty((c.R, c.E + c.B + 1), **i32)
        self.replica_expert = torch.empty((c.R, max(c.B, 1)), **i32)
        self.slot_map = torch.empty((NK,), **i32)
        self.src_index = torch.empty((NK,), **i32)
        self.ws = torch.empty((max(L.moonep_workspace_bytes(sh) for sh in shapes) // 4,), **i32)
        L.moonep_workspace_init(shapes[0], self.ws)
        self.xq, self.xs = buffers(c.R * c.S, c.H, self.device)

    def quantise(self, x, stream=None):
        c = self.cfg
        L.moonep_mx_quantize(self.shape, c.R * c.S, c.H, x, self.xq, self.xs, stream)

    def error_flags(self, clear=False) -> int:
        return L.moonep_get_error(self.shape, self.ws, clear)


class MXProjection(_MXBase):
    """One expert projection [H, H'] with 4-bit weights of E + R*B rows (wq, wscales)."""

    def __init__(self, cfg, device="cuda"):
        c = cfg
        self.shape = L.Shape.of(c)
        super().__init__(c, (self.shape,), device)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.wq, self.wscales = weight_buffers(c.E + c.R * c.B, c.H, c.Hp, self.device)
        self.out = torch.empty((max(c.R * c.S * c.K, 1), c.Hp), **f32)
        self.y = torch.empty((max(c.R * c.S, 1), c.Hp), **f32)

    def quantise_weights(self, w, stream=None):
        """w dtype [E, H, H']: the home experts."""
        L.moonep_mx_quantize_weight(self.shape, w, self.wq, self.wscales, stream)

    def plan(self, topk_idx, stream=None):
        L.moonep_plan(self.shape, topk_idx, self.cu_seqlens, self.replica_expert, self.slot_map,
                      self.src_index, self.ws, stream)

    def prefetch(self, stream=None):
        L.moonep_mx_prefetch_weight(self.shape, self.replica_expert, self.wq, self.wscales, stream)

    def gemm(self, stream=None):
        L.moonep_mx_grouped_gemm(self.shape, self.xq, self.xs, self.src_index, self.wq,
                                 self.wscales, self.cu_seqlens, self.out, self.ws, stream)

    def combine(self, gates, stream=None):
        L.moonep_combine(self.shape, self.cfg.Hp, self.out, self.slot_map, gates, self.y, stream)

    def forward(self, topk_idx, x, gates, stream=None):
        self.plan(topk_idx, stream)
        self.prefetch(stream)
        self.quantise(x, stream)
        self.gemm(stream)
        self.combine(gates, stream)
        return self.y


class MXFFN(_MXBase):
    """The full expert FFN with 4-bit W1 (gate/up columns interleaved in 32-column blocks)
    and W2: gate/up GEMM -> SwiGLU -> act in 4 bits -> down GEMM -> combine."""

    def __init__(self, cfg, device="cuda"):
        c = cfg
        mode = L.TRAIN if c.mode == "train" else L.INFER
        dt = L.BF16 if c.dtype == "bf16" else L.FP32
        self.shape, self.up, self.down = (L.Shape(c.R, c.S, c.E, c.K, c.B, h, hp, mode, dt)
                                          for h, hp in ((c.H, c.Hp), (c.H, 2 * c.Hp), (c.Hp, c.H)))
        super().__init__(c, (self.up, self.down, self.shape), device)
        rows, W = max(c.R * c.S * c.K, 1), c.E + c.R * c.B
        f32 = dict(dtype=torch.float32, device=self.device)
        self.w1q, self.w1s = weight_buffers(W, c.H, 2 * c.Hp, self.device)
        self.w2q, self.w2s = weight_buffers(W, c.Hp, c.H, self.device)
        self.h = torch.empty((rows, 2 * c.Hp), **f32)
        self.act = torch.empty((rows, c.Hp), dtype=self.dtype, device=self.device)
        self.aq, self.as_ = buffers(rows, c.Hp, self.device)
        self.z = torch.empty((rows, c.H), **f32)
        self.y = torch.empty((max(c.R * c.S, 1), c.H), **f32)

    def quantise_weights(self, w1, w2, stream=None):
        """w1 dtype [E, H, 2H'], w2 dtype [E, H', H]: the home experts."""
        L.moonep_mx_quantize_weight(self.up, w1, self.w1q, self.w1s, stream)
        L.moonep_mx_quantize_weight(self.down, w2, self.w2q, self.w2s, stream)

    def plan(self, topk_idx, stream=None):
        L.moonep_plan(self.up, topk_idx, self.cu_seqlens, self.replica_expert, self.slot_map,
                      self.src_index, self.ws, stream)

    def prefetch(self, stream=None):
        L.moonep_mx_prefetch_weight(self.up, self.replica_expert, self.w1q, self.w1s, stream)
        L.moonep_mx_prefetch_weight(self.down, self.replica_expert, self.w2q, self.w2s, stream)

    def gate_up(self, stream=None):
        c = self.cfg
        L.moonep_mx_grouped_gemm(self.up, self.xq, self.xs, self.src_index, self.w1q, self.w1s,
                                 self.cu_seqlens, self.h, self.ws, stream)
        L.moonep_swiglu(self.shape, self.h, self.act, None, stream)
        L.moonep_mx_quantize(self.shape, c.R * c.S * c.K, c.Hp, self.act, self.aq, self.as_, stream)

    def down_proj(self, stream=None):
        L.moonep_mx_grouped_gemm(self.down, self.aq, self.as_, None, self.w2q, self.w2s,
                                 self.cu_seqlens, self.z, self.ws, stream)

    def combine(self, gates, stream=None):
        L.moonep_combine(self.up, self.cfg.H, self.z, self.slot_map, gates, self.y, stream)

    def forward(self, topk_idx, x, gates, stream=None):
        self.plan(topk_idx, stream)
        self.prefetch(stream)
        self.quantise(x, stream)
        self.gate_up(stream)
        self.down_proj(stream)
        self.combine(gates, stream)
        return self.y
