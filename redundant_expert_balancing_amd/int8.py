"""Layers whose experts are held in 8-bit integers (moonep.h, "Experts in 8-bit integers"), and
their hot path as a sequence of library calls (no computation here).

Set-up  : quantise_weights(w), once
Forward : plan -> prefetch -> quantise(x), one row per token -> grouped GEMM, which reads
          each position's token through src_index (nothing is permuted) -> combine

IntFFN can have a shared expert, an FFN of its own intermediate size that every token passes
besides its routed experts: its down projection adds to the combined output.

With backward=True an IntFFN gives the gradient of x (and of the gates, for the router's
backward) through its experts, which stay as they are: the upstream rows times the scales of
their expert's columns are held in 8 bits too, and multiplied with the transposed weights.
  quantise_grad(dy, gates) -> product with W2^T -> SwiGLU backward -> quantise_grad(dh)
  -> product with W1^T -> combine(dxp, no gates)
"""
from __future__ import annotations

import torch

from . import _lib as L


def buffers(rows: int, width: int, device="cuda"):
    """(q, scales) of `rows` token rows of `width` values."""
    return (torch.empty((max(rows, 1), L.int_row_bytes(width)), dtype=torch.int8, device=device),
            torch.empty((max(rows, 1),), dtype=torch.float32, device=device))


def weight_buffers(rows: int, H: int, Hp: int, device="cuda"):
    """(q, scales) of `rows` experts' weights [H, Hp]."""
    NB = -(-Hp // 16)
    return (torch.empty((rows, NB, 2 * -(-H // 128), 64, 16), dtype=torch.int8, device=device),
            torch.empty((rows, NB * 16), dtype=torch.float32, device=device))


class _IntBase:
    """Plan buffers and the workspace of a layer on `shapes` (the largest workspace first)."""

    def __init__(self, cfg, shapes, device):
        for sh in shapes:
            st = L.moonep_validate_shape(sh)
            if st != L.OK:
                raise L.MoonepError("moonep_validate_shape", st)
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
        L.moonep_int_quantize(self.shape, c.R * c.S, c.H, x, self.xq, self.xs, stream)

    def error_flags(self, clear=False) -> int:
        return L.moonep_get_error(self.shape, self.ws, clear)


class IntProjection(_IntBase):
    """One expert projection [H, H'] with 8-bit weights of E + R*B rows (wq, wscales)."""

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
        L.moonep_int_quantize_weight(self.shape, w, self.wq, self.wscales, stream)

    def plan(self, topk_idx, stream=None):
        L.moonep_plan(self.shape, topk_idx, self.cu_seqlens, self.replica_expert, self.slot_map,
                      self.src_index, self.ws, stream)

    def prefetch(self, stream=None):
        L.moonep_int_prefetch_weight(self.shape, self.replica_expert, self.wq, self.wscales, stream)

    def gemm(self, stream=None):
        L.moonep_int_grouped_gemm(self.shape, self.xq, self.xs, self.src_index, self.wq,
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


class IntFFN(_IntBase):
    """The full expert FFN with 8-bit W1 (gate/up columns interleaved in 32-column blocks) and
    W2: gate/up GEMM with SwiGLU -> act in 8 bits -> down GEMM -> combine (-> shared expert of
    intermediate size `shared`, its output added). backward=True: see the module."""

    def __init__(self, cfg, device="cuda", shared: int = 0, backward: bool = False):
        c = cfg
        mode = L.TRAIN if c.mode == "train" else L.INFER
        dt = L.BF16 if c.dtype == "bf16" else L.FP32
        if backward and mode != L.TRAIN:
            raise L.MoonepError("IntFFN (backward of an inference layer)", L.EMODE)
        if c.Hp % L.SWIGLU_BLOCK or shared % L.SWIGLU_BLOCK or shared < 0:
            raise L.MoonepError("IntFFN (H' and shared must be multiples of 32)", L.EINVAL)
        # the products (H, 2H') and (H', H), and back through them
        self.shape, self.up, self.down, self.up_back, self.down_back = (
            L.Shape(c.R, c.S, c.E, c.K, c.B, h, hp, mode, dt)
            for h, hp in ((c.H, c.Hp), (c.H, 2 * c.Hp), (c.Hp, c.H), (2 * c.Hp, c.H), (c.H, c.Hp)))
        super().__init__(c, (self.up, self.down, self.shape), device)
        self.backward_pass, self.shared = backward, shared
        N, rows, W = c.R * c.S, max(c.R * c.S * c.K, 1), c.E + c.R * c.B
        f32 = dict(dtype=torch.float32, device=self.device)
        dtd = dict(dtype=self.dtype, device=self.device)
        self.w1q, self.w1s = weight_buffers(W, c.H, 2 * c.Hp, self.device)
        self.w2q, self.w2s = weight_buffers(W, c.Hp, c.H, self.device)
        self.act = torch.empty((rows, c.Hp), **dtd)
        self.aq, self.as_ = buffers(rows, c.Hp, self.device)
        self.z = torch.empty((rows, c.H), **f32)
        self.y = torch.empty((max(N, 1), c.H), **f32)
        self.hs = None
        if backward:
            self.hs = torch.empty((rows, 2 * c.Hp), **dtd)
            self.w1t, _ = weight_buffers(W, 2 * c.Hp, c.H, self.device)
            self.w2t, _ = weight_buffers(W, c.H, c.Hp, self.device)
            self.dyq, self.dys = buffers(rows, c.H, self.device)
            self.da = torch.empty((rows, c.Hp), **f32)
            self.dh = torch.empty((rows, 2 * c.Hp), **dtd)
            self.dhq, self.dhs = buffers(rows, 2 * c.Hp, self.device)
            self.dxp = torch.empty((rows, c.H), **f32)
            self.dx = torch.empty((max(N, 1), c.H), **f32)
            self.dgates = torch.empty((max(N, 1), c.K), **f32)
        if not shared:
            return
        # the shared expert: a layer of one expert on one rank, whose plan is the identity
        B = 1 if mode == L.TRAIN else 0
        self.s_shape, self.s_up, self.s_down, self.s_up_back, self.s_down_back = (
            L.Shape(1, N, 1, 1, B, h, hp, mode, dt)
            for h, hp in ((c.H, shared), (c.H, 2 * shared), (shared, c.H), (2 * shared, c.H),
                          (c.H, shared)))
        n = max(N, 1)
        self.s1q, self.s1s = weight_buffers(1, c.H, 2 * shared, self.device)
        self.s2q, self.s2s = weight_buffers(1, shared, c.H, self.device)
        self.s_act = torch.empty((n, shared), **dtd)
        self.s_aq, self.s_as = buffers(N, shared, self.device)
        self.s_hs = None
        if backward:
            self.s_hs = torch.empty((n, 2 * shared), **dtd)
            self.s1t, _ = weight_buffers(1, 2 * shared, c.H, self.device)
            self.s2t, _ = weight_buffers(1, c.H, shared, self.device)
            self.s_dyq, self.s_dys = buffers(N, c.H, self.device)
            self.s_da = torch.empty((n, shared), **f32)
            self.s_dh = torch.empty((n, 2 * shared), **dtd)
            self.s_dhq, self.s_dhs = buffers(N, 2 * shared, self.device)

    def quantise_weights(self, w1, w2, s1=None, s2=None, stream=None):
        """w1 dtype [E, H, 2H'], w2 dtype [E, H', H]: the home experts; s1 [H, 2*shared] and s2
        [shared, H]: the shared expert, of a layer that has one."""
        if (s1 is None, s2 is None) != (not self.shared,) * 2:
            raise ValueError("s1, s2: both, of a layer with a shared expert, and neither otherwise")
        L.moonep_int_quantize_weight(self.up, w1, self.w1q, self.w1s, stream)
        L.moonep_int_quantize_weight(self.down, w2, self.w2q, self.w2s, stream)
        if self.shared:
            L.moonep_int_quantize_weight(self.s_up, s1, self.s1q, self.s1s, stream)
            L.moonep_int_quantize_weight(self.s_down, s2, self.s2q, self.s2s, stream)
        if self.backward_pass:
            L.moonep_int_transpose_weight(self.up, self.w1q, self.w1t, stream)
            L.moonep_int_transpose_weight(self.down, self.w2q, self.w2t, stream)
            if self.shared:
                L.moonep_int_transpose_weight(self.s_up, self.s1q, self.s1t, stream)
                L.moonep_int_transpose_weight(self.s_down, self.s2q, self.s2t, stream)

    def plan(self, topk_idx, stream=None):
        L.moonep_plan(self.up, topk_idx, self.cu_seqlens, self.replica_expert, self.slot_map,
                      self.src_index, self.ws, stream)

    def prefetch(self, stream=None):
        r = self.replica_expert
        L.moonep_int_prefetch_weight(self.up, r, self.w1q, self.w1s, stream)
        L.moonep_int_prefetch_weight(self.down, r, self.w2q, self.w2s, stream)
        if self.backward_pass:
            L.moonep_int_prefetch_weight(self.up_back, r, self.w1t, None, stream)
            L.moonep_int_prefetch_weight(self.down_back, r, self.w2t, None, stream)

    def gate_up(self, stream=None):
        c = self.cfg
        L.moonep_int_grouped_gemm_swiglu(self.shape, self.xq, self.xs, self.src_index, self.w1q,
                                         self.w1s, self.cu_seqlens, self.act, self.hs, self.ws,
                                         stream)
        L.moonep_int_quantize(self.shape, c.R * c.S * c.K, c.Hp, self.act, self.aq, self.as_, stream)

    def down_proj(self, stream=None):
        L.moonep_int_grouped_gemm(self.down, self.aq, self.as_, None, self.w2q, self.w2s,
                                  self.cu_seqlens, self.z, self.ws, stream)

    def combine(self, gates, stream=None):
        L.moonep_combine(self.up, self.cfg.H, self.z, self.slot_map, gates, self.y, stream)

    def shared_expert(self, stream=None):
        """y += the shared expert's output."""
        N = self.cfg.R * self.cfg.S
        L.moonep_int_gemm_swiglu(self.s_shape, N, self.xq, self.xs, self.s1q, self.s1s, self.s_act,
                                 self.s_hs, stream)
        L.moonep_int_quantize(self.s_shape, N, self.shared, self.s_act, self.s_aq, self.s_as, stream)
        L.moonep_int_gemm(self.s_down, N, self.s_aq, self.s_as, self.s2q, self.s2s, self.y, self.y,
                          stream)

    def forward(self, topk_idx, x, gates, stream=None):
        self.plan(topk_idx, stream)
        self.prefetch(stream)
        self.quantise(x, stream)
        self.gate_up(stream)
        self.down_proj(stream)
        self.combine(gates, stream)
        if self.shared:
            self.shared_expert(stream)
        return self.y

    # ---- backward
    def gate_grad(self, dy, stream=None):
        """Gradient of the gates [N,K], from the forward's outputs and dy."""
        L.moonep_gate_grad(self.up, self.cfg.H, self.z, self.slot_map, dy, self.dgates, stream)
        return self.dgates

    def backward(self, dy, gates, stream=None):
        """dx float32 [N, H] through the last forward's experts; dy dtype [N, H]."""
        c = self.cfg
        L.moonep_int_quantize_grad(self.down, dy, self.src_index, gates, self.w2s, self.cu_seqlens,
                                   self.dyq, self.dys, stream)
        L.moonep_int_grouped_gemm(self.down_back, self.dyq, self.dys, None, self.w2t, None,
                                  self.cu_seqlens, self.da, self.ws, stream)
        L.moonep_swiglu_backward(self.shape, self.hs, self.da, self.dh, stream)
        L.moonep_int_quantize_grad(self.up, self.dh, None, None, self.w1s, self.cu_seqlens,
                                   self.dhq, self.dhs, stream)
        L.moonep_int_grouped_gemm(self.up_back, self.dhq, self.dhs, None, self.w1t, None,
                                  self.cu_seqlens, self.dxp, self.ws, stream)
        L.moonep_combine(self.up, c.H, self.dxp, self.slot_map, None, self.dx, stream)
        if self.shared:
            N = c.R * c.S
            L.moonep_int_quantize_grad(self.s_down, dy, None, None, self.s2s, None, self.s_dyq,
                                       self.s_dys, stream)
            L.moonep_int_gemm(self.s_down_back, N, self.s_dyq, self.s_dys, self.s2t, None, None,
                              self.s_da, stream)
            L.moonep_swiglu_backward(self.s_shape, self.s_hs, self.s_da, self.s_dh, stream)
            L.moonep_int_quantize_grad(self.s_up, self.s_dh, None, None, self.s1s, None,
                                       self.s_dhq, self.s_dhs, stream)
            L.moonep_int_gemm(self.s_up_back, N, self.s_dhq, self.s_dhs, self.s1t, None, self.dx,
                              self.dx, stream)
        return self.dx
