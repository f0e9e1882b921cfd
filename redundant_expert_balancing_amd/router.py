"""Device buffers of a layer's router and its calls (no computation here): from the
router's logits to the plan's topk_idx and gates, and from the gates' gradient back.

Forward  : route(logits) -> topk_idx, gates, for MoEProjection / MoEFFN forward
Backward : gates' gradient (gate_grad of the layer) -> dlogits
Buffer layout: topk_idx int32 [N,K]; gates fp32 [N,K]; dlogits logits' dtype [N,E].
"""
from __future__ import annotations

import torch

from . import _lib as L


class MoERouter:
    """score: "softmax" or "sigmoid"; groups of consecutive experts of which top_groups stay
    (a group scores the sum of its group_top best); renorm: gates sum to `scale`; dtype of
    the logits. moonep.h (moonep_route) states the rule."""

    def __init__(self, cfg, score: str = "softmax", dtype: str = "fp32", groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
                 device="cuda", backward: bool = False):
        if score not in ("softmax", "sigmoid"):
            raise ValueError(f"unknown score {score!r}")
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f"unknown dtype {dtype!r}")
        self.cfg = cfg
        self.shape = L.Shape.of(cfg)
        st = L.moonep_validate_shape(self.shape)
        if st != L.OK:
            raise L.MoonepError("moonep_validate_shape", st)
        self.router = L.Router(L.SOFTMAX if score == "softmax" else L.SIGMOID,
                               L.BF16 if dtype == "bf16" else L.FP32, groups, top_groups,
                               group_top, int(renorm), scale)
        N = max(cfg.R * cfg.S, 1)
        self.topk_idx = torch.empty((N, cfg.K), dtype=torch.int32, device=device)
        self.gates = torch.empty((N, cfg.K), dtype=torch.float32, device=device)
        if backward:
            self.dlogits = torch.empty((N, cfg.E), device=device,
                                       dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)

    def forward(self, logits, bias=None, stream=None):
        L.moonep_route(self.shape, self.router, logits, bias, self.topk_idx, self.gates, stream)
        return self.topk_idx, self.gates

    def backward(self, logits, dgates, bias=None, stream=None):
        """dlogits, from the logits (and bias) of the last forward."""
        L.moonep_route_backward(self.shape, self.router, logits, bias, self.topk_idx, self.gates,
                                dgates, self.dlogits, stream)
        return self.dlogits
