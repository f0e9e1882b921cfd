"""Buffers of an 8-bit activation checkpoint (moonep.h, "8-bit activation checkpoints")."""
from __future__ import annotations

import torch

from . import _lib as L


def buffers(rows: int, width: int, device="cuda"):
    """(q uint8 [rows, width], scales uint8 [rows, 4*ceil(width/128)]) of a checkpoint."""
    u8 = dict(dtype=torch.uint8, device=device)
    return (torch.empty((max(rows, 1), width), **u8),
            torch.empty((max(rows, 1), L.checkpoint_scale_bytes(width)), **u8))
