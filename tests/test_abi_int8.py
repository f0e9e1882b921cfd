"""Argument checks of the 8-bit integer experts: every refusal comes back before a launch (no
GPU call is made here)."""
import ctypes
import dataclasses

import pytest
import torch

from redundant_expert_balancing_amd import _lib as L

P = ctypes.c_void_p(0x1000)       # aligned, never dereferenced
BAD = ctypes.c_void_p(0x1008)
BIG = 1 << 40
LONG = 131080                     # a reduction that could overflow int32
WIDE = (1 << 24) + 32             # more columns than a weight may have


def S(**kw):
    base = dict(R=4, S=64, E=16, K=2, B=4, H=128, Hp=64, mode=L.TRAIN, dtype=L.BF16)
    base.update(kw)
    return L.Shape(*[base[k] for k in ("R", "S", "E", "K", "B", "H", "Hp", "mode", "dtype")])


def call(name, sh, *args):
    return getattr(L.lib(), "moonep_int_" + name)(ctypes.byref(sh), *args, None)


def broken(good, at, bad=(BAD, None)):
    """The pointers `good` with one at a time replaced, at the places `at`."""
    for i in at:
        for b in bad:
            yield good[:i] + (b,) + good[i + 1:]


def test_quantise_rules():
    sh = S()
    assert call("quantize", sh, -1, 128, P, P, P) == L.EINVAL
    assert call("quantize", sh, 1 << 31, 128, P, P, P) == L.EINVAL
    assert call("quantize", sh, 4, 0, P, P, P) == L.EINVAL
    assert call("quantize", sh, 4, 44, P, P, P) == L.EINVAL
    assert call("quantize", S(dtype=L.FP32), 4, 42, P, P, P) == L.EINVAL
    assert call("quantize", sh, 4, LONG, P, P, P) == L.ELIMIT
    assert call("quantize", sh, 0, 128, None, None, None) == L.OK
    assert call("quantize", S(E=18), 0, 128, None, None, None) == L.EINVAL
    for p in broken((P, P, P), range(3)):
        assert call("quantize", sh, 4, 128, *p) == L.EINVAL


def test_weight_rules():
    sh = S()
    for name, n in (("quantize_weight", 3), ("transpose_weight", 2)):
        for p in broken((P,) * n, range(n)):
            assert call(name, sh, *p) == L.EINVAL
        assert call(name, S(H=LONG), *(P,) * n) == L.ELIMIT
        assert call(name, S(H=100), *(P,) * n) == L.EINVAL
    assert call("transpose_weight", S(Hp=LONG), P, P) == L.ELIMIT
    for p in broken((P, P, P), (0, 1)):
        assert call("prefetch_weight", sh, *p) == L.EINVAL
    assert call("prefetch_weight", sh, P, P, BAD) == L.EINVAL
    assert call("prefetch_weight", S(mode=L.INFER, B=0), None, None, None) == L.OK
    assert call("quantize_weight", S(Hp=WIDE), P, P, P) == L.ELIMIT
    assert call("prefetch_weight", S(Hp=WIDE), P, P, P) == L.ELIMIT


def test_grouped_rules():
    sh = S()
    good = (P,) * 8               # xq, xscales, src_index, wq, wscales, cu_seqlens, c, ws
    for p in list(broken(good, (0, 1, 3, 5, 6, 7))) + list(broken(good, (2, 4), (BAD,))):
        assert call("grouped_gemm", sh, *p, BIG) == L.EINVAL
    assert call("grouped_gemm", sh, *good, 16) == L.EWORKSPACE
    assert call("grouped_gemm", S(H=LONG), *good, BIG) == L.ELIMIT
    assert call("grouped_gemm", S(Hp=WIDE), *good, BIG) == L.ELIMIT
    assert call("grouped_gemm", S(H=100), *good, BIG) == L.EINVAL
    empty = (None,) * 5 + (P, None, P)
    assert call("grouped_gemm", S(S=0), *empty, BIG) == L.OK
    good = (P,) * 9               # xq, xscales, src_index, wq, wscales, cu, act, h_saved, ws
    for p in list(broken(good, (0, 1, 3, 5, 6, 8))) + list(broken(good, (2, 4, 7), (BAD,))):
        assert call("grouped_gemm_swiglu", sh, *p, BIG) == L.EINVAL
    assert call("grouped_gemm_swiglu", sh, *good, 16) == L.EWORKSPACE
    assert call("grouped_gemm_swiglu", S(Hp=48), *good, BIG) == L.EINVAL
    assert call("grouped_gemm_swiglu", S(Hp=1 << 30), *good, BIG) == L.ELIMIT    # 2 Hp past int32
    assert call("grouped_gemm_swiglu", S(H=LONG), *good, BIG) == L.ELIMIT
    empty = (None,) * 5 + (P, None, None, P)
    assert call("grouped_gemm_swiglu", S(S=0), *empty, BIG) == L.OK


def test_dense_rules():
    sh = S()
    for name in ("gemm", "gemm_swiglu"):
        # xq, xscales, wq, wscales, then add, c or act, h_saved
        must, may = ((0, 1, 2, 5), (3, 4)) if name == "gemm" else ((0, 1, 2, 4), (3, 5))
        good = (P,) * 6
        for p in list(broken(good, must)) + list(broken(good, may, (BAD,))):
            assert call(name, sh, 4, *p) == L.EINVAL
        assert call(name, sh, -1, *good) == L.EINVAL
        assert call(name, sh, 1 << 31, *good) == L.EINVAL
        assert call(name, S(H=LONG), 4, *good) == L.ELIMIT
        assert call(name, S(Hp=WIDE), 4, *good) == L.ELIMIT
        assert call(name, sh, 0, *(None,) * 6) == L.OK
    assert call("gemm_swiglu", S(Hp=48), 4, *(P,) * 6) == L.EINVAL


def test_gradient_rules():
    sh = S()
    good = (P,) * 7               # src, src_index, gates, wscales, cu_seqlens, q, scales
    for p in list(broken(good, (0, 3, 5, 6))) + list(broken(good, (1, 2, 4), (BAD,))):
        assert call("quantize_grad", sh, *p) == L.EINVAL
    assert call("quantize_grad", sh, P, None, P, P, P, P, P) == L.EINVAL     # gates, no src_index
    assert call("quantize_grad", S(mode=L.INFER, B=2), *good) == L.EMODE
    assert call("quantize_grad", S(Hp=LONG), *good) == L.ELIMIT
    assert call("quantize_grad", S(S=0), *(None,) * 7) == L.OK


def test_binding_refuses_host_missing_and_small_tensors():
    sh = S()
    f = torch.zeros((256, 16))
    with pytest.raises(ValueError, match="GPU tensor"):
        L.moonep_int_quantize(sh, 4, 128, f, f, f)
    with pytest.raises(ValueError, match="required"):
        L.moonep_int_gemm(sh, 4, None, f, f, f, None, f)
    with pytest.raises(ValueError, match="required"):
        L.moonep_int_grouped_gemm(sh, None, f, None, f, f, f, f, f)


def test_layer_arguments():
    from redundant_expert_balancing_amd.int8 import IntFFN
    from redundant_expert_balancing_amd.synth import CONFIGS
    cfg = CONFIGS["tiny_fp32_train"]
    with pytest.raises(L.MoonepError):
        IntFFN(dataclasses.replace(cfg, Hp=48), device="cpu")
    with pytest.raises(L.MoonepError):
        IntFFN(cfg, device="cpu", shared=40)
    with pytest.raises(L.MoonepError):
        IntFFN(dataclasses.replace(cfg, mode="infer"), device="cpu", backward=True)
