"""The compiled binding of the 8-bit integer calls, on the CPU: what it takes as a number, and
what it needs to be built."""
import numpy as np
import pytest
import torch

from redundant_expert_balancing_amd import _lib as L


def _shape():
    return L.Shape(4, 64, 16, 2, 4, 128, 64, L.TRAIN, L.BF16)


CALLS = {
    "quantize rows": lambda n: L.moonep_int_quantize(_shape(), n, 128, *(torch.zeros(4),) * 3),
    "quantize width": lambda n: L.moonep_int_quantize(_shape(), 4, n, *(torch.zeros(4),) * 3),
    "gemm": lambda n: L.moonep_int_gemm(_shape(), n, *(torch.zeros(4),) * 6),
    "gemm_swiglu": lambda n: L.moonep_int_gemm_swiglu(_shape(), n, *(torch.zeros(4),) * 6),
}


@pytest.mark.parametrize("call", CALLS)
def test_numbers_are_whole_numbers(call):
    """Nothing is cut to a whole number: a row count that came out as a float is refused."""
    for bad in (4.0, 4.9, np.float32(4), torch.tensor(4.5), None, [4]):
        with pytest.raises(TypeError):
            CALLS[call](bad)
    for bad in ("4", "four", b"4"):
        with pytest.raises((TypeError, ValueError)) as e:
            CALLS[call](bad)
        assert "GPU tensor" not in str(e.value)
    with pytest.raises(OverflowError):
        CALLS[call](1 << 70)
    for good in (4, True, np.int32(4), np.int64(4), torch.tensor(4)):        # on to the tensors
        with pytest.raises(ValueError, match="GPU tensor"):
            CALLS[call](good)


@pytest.mark.slow
def test_the_binding_builds_with_the_compiler_beside_hipcc(monkeypatch, tmp_path):
    """No host compiler on the path: hipcc alone builds the library, so its own C++ compiler builds
    the binding."""
    import importlib.util

    from redundant_expert_balancing_amd import build
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setenv("PATH", str(tmp_path))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    path = build.build_binding()
    spec = importlib.util.spec_from_file_location("_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert all(hasattr(module, n) for n in ("bind", *L._INT_CALLS))


def test_shared_weights_go_with_a_shared_expert():
    """A layer without a shared expert does not drop its weights, one with it does not go without."""
    from redundant_expert_balancing_amd.int8 import IntFFN
    w = torch.zeros(4)
    for shared, s1, s2 in ((0, w, w), (0, w, None), (0, None, w), (64, None, None), (64, w, None), (64, None, w)):
        l = IntFFN.__new__(IntFFN)          # no GPU here: the rule comes before everything else
        l.shared = shared
        with pytest.raises(ValueError, match="shared expert"):
            l.quantise_weights(w, w, s1, s2)
