"""Limits of include/moe_experts.h that a call must not refuse before (no GPU
needed, and no launch where there is one: nothing is placed)."""
import ctypes

import pytest

api = pytest.importorskip("combine_moe_dispatch_amd.api",
                          reason="libmoe_dispatch.so not built")

A = 4096       # an aligned stand-in address, never touched on these paths
UNSUPPORTED = 2


@pytest.mark.parametrize("E,P", [(520, 1 << 22), (1024, 1 << 22), (512, 1 << 22)])
def test_only_a_wanted_bias_gradient_is_limited_by_its_entries(E, P):
    lay = api._Layout(A, A, None, None, None, None, None)
    shape, lin = api._Shape(0, 64, E, 2, 8, 0, 0), api._Linear(8, P, 0)

    def backward(gb):
        return api._lib.moe_expert_matmul_backward(
            ctypes.byref(shape), ctypes.byref(lin), None, None, ctypes.byref(lay), None, None, A,
            None, gb, None, 0, None)

    assert backward(None) != UNSUPPORTED
    if E * P > (1 << 31) - 1:
        assert backward(A) == UNSUPPORTED
