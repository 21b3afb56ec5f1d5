"""The entry points between the layers of a step (norm with the 8-bit cast) on
the CPU: declared, and bad arguments rejected on the host before anything would
reach a GPU.  Nothing here launches a kernel."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.test_abi import A1, A16, INVALID, MISALIGNED, NUL, P, S, SHAPE, L, declared_symbols  # noqa: F401

A8 = P(0x10008)


def test_entry_points_are_declared():
    names = declared_symbols()
    for n in ("fp8_rmsnorm_quant_act", "fp8_mx_rmsnorm_quant_act"):
        assert n in names


@pytest.mark.parametrize("name", ["fp8_rmsnorm_quant_act", "fp8_mx_rmsnorm_quant_act"])
def test_norm_validation(L, name):
    def call(x=A16, ldx=512, res=A16, ldr=512, out=A16, ldo=512, gamma=A16, gt=1, eps=1e-5, M=8, K=512, y=NUL, xq=A16,
             xs=A16, flags=0):
        return getattr(L, name)(x, ldx, res, ldr, out, ldo, gamma, gt, eps, M, K, y, xq, xs, flags, S)

    for nul in ("x", "gamma", "xq", "xs"):
        assert call(**{nul: NUL}) == INVALID
    assert call(res=NUL) == INVALID and call(out=NUL) == INVALID      # both or neither
    assert call(res=NUL, out=NUL) not in (INVALID, SHAPE, MISALIGNED)
    assert call(M=0) == INVALID and call(K=0) == INVALID and call(gt=2) == INVALID
    assert call(ldx=256) == INVALID and call(ldr=256) == INVALID and call(ldo=256) == INVALID
    for eps in (0.0, -1.0, 1e-31, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    assert call(flags=2) == INVALID
    assert call(K=500, ldx=504, ldr=504, ldo=504) == SHAPE
    assert call(K=32896, ldx=32896, ldr=32896, ldo=32896) == SHAPE
    assert (call(M=513) == SHAPE) == (name == "fp8_mx_rmsnorm_quant_act")
    for mis in ("x", "res", "out", "gamma", "y", "xq"):
        assert call(**{mis: A8}) == MISALIGNED
    assert call(xs=A1) == MISALIGNED
    for ld in ("ldx", "ldr", "ldo"):
        assert call(**{ld: 516}) == MISALIGNED


@pytest.mark.parametrize("bad", [[[1.0, 2.0]], np.zeros((2, 128), np.float32), None, 3, "x"])
def test_the_first_argument_has_to_be_a_tensor(bad):
    for call in (fb.fp8_rmsnorm_quant_act, fb.fp8_mx_rmsnorm_quant_act):
        with pytest.raises(TypeError, match="^x must be"):
            call(bad, None)


def test_a_tensor_on_the_cpu_is_refused_as_such():
    for call in (fb.fp8_rmsnorm_quant_act, fb.fp8_mx_rmsnorm_quant_act):
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(128))
