"""The entry points between the layers of a step (norm with the 8-bit cast,
verification of drafted tokens) on
the CPU: declared, and bad arguments rejected on the host before anything would
reach a GPU.  Nothing here launches a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.test_abi import A1, A16, INVALID, MISALIGNED, NUL, OK, P, S, SHAPE, L, declared_symbols  # noqa: F401
from tests.verify_reference import verify

A8 = P(0x10008)


def test_entry_points_are_declared():
    names = declared_symbols()
    for n in ("fp8_rmsnorm_quant_act", "fp8_mx_rmsnorm_quant_act", "speculative_verify", "speculative_verify_workspace_size"):
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


def test_verify_validation(L):
    def call(x=A16, xt=1, ldl=512, draft=A16, dlen=NUL, q=NUL, ldq=512, au=A16, su=A16, T=NUL, B=2, n=3, V=512, tok=A16,
             acc=A16, probs=A16, ws=A16, size=1 << 40, flags=0):
        return L.speculative_verify(x, xt, ldl, draft, dlen, q, ldq, au, su, T, B, n, V, tok, acc, probs, ws, size, flags, S)

    fine = (INVALID, SHAPE, MISALIGNED)
    assert call() not in fine and call(n=0, draft=NUL, au=NUL) not in fine and call(dlen=A16, q=A16, T=A16) not in fine
    for nul in ("x", "draft", "au", "su", "tok", "acc", "probs", "ws"):
        assert call(**{nul: NUL}) == INVALID
    assert call(xt=2) == INVALID and call(ldl=511) == INVALID and call(q=A16, ldq=511) == INVALID and call(flags=2) == INVALID
    assert call(B=0) == INVALID and call(n=-1) == INVALID and call(V=0) == INVALID
    for extra in (dict(draft=A16), dict(au=A16), dict(dlen=A16), dict(q=A16)):  # no draft, but something of one
        assert call(**{**dict(n=0, draft=NUL, au=NUL), **extra}) == INVALID
    assert call(n=32) == SHAPE and call(B=1025) == SHAPE and call(V=1048577, ldl=1048577) == SHAPE
    for mis in ("draft", "dlen", "q", "au", "su", "T", "tok", "acc", "probs", "x"):
        assert call(**{mis: A1}) == MISALIGNED
    assert call(x=P(0x10002)) not in fine and call(x=P(0x10002), xt=0) == MISALIGNED
    assert call(ws=P(0x10080)) == MISALIGNED
    sz = ctypes.c_size_t(3)
    assert L.speculative_verify_workspace_size(2, 32, 512, ctypes.byref(sz)) == SHAPE and sz.value == 0
    assert L.speculative_verify_workspace_size(64, 7, 248320, ctypes.byref(sz)) == OK and sz.value > 512 * 31 * 16
    assert L.speculative_verify_workspace_size(1, 0, 1, None) == INVALID


def test_the_reference_of_the_verification():
    """Hand-worked: p = (1/2, 1/4, 1/4); q = (1/4, 1/4, 1/2), so that p - q leaves
    the first token alone; a certain draft; T = 0."""
    x = np.log(np.array([[2.0, 1.0, 1.0]] * 2))
    q = np.array([[0.25, 0.25, 0.5]])
    u = np.array([0.7])

    def run(draft, a, **kw):
        return verify(x, u, np.array([[draft]]), np.array([[a]]), **kw)[:2]
    tok, acc = run(2, 0.49, draft_probs=q)          # 0.49 * 0.5 < 0.25
    assert acc.tolist() == [1] and tok.tolist() == [[2, 1]]   # 0.7: past 1/2, before 3/4
    tok, acc = run(2, 0.51, draft_probs=q)
    assert acc.tolist() == [0] and tok.tolist() == [[0, -1]]
    tok, acc = run(0, 0.51)                          # certain: accepted below p = 1/2
    assert acc.tolist() == [0] and tok.tolist() == [[2, -1]]  # (1/4, 1/4) are left, 0.7 is in the second
    assert run(0, 0.49)[1].tolist() == [1]
    tok, acc = run(1, 0.0, temperature=np.array([0.0]))
    assert acc.tolist() == [0] and tok.tolist() == [[0, -1]]
