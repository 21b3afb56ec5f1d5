"""The entry points between the layers of a step (norm with the 8-bit cast,
verification of drafted tokens, routing with scores and groups) on
the CPU: declared, and bad arguments rejected on the host before anything would
reach a GPU.  Nothing here launches a kernel."""
import ctypes
import glob
import os
import re

import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.test_abi import A1, A16, INVALID, MISALIGNED, NUL, OK, P, S, SHAPE, L, declared_symbols  # noqa: F401
from tests.route_reference import route
from tests.verify_reference import verify

A8 = P(0x10008)


def test_entry_points_are_declared():
    names = declared_symbols()
    for n in ("fp8_rmsnorm_quant_act", "fp8_mx_rmsnorm_quant_act", "speculative_verify", "speculative_verify_workspace_size",
              "moe_route_grouped", "fp8_moe_layer_grouped"):
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
    for eps in (0.0, -1.0, 1e-31, 1.3e30, float("nan"), float("inf")):
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


def test_grouped_routing_validation(L):
    def route(x=A16, ldx=512, wr=A16, wt=1, bias=NUL, M=8, H=512, E=16, k=2, sc=1, G=4, tg=2, best=2, scale=1.0, ids=A16,
              w=A16, ws=A16, n=1 << 40, flags=0):
        return L.moe_route_grouped(x, ldx, wr, wt, bias, M, H, E, k, sc, G, tg, best, 1, scale, ids, w, ws, n, flags, S)

    def layer(x=A16, ldx=512, wr=A16, wt=1, bias=NUL, M=8, H=512, E=16, k=2, sc=1, G=4, tg=2, best=2, scale=1.0, ids=A16,
              w=A16, ws=A16, n=1 << 40, flags=2, w13=A16, s13=A16, w2=A16, s2=A16, y=A16, I=256):
        return L.fp8_moe_layer_grouped(x, ldx, wr, wt, bias, sc, G, tg, best, 1, scale, w13, s13, w2, s2, y, ids, w, M, H, I,
                                       E, k, ws, n, flags, S)

    fine = (INVALID, SHAPE, MISALIGNED)
    for call in (route, layer):
        assert call() not in fine and call(bias=A16) not in fine and call(G=1, tg=1) not in fine
        for nul in ("x", "wr", "ws"):
            assert call(**{nul: NUL}) == INVALID
        for kw in (dict(wt=2), dict(sc=2), dict(sc=-1), dict(G=0), dict(tg=0), dict(tg=5), dict(best=0), dict(best=3),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(M=0), dict(k=0), dict(ldx=256), dict(flags=4)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(M=65), dict(E=513, G=1, tg=1), dict(k=17, G=1, tg=1), dict(G=3), dict(k=9), dict(G=16, tg=4),
                   dict(E=66, G=33), dict(H=576, ldx=576)):
            assert call(**kw) == SHAPE, kw
        assert call(G=16, tg=16) not in fine  # every group is open: their scores do not matter
        assert call(wr=A8) == MISALIGNED and call(bias=A1) == MISALIGNED and call(ws=P(0x10080)) == MISALIGNED
    assert route(ids=NUL) == INVALID and route(w=NUL) == INVALID and layer(ids=NUL, w=NUL) not in fine
    assert route(flags=2) == INVALID


def test_the_reference_of_the_routing():
    """Hand-worked: four experts in two groups, scores 1/2, 3/4 | 1/4, 4/5."""
    l = np.log(np.array([[1.0, 3.0, 1.0 / 3.0, 4.0]]))
    ids, w, gap = route(l, 2, groups=2, top_groups=1, group_best=2)     # 5/4 against 21/20
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.6, 0.4]]) and np.isclose(gap, 0.2)
    assert route(l, 2, groups=2, top_groups=1, group_best=1)[0].tolist() == [[3, 2]]
    assert route(l, 2, groups=2, top_groups=2)[0].tolist() == [[3, 1]]
    ids, w, _ = route(l, 2, bias=np.array([0.5, 0.0, 0.0, 0.0]), renorm=False, scale=2.0)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[1.0, 1.6]])
    ids, w, _ = route(l, 1, sigmoid=False, renorm=False)                # 4 of 1 + 3 + 1/3 + 4
    assert ids.tolist() == [[3]] and np.allclose(w, [[4.0 / (25.0 / 3.0)]])
    assert route(np.array([[0.0, 0.0, np.nan, 0.0]]), 4)[0].tolist() == [[0, 1, 3, 2]]


def test_dynamic_shared_memory_states_its_alignment():
    """16-byte copies and loads go to it: declared with that alignment, or rounded up
    by hand in the next lines; a plain element type promises no more than its own."""
    csrc = os.path.join(os.path.dirname(fb.__file__), "csrc")
    found = 0
    for path in glob.glob(os.path.join(csrc, "*.cu*")):
        with open(path) as f:
            text = f.read()
        for at in re.finditer(r"extern __shared__", text):
            lines = text[at.start():].split("\n")[:3]
            declared = re.search(r"__align__\((\d+)\)", lines[0])
            rounded = re.search(r"\+ (\d+)u\) & ~\1u", " ".join(lines[1:]))
            assert (declared and int(declared[1]) >= 16) or (rounded and int(rounded[1]) >= 15), "%s: %s" % (path, lines[0])
            found += 1
    assert found >= 3
