"""The expert and 4-bit entry points on the CPU: declared, and bad arguments
rejected on the host before anything would reach a GPU.  Nothing here launches
a kernel."""
import ctypes

from tests.test_abi import A1, A16, INVALID, MISALIGNED, NUL, OK, P, S, SHAPE, L, declared_symbols  # noqa: F401


def test_entry_points_are_declared():
    names = declared_symbols()
    for n in ("fp4_quant_weights", "fp4_dequant_weights", "fp4_quant_act", "fp4_gemm_workspace_size", "fp4_gemm",
              "fp4_gemm_fused", "moe_route_workspace_size", "moe_route", "fp8_moe_workspace_size", "fp8_moe_experts",
              "fp8_moe_layer", "fp8bs_testhook_fp4_stall", "fp8bs_testhook_moe_stall"):
        assert n in names


def test_fp4_validation(L):
    NV, MX = 0, 1
    for q in (L.fp4_quant_weights, None):
        def call(w=A16, wt=0, N=256, K=512, fmt=NV, wq=A16, wa=A16, rows=A16):
            if q is not None:
                return q(w, wt, N, K, fmt, wq, wa, rows, S)
            return L.fp4_dequant_weights(wq, wa, rows, N, K, fmt, w, wt, S)
        assert call(w=NUL) == INVALID
        assert call(wt=2) == INVALID
        assert call(fmt=2) == INVALID
        assert call(N=0) == INVALID
        assert call(rows=NUL) == INVALID                       # NV needs the row scales
        assert call(rows=NUL, fmt=MX) not in (INVALID, SHAPE, MISALIGNED)
        assert call(K=48) == SHAPE
        assert call(N=1 << 30, K=1 << 20) == SHAPE             # tile coordinates past 31 bits
        assert call(wq=P(0x10008)) == MISALIGNED
        assert call(rows=P(0x10002)) == MISALIGNED
    a = L.fp4_quant_act
    assert a(A16, 513, 512, 512, NV, A16, A16, A16, 0, S) == SHAPE
    assert a(A16, 8, 512, 256, NV, A16, A16, A16, 0, S) == INVALID          # ldx < K
    assert a(A16, 8, 512, 512, NV, A16, A16, A16, 2, S) == INVALID          # unknown flag
    assert a(A16, 8, 512, 512, NV, A16, A16, NUL, 0, S) == INVALID
    assert a(A16, 8, 512, 516, NV, A16, A16, A16, 0, S) == MISALIGNED       # ldx % 8
    g = L.fp4_gemm
    assert g(A16, A16, A16, A16, A16, A16, A16, 513, 256, 512, NV, A16, 1 << 20, 0, S) == SHAPE
    assert g(A16, A16, A16, A16, A16, A16, A16, 8, 256, 40, NV, A16, 1 << 20, 0, S) == SHAPE
    assert g(A16, A16, NUL, A16, A16, A16, A16, 8, 256, 512, NV, A16, 1 << 20, 0, S) == INVALID
    assert g(A16, A16, A16, A16, A16, A16, A16, 8, 256, 512, 3, A16, 1 << 20, 0, S) == INVALID
    assert g(A16, A16, A16, A16, A16, A16, A16, 8, 256, 512, NV, A16, 1 << 20, 2, S) == INVALID
    assert g(A16, A16, A16, A16, P(0x10008), A16, A16, 8, 256, 512, NV, A16, 1 << 20, 0, S) == MISALIGNED
    f = L.fp4_gemm_fused
    assert f(A16, 256, A16, A16, A16, A16, 8, 256, 512, NV, A16, 1 << 20, 0, S) == INVALID      # ldx < K
    assert f(A16, 512, A16, A16, NUL, A16, 8, 256, 512, NV, A16, 1 << 20, 0, S) == INVALID
    assert f(A16, 512, A16, A16, A16, A16, 8, 256, 512, NV, P(0x10010), 1 << 20, 0, S) == MISALIGNED
    sz = ctypes.c_size_t(3)
    assert L.fp4_gemm_workspace_size(513, 256, 512, NV, ctypes.byref(sz)) == SHAPE and sz.value == 0
    assert L.fp4_gemm_workspace_size(8, 256, 512, 7, ctypes.byref(sz)) == INVALID


def test_moe_validation(L):
    def layer(x=A16, ldx=512, wr=A16, wt=1, w13=A16, s13=A16, w2=A16, s2=A16, y=A16, ids=NUL, w=NUL, M=8, H=512, I=256,
              E=8, k=2, ws=A16, n=1 << 40, flags=2):
        return L.fp8_moe_layer(x, ldx, wr, wt, 1, w13, s13, w2, s2, y, ids, w, M, H, I, E, k, ws, n, flags, S)

    def experts(ids=A16, w=A16, **kw):
        d = dict(x=A16, ldx=512, w13=A16, s13=A16, w2=A16, s2=A16, y=A16, M=8, H=512, I=256, E=8, k=2, ws=A16, n=1 << 40,
                 flags=2)
        d.update(kw)
        return L.fp8_moe_experts(d["x"], d["ldx"], ids, w, d["w13"], d["s13"], d["w2"], d["s2"], d["y"], d["M"], d["H"],
                                 d["I"], d["E"], d["k"], d["ws"], d["n"], d["flags"], S)

    for call in (layer, experts):
        for nul in ("x", "w13", "s13", "w2", "s2", "y", "ws"):
            assert call(**{nul: NUL}) == INVALID
        assert call(M=65) == SHAPE and call(M=0) == INVALID
        assert call(E=513) == SHAPE and call(k=9) == SHAPE and call(E=64, k=17) == SHAPE and call(k=0) == INVALID
        assert call(H=576) == SHAPE and call(I=192) == SHAPE and call(I=0) == INVALID
        assert call(E=512, H=1 << 14, I=1 << 14, ldx=1 << 14) == SHAPE  # tile coordinates past 31 bits
        assert call(ldx=256) == INVALID and call(ldx=516) == MISALIGNED
        assert call(flags=4) == INVALID
        assert call(w13=P(0x10008)) == MISALIGNED and call(s2=A1) == MISALIGNED and call(ws=P(0x10080)) == MISALIGNED
    assert layer(wr=NUL) == INVALID and layer(wt=5) == INVALID and layer(wr=P(0x10008)) == MISALIGNED
    assert layer(ids=A1) == MISALIGNED
    assert experts(ids=NUL) == INVALID and experts(w=NUL) == INVALID and experts(w=A1) == MISALIGNED
    r = L.moe_route
    assert r(A16, 512, A16, 1, 8, 512, 8, 2, 1, NUL, A16, A16, 1 << 20, 0, S) == INVALID
    assert r(A16, 512, A16, 1, 8, 512, 8, 9, 1, A16, A16, A16, 1 << 20, 0, S) == SHAPE
    assert r(A16, 512, A16, 1, 8, 512, 8, 2, 1, A16, A16, A16, 1 << 20, 2, S) == INVALID    # no weights to be tiled
    sz = ctypes.c_size_t(3)
    assert L.moe_route_workspace_size(8, 600, ctypes.byref(sz)) == SHAPE and sz.value == 0
    assert L.moe_route_workspace_size(8, 64, ctypes.byref(sz)) == OK and sz.value >= 8 * 64 * 4
    assert L.fp8_moe_workspace_size(8, 512, 100, 8, 2, ctypes.byref(sz)) == SHAPE and sz.value == 0
