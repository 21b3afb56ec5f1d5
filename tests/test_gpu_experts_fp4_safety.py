"""The expert and 4-bit layers' failure detection and device-side checks.

Bounded waits: a test hook makes the producer never fill one pipeline stage;
the kernel must report the time-out in the status word, return, and leave the
context usable.  Debug build: the checks of every tile coordinate, split-K
slot and counter stay silent on clean runs, which give the normal build's bits.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from fp8_block_scaled_token_gb300 import synth
from tests.gpu_helpers import Ran, check_y
from tests.test_gpu_fp4 import _layer
from tests.test_gpu_moe import Layer
from tests import moe_reference as ref

pytestmark = pytest.mark.gpu

LIMIT_NS = 100_000_000  # 0.1 s
INVALID = 1


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _fp4_stall(x, packed, N, fmt, work, skip, limit):
    M, K = x.shape
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    a = fb.fp4_quant_act(x, fmt)
    ptrs = [t.data_ptr() if t is not None else None for t in (*a, *packed)]
    return fb.lib().fp8bs_testhook_fp4_stall(*ptrs, y.data_ptr(), M, N, K, fmt, work.data_ptr(), work.numel(), skip,
                                             limit, _stream())


@pytest.mark.parametrize("fmt", [fb.FP4_NV, fb.FP4_MX])
@pytest.mark.parametrize("M,N,K,skip", [(8, 256, 512, 0), (8, 5120, 5120, 3), (33, 5120, 5120, 2),
                                        (128, 5120, 5120, 4), (512, 640, 1024, 0)])  # (that has at most one unit a CTA)
def test_fp4_bounded_wait(M, N, K, skip, fmt):
    x, packed, y_ref, bound = _layer(M, N, K, fmt, seed=70)
    work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
    assert _fp4_stall(x, packed, N, fmt, work, skip, LIMIT_NS) == 0
    assert fb.workspace_status(work) != 0, "the stalled kernel did not report its time-out"
    work.zero_()
    y = fb.fp4_gemm_fused(x, *packed, N, fmt, workspace=work)
    assert fb.workspace_status(work) == 0
    check_y(y, y_ref, bound, "after time-out")


def _moe_stall(t, ops, ids, w, y, work, phase, skip, limit):
    M, E, k, H, I = t.dims
    w13, s13, w2, s2 = ops
    return fb.lib().fp8bs_testhook_moe_stall(t.x_dev.data_ptr(), H, ids.data_ptr(), w.data_ptr(), w13.data_ptr(),
                                             s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), y.data_ptr(), M, H, I, E, k,
                                             work.data_ptr(), work.numel(), fb.FLAG_WEIGHTS_TILED, phase, skip, limit,
                                             _stream())


def _moe(M, E, k, H, I, seed):
    t = Layer(M, E, k, H, I, seed=seed)
    t.x_dev = t.x.cuda()
    rng = np.random.RandomState(seed)
    ids = torch.from_numpy(rng.randint(0, E, (M, k)).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.uniform(0.1, 1, (M, k)).astype(np.float32)).cuda()
    y = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    return t, t.operands(), ids, w, y


@pytest.mark.parametrize("phase", [0, 1])
@pytest.mark.parametrize("M,E,k,H,I,skip", [(4, 8, 2, 512, 256, 0), (20, 12, 4, 1024, 384, 1), (64, 16, 4, 1024, 384, 1)])
def test_moe_bounded_wait(M, E, k, H, I, skip, phase):
    t, ops, ids, w, y = _moe(M, E, k, H, I, seed=M)
    work = t.workspace()
    assert _moe_stall(t, ops, ids, w, y, work, phase, skip, LIMIT_NS) == 0
    assert fb.workspace_status(work) != 0, "the stalled kernel did not report its time-out"
    work.zero_()
    y = fb.fp8_moe_experts(t.x_dev, ids, w, *ops, experts=E, workspace=work)
    assert fb.workspace_status(work) == 0
    y_ref, bound = ref.experts(t.x64(), ids.cpu().numpy(), w.cpu().numpy(), t.v13, t.v2)
    check_y(y, y_ref, bound, "after time-out")


def test_stall_hooks_reject_bad_arguments():
    t, ops, ids, w, y = _moe(2, 4, 2, 256, 128, seed=1)
    work = t.workspace()
    for phase, skip, limit in ((2, 0, 1000), (0, -1, 1000), (0, 0, 0), (1, 0, 20_000_000_000)):
        assert _moe_stall(t, ops, ids, w, y, work, phase, skip, limit) == INVALID
    torch.cuda.synchronize()
    assert not work.any(), "a rejected call must not launch"
    x, packed, _, _ = _layer(2, 256, 512, fb.FP4_NV, seed=1)
    fwork = fb.make_workspace(fb.fp4_gemm_workspace_size(2, 256, 512))
    for skip, limit in ((-1, 1000), (0, 0), (0, 20_000_000_000)):
        assert _fp4_stall(x, packed, 256, fb.FP4_NV, fwork, skip, limit) == INVALID
    torch.cuda.synchronize()
    assert not fwork.any()


@pytest.fixture(scope="module")
def debug_lib_built():
    from fp8_block_scaled_token_gb300 import build as fbuild
    fbuild.build(variants=("release", "debug"))


@pytest.mark.parametrize("M,E,k,H,I", [(1, 8, 2, 512, 256), (13, 43, 3, 1408, 640), (32, 16, 4, 256, 384),
                                       (64, 24, 8, 640, 256)])
def test_debug_build_moe_clean(M, E, k, H, I, debug_lib_built):
    t = Layer(M, E, k, H, I, seed=M + 5)
    ops, x, wr = t.operands(), t.x.cuda(), t.wr.cuda()
    want = fb.fp8_moe_layer(x, wr, k, *ops)
    with fb.debug_library() as L:
        assert L.fp8bs_testhook_debug_build() == 1
        work = t.workspace()
        with Ran() as r:
            got = fb.fp8_moe_layer(x, wr, k, *ops, workspace=work)
        assert sum(r.launched().values()) == 3
        assert fb.workspace_status(work) == 0, "a device-side check fired"
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", [fb.FP4_NV, fb.FP4_MX])
@pytest.mark.parametrize("M,N,K", [(8, 256, 512), (1, 5120, 5120), (13, 300, 1312), (33, 1000, 2080), (64, 1024, 2048),
                                   (300, 640, 1024), (512, 384, 512)])
def test_debug_build_fp4_clean(M, N, K, fmt, debug_lib_built):
    x = synth.activations(M, K, seed=M + 6, outlier_p=0.001).cuda()
    packed = fb.fp4_quant_weights(synth.weights(N, K, seed=M + 7).cuda(), fmt)
    want = fb.fp4_gemm_fused(x, *packed, N, fmt)
    with fb.debug_library():
        work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
        got = fb.fp4_gemm_fused(x, *packed, N, fmt, workspace=work)
        assert fb.workspace_status(work) == 0, "a device-side check fired"
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
