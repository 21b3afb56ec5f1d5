"""The expert layer in the forms that its routing and products choose by size:
rows of H above 4,096 (up to 1,024 routing threads, one step of them or more),
four experts a CTA with a number of experts that four does not divide, and
row-major expert weights in every token tile.

Logits are fp32 sums of at most 16,512 products of order 1 / sqrt(H): they err by
less than 2^-24 * sqrt(16,512) * |l| ~ 2e-5, hence the 1e-4 of test_gpu_moe.py
here as well, as its bound for Y.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests import moe_reference as ref
from tests.gpu_helpers import check_y
from tests.test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


def _check_choice(t, ids, w, renorm):
    k = t.dims[2]
    x, wr = t.x64(), t.wr.double().numpy()
    want, ww, gap = ref.route(x, wr, k, renorm)
    if gap > 1e-4:
        assert np.array_equal(ids, want)
    logits = x @ wr.T
    got = np.take_along_axis(logits, ids.astype(np.int64), axis=1)
    assert np.allclose(got, np.take_along_axis(logits, want, axis=1), atol=1e-4)
    assert all(len(set(row)) == k for row in ids.tolist())
    assert np.allclose(w, ww, atol=1e-4)


def _check_layer(t, renorm):
    M, E, k, H, I = t.dims
    work = t.workspace()
    x, wr, ops = t.x.cuda(), t.wr.cuda(), t.operands()
    y, ids, w = fb.fp8_moe_layer(x, wr, k, *ops, renormalize=renorm, workspace=work)
    assert fb.workspace_status(work) == 0
    i, v = ids.cpu().numpy(), w.cpu().numpy()
    _check_choice(t, i, v, renorm)
    y_ref, bound = ref.experts(t.x64(), i, v, t.v13, t.v2)
    check_y(y, y_ref, bound, "moe %s" % (t.dims,))
    ids2, w2 = fb.moe_route(x, wr, k, renormalize=renorm)          # the choice alone: the same bits
    assert torch.equal(ids2, ids) and torch.equal(w2, w)
    y2 = fb.fp8_moe_experts(x, ids, w, *ops, experts=E, workspace=work)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,E,k,H", [(3, 12, 4, 4224), (8, 7, 2, 5120), (13, 10, 3, 8192), (1, 12, 5, 8320),
                                     (8, 5, 1, 8320)])
def test_long_rows(M, E, k, H, dtype):
    _check_layer(Layer(M, E, k, H, 128, seed=H + M, wr_dtype=dtype), renorm=dtype is torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,E,k,H", [(1, 300, 16, 4224), (2, 130, 8, 16512), (16, 152, 6, 5120), (11, 33, 4, 4608)])
def test_routing_of_long_rows_alone(M, E, k, H, dtype):
    t = Layer.__new__(Layer)
    g = torch.Generator().manual_seed(H + E)
    t.dims = M, E, k, H, 128
    t.x = torch.randn((M, H), generator=g).to(torch.bfloat16)
    t.wr = (torch.randn((E, H), generator=g) * 2 / H ** 0.5).to(dtype)
    wide = torch.full((M, H + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = t.x
    for renorm in (True, False):
        ids, w = fb.moe_route(wide[:, :H], t.wr.cuda(), k, renormalize=renorm)
        _check_choice(t, ids.cpu().numpy(), w.cpu().numpy(), renorm)


@pytest.mark.parametrize("M,E,k,H,I", [(64, 97, 8, 256, 128), (64, 301, 6, 128, 128), (17, 103, 4, 384, 128),
                                       (33, 63, 3, 256, 128), (64, 39, 2, 5120, 128)])
def test_numbers_of_experts_that_four_does_not_divide(M, E, k, H, I):
    for dtype in (torch.bfloat16, torch.float32):
        _check_layer(Layer(M, E, k, H, I, seed=M + E, wr_dtype=dtype), renorm=dtype is torch.float32)


@pytest.mark.parametrize("M,E,k,H,I", [(1, 8, 2, 512, 256), (16, 24, 4, 640, 384), (17, 20, 6, 640, 128),
                                       (32, 16, 3, 256, 640), (33, 12, 2, 1024, 256), (64, 40, 8, 384, 384),
                                       (50, 24, 6, 896, 640), (1, 24, 8, 128, 1152)])
def test_row_major_weights_give_the_tiled_ones_bits(M, E, k, H, I):
    t = Layer(M, E, k, H, I, seed=M + H)
    a = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), k, *t.operands(True))
    b = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), k, *t.operands(False))
    for s, r in zip(a, b):
        assert torch.equal(s.view(torch.int16), r.view(torch.int16))
    y_ref, bound = ref.experts(t.x64(), a[1].cpu().numpy(), a[2].cpu().numpy(), t.v13, t.v2)
    check_y(b[0], y_ref, bound, "row-major %s" % (t.dims,))
    y = fb.fp8_moe_experts(t.x.cuda(), a[1], a[2], *t.operands(False))
    assert torch.equal(y.view(torch.int16), a[0].view(torch.int16))
