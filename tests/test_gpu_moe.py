"""GPU parity of the expert layer (router, choice, gate/up product, SwiGLU,
re-quantisation, down product, weighted sum) against the definition in 64
bits.

Router: logits are fp32 sums, so ids must agree wherever the 64-bit logits
differ by more than 1e-4 (H <= 2048 products of order 1 summed in fp32 err by
less than 2^-24 * sqrt(2048) * |l| ~ 1e-5), and the weights to 1e-4.

Y: |y - y64| <= 4e-3 * sum |w| |h| |w2| + 1e-6.  One bf16 rounding is 2^-9 of
|y|; fp32 sums are far below; an intermediate whose fp32 value rounds to the
other E4M3 neighbour moves by 1/8 of itself, one of at least 128 terms: 1e-3 of
the sum.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests import moe_reference as ref
from tests.gpu_helpers import Ran, check_y

pytestmark = pytest.mark.gpu

RUNS_MOE_ROUTE, RUNS_MOE_PLAN = 88, 89


def runs_moe_gemm(phase, M):
    return 90 + phase * 3 + (0 if M <= 16 else 1 if M <= 32 else 2)


class Layer:
    """A random layer: its device operands and their 64-bit values."""

    def __init__(self, M, E, k, H, I, seed=0, wr_dtype=torch.bfloat16):
        rng = np.random.RandomState(seed)
        self.dims = M, E, k, H, I
        self.x = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(torch.bfloat16)
        self.wr = torch.from_numpy((rng.standard_normal((E, H)) * 2 / np.sqrt(H)).astype(np.float32)).to(wr_dtype)
        self.c13, self.s13, self.v13 = ref.weights(E, 2 * I, H, rng)
        self.c2, self.s2, self.v2 = ref.weights(E, H, I, rng)

    def x64(self):
        return self.x.double().numpy()

    def operands(self, tiled=True):
        f = ref.tile if tiled else (lambda c: c)
        return [torch.from_numpy(a).cuda() for a in (f(self.c13), self.s13, f(self.c2), self.s2)]

    def workspace(self):
        M, E, k, H, I = self.dims
        return fb.make_workspace(fb.fp8_moe_workspace_size(M, H, I, E, k))


SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 512, 256), (3, 5, 5, 128, 384), (8, 16, 4, 1024, 256), (13, 43, 3, 1408, 640),
          (16, 24, 4, 256, 384), (17, 33, 6, 640, 128), (32, 64, 8, 512, 256), (33, 12, 2, 256, 128),
          (64, 96, 8, 384, 256), (64, 300, 16, 128, 128), (2, 160, 6, 2048, 128)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,k,H,I", SHAPES)
def test_layer_matches_64_bits(M, E, k, H, I, renorm):
    t = Layer(M, E, k, H, I, seed=M * 1000 + E, wr_dtype=torch.float32 if renorm else torch.bfloat16)
    work = t.workspace()
    with Ran() as r:
        y, ids, w = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), k, *t.operands(), renormalize=renorm, workspace=work)
    assert r.launched() == {RUNS_MOE_ROUTE: 1, runs_moe_gemm(0, M): 1, runs_moe_gemm(1, M): 1}
    assert fb.workspace_status(work) == 0
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    logits = t.x64() @ t.wr.double().numpy().T
    want, ww, gap = ref.route(t.x64(), t.wr.double().numpy(), k, renorm)
    if gap > 1e-4:
        assert np.array_equal(ids, want)
    mine = np.take_along_axis(logits, ids.astype(np.int64), axis=1)
    assert np.allclose(mine, np.take_along_axis(logits, want, axis=1), atol=1e-4)
    assert np.allclose(w, ww, atol=1e-4)
    y_ref, bound = ref.experts(t.x64(), ids, w, t.v13, t.v2)
    check_y(y, y_ref, bound, "moe %s" % (t.dims,))
    # the choice on its own, and the experts on that choice: the same bits
    ids2, w2 = fb.moe_route(t.x.cuda(), t.wr.cuda(), k, renormalize=renorm)
    assert np.array_equal(ids2.cpu().numpy(), ids) and np.array_equal(w2.cpu().numpy(), w)
    with Ran() as r:
        y2 = fb.fp8_moe_experts(t.x.cuda(), ids2, w2, *t.operands(), experts=E, workspace=work)
    assert r.launched() == {RUNS_MOE_PLAN: 1, runs_moe_gemm(0, M): 1, runs_moe_gemm(1, M): 1}
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))


# few tiles of Y and many K blocks to each (7 to 41 contributors to a tile where
# every SM takes part), and tokens that do not divide by the warps of the sum
DEEP = [(50, 24, 6, 896, 640), (20, 16, 2, 512, 256), (29, 58, 8, 1024, 256), (64, 40, 8, 128, 1408),
        (40, 8, 2, 1280, 384), (15, 60, 4, 384, 768), (1, 24, 8, 128, 1152)]


@pytest.mark.parametrize("M,E,k,H,I", DEEP)
def test_deep_tiles_and_an_output_at_any_two_byte_address(M, E, k, H, I):
    t = Layer(M, E, k, H, I, seed=M + E)
    ops, work = t.operands(), t.workspace()
    y, ids, w = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), k, *ops, workspace=work)
    y_ref, bound = ref.experts(t.x64(), ids.cpu().numpy(), w.cpu().numpy(), t.v13, t.v2)
    check_y(y, y_ref, bound, "moe %s" % (t.dims,))
    buf = torch.full((M * H + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    for first in (1, 2, 3, 4):
        buf.fill_(7.0)
        out = buf[first:first + M * H].view(M, H)
        fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), k, *ops, y=out, workspace=work)
        assert torch.equal(out.view(torch.int16), y.view(torch.int16))
        assert (buf[:first] == 7.0).all() and (buf[first + M * H:] == 7.0).all()
    assert fb.workspace_status(work) == 0


def test_row_major_weights_give_the_same_bits():
    t = Layer(9, 12, 3, 640, 384, seed=3)
    a = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), 3, *t.operands(True))[0]
    b = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), 3, *t.operands(False))[0]
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_weights_from_the_librarys_quantiser():
    """fp8_quant_weight_blocks of the stacked experts is the operand."""
    M, E, k, H, I = 4, 6, 2, 256, 128
    g = torch.Generator().manual_seed(5)
    w13 = (torch.randn((E, 2 * I, H), generator=g) * 0.05).cuda()
    w2 = (torch.randn((E, H, I), generator=g) * 0.05).cuda()
    x = torch.randn((M, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((E, H), generator=g) / 8).cuda()
    out = []
    for tiled in (True, False):
        q13, s13 = fb.fp8_quant_weight_blocks(w13.view(E * 2 * I, H), tiled=tiled)
        q2, s2 = fb.fp8_quant_weight_blocks(w2.view(E * H, I), tiled=tiled)
        if not tiled:
            q13, q2 = q13.view(E, 2 * I, H), q2.view(E, H, I)
        out.append(fb.fp8_moe_layer(x, wr, k, q13, s13, q2, s2))
    y, ids, w = out[0]
    assert torch.equal(out[1][0].view(torch.int16), y.view(torch.int16))
    # E4M3 of weights and activations err by 2^-4 each at most: against the unquantised layer
    xd = x.double()
    want = torch.zeros((M, H), dtype=torch.float64, device="cuda")
    for m in range(M):
        for j in range(k):
            e = int(ids[m, j])
            gu = w13[e].double() @ xd[m]
            h = torch.nn.functional.silu(gu[:I]) * gu[I:]
            want[m] += w[m, j].double() * (w2[e].double() @ h)
    assert float((y.double() - want).norm() / want.norm()) < 0.1


def test_ties_go_to_the_lowest_expert():
    t = Layer(5, 40, 4, 256, 128, seed=8)
    t.wr[:] = t.wr[0]                                              # every expert's logit is the same number
    ids, w = fb.moe_route(t.x.cuda(), t.wr.cuda(), 4)
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 5
    assert torch.equal(w.cpu(), torch.full((5, 4), 0.25))
    t.wr[7] = 0
    t.x[:] = t.x.abs()
    t.wr[:] = -t.wr.abs()
    ids, _ = fb.moe_route(t.x.cuda(), t.wr.cuda(), 4)
    assert ids.cpu().tolist() == [[7, 0, 1, 2]] * 5               # 0 is the largest, the others tie


def test_given_choice_skips_repeats_and_zero_weights():
    """Ids outside the experts, an expert named twice, weights of zero, a
    token with nothing left, negative weights."""
    t = Layer(6, 10, 4, 384, 256, seed=12)
    ids = np.array([[0, 1, 2, 3], [-1, 4, -1, 10], [5, 5, 5, 0], [-1, -1, -1, -1], [9, 2, 2 ** 30, -2 ** 31],
                    [1, 2, 3, 4]], np.int32)
    w = np.array([[.1, .2, .3, .4], [1, .5, 1, 1], [.25, .5, .125, .1], [1, 1, 1, 1], [-.5, 2, 1, 1], [0, 0, .5, 0]],
                 np.float32)
    work = t.workspace()
    y = fb.fp8_moe_experts(t.x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *t.operands(),
                           experts=10, workspace=work)
    assert fb.workspace_status(work) == 0
    y_ref, bound = ref.experts(t.x64(), ids, w, t.v13, t.v2)
    check_y(y, y_ref, bound, "given choice")
    assert not y[3].any()


def test_no_expert_at_all_gives_zeros():
    t = Layer(3, 4, 2, 256, 128, seed=2)
    ids = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    y = torch.full((3, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    work = t.workspace()
    fb.fp8_moe_experts(t.x.cuda(), ids, w, *t.operands(), experts=4, y=y, workspace=work)
    assert not y.any() and fb.workspace_status(work) == 0
    ids[1, 0] = 2                                                  # and the workspace serves the next call
    y = fb.fp8_moe_experts(t.x.cuda(), ids, w, *t.operands(), experts=4, workspace=work)
    y_ref, bound = ref.experts(t.x64(), ids.cpu().numpy(), w.cpu().numpy(), t.v13, t.v2)
    check_y(y, y_ref, bound, "after none")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_keeps_to_its_own_row(bad):
    t = Layer(7, 12, 3, 256, 128, seed=21)
    good = fb.fp8_moe_layer(t.x.cuda(), t.wr.cuda(), 3, *t.operands())[0]
    x = t.x.clone()
    x[4, 77] = bad
    work = t.workspace()
    y, ids, w = fb.fp8_moe_layer(x.cuda(), t.wr.cuda(), 3, *t.operands(), workspace=work)
    keep = [m for m in range(7) if m != 4]
    assert torch.equal(y[keep].view(torch.int16), good[keep].view(torch.int16))
    assert y[4].isnan().all()
    assert len(set(ids[4].tolist())) == 3 and 0 <= int(ids.min()) and int(ids.max()) < 12
    assert fb.workspace_status(work) == 0


def test_an_unchosen_experts_overflow_is_not_seen():
    """Expert 1 overflows for every token; only token 0 chooses it."""
    t = Layer(3, 3, 1, 256, 128, seed=4)
    ops = t.operands()
    ops[1][2:4] = 3e38                                             # s13 of expert 1 (two tiles of 128 rows)
    ids = torch.tensor([[1], [0], [2]], dtype=torch.int32, device="cuda")
    w = torch.ones((3, 1), device="cuda")
    y = fb.fp8_moe_experts(t.x.cuda(), ids, w, *ops, experts=3)
    y_ref, bound = ref.experts(t.x64(), ids.cpu().numpy(), w.cpu().numpy(), t.v13, t.v2)
    check_y(y[1:], y_ref[1:], bound[1:], "tokens beside an overflow")


@pytest.mark.parametrize("where", ["w2", "w13", "s2", "s13"])
@pytest.mark.parametrize("M", [3, 20, 50])
def test_an_unchosen_experts_bad_weights_are_not_seen(M, where):
    """Expert 1 has a NaN code or an infinite or NaN block scale; tokens 0 and M - 1 choose it."""
    t = Layer(M, 4, 2, 256, 384, seed=M)
    ids = np.stack([np.full(M, 2), np.arange(M) % 2 * 3], 1).astype(np.int32)
    ids[[0, M - 1], 1] = 1
    w = np.random.RandomState(M).uniform(0.2, 1, (M, 2)).astype(np.float32)
    y_ref, bound = ref.experts(t.x64(), ids, w, t.v13, t.v2)
    keep = np.arange(1, M - 1)
    if where == "w2":
        t.c2[1, :, 130] = 0x7F                                     # a NaN in every row
    elif where == "w13":
        t.c13[1, 5:: 384, 7] = 0xFF                                # of one gate and one up row
    else:
        s = getattr(t, where)                                      # [128-row tiles of all experts, K blocks]
        n = s.shape[0] // 4
        s[n:2 * n] = np.where(np.arange(s.shape[1]) % 2, np.nan, np.inf)
    work = t.workspace()
    y = fb.fp8_moe_experts(t.x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *t.operands(),
                           experts=4, workspace=work)
    assert fb.workspace_status(work) == 0
    check_y(y[1:-1], y_ref[keep], bound[keep], "tokens beside a bad expert")
    assert y[[0, M - 1]].isnan().all()


def test_strides_streams_reruns_and_a_clean_workspace():
    M, E, k, H, I = 11, 20, 4, 640, 256
    t = Layer(M, E, k, H, I, seed=33)
    ops, wr, x = t.operands(), t.wr.cuda(), t.x.cuda()
    wide = torch.full((M, H + 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = x
    work = t.workspace()
    first = fb.fp8_moe_layer(x, wr, k, *ops, workspace=work)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [fb.fp8_moe_layer(wide[:, :H], wr, k, *ops, workspace=work, flags=fb.FLAG_OVERLAP_PREV if i % 2 else 0)
                for i in range(10)]
    s.synchronize()
    for o in outs:
        for a, b in zip(o, first):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert fb.workspace_status(work) == 0
    assert not work[:1024 + 65536].any(), "routing words and counters back at zero"


def test_one_workspace_serves_calls_of_different_choices():
    t = Layer(16, 64, 4, 256, 128, seed=50)
    ops, work = t.operands(), t.workspace()
    rng = np.random.RandomState(1)
    for n in range(6):
        ids = rng.randint(-1, 64 if n % 2 else 3, (16, 4)).astype(np.int32)
        w = rng.uniform(0, 1, (16, 4)).astype(np.float32)
        y = fb.fp8_moe_experts(t.x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *ops, experts=64,
                               workspace=work)
        y_ref, bound = ref.experts(t.x64(), ids, w, t.v13, t.v2)
        check_y(y, y_ref, bound, "call %d" % n)


def test_layer_in_a_cuda_graph():
    t = Layer(8, 16, 2, 512, 256, seed=60)
    ops, work, wr, x = t.operands(), t.workspace(), t.wr.cuda(), t.x.cuda()
    want = fb.fp8_moe_layer(x, wr, 2, *ops, workspace=work)[0]
    y = torch.empty_like(want)
    ids = torch.empty((8, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((8, 2), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            fb.fp8_moe_layer(x, wr, 2, *ops, y=y, ids=ids, weights=w, workspace=work)
    y.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_refusals():
    t = Layer(2, 4, 2, 256, 128, seed=1)
    ops, wr, x = t.operands(), t.wr.cuda(), t.x.cuda()
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp8_moe_layer(x, wr, 5, *ops)                           # more than the experts
    assert e.value.code == 2
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp8_moe_workspace_size(65, 256, 128, 4, 2)
    assert e.value.code == 2
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp8_moe_layer(x, wr, 2, *ops, workspace=fb.make_workspace(4096))
    assert e.value.code == 4
    with pytest.raises(ValueError):
        fb.fp8_moe_layer(x[:, :128], wr, 2, *ops)                  # H of x is not the router's
    with pytest.raises(ValueError):
        fb.fp8_moe_experts(x, torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.ones((2, 2), device="cuda"),
                           *ops)                                   # tiled without experts=
    with pytest.raises(TypeError):
        fb.fp8_moe_experts(x, torch.zeros((2, 2), dtype=torch.int64, device="cuda"), torch.ones((2, 2), device="cuda"),
                           *ops, experts=4)
    with pytest.raises(ValueError):
        fb.fp8_moe_layer(x.cpu(), wr, 2, *ops)
