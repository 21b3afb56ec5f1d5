"""GPU parity of the routing with scores, bias and groups, and of the expert
layer behind it, against the definition in 64 bits.

Logits are sums of H products in fp32, put together from 256 or more partial
sums: H roundings of at most 2^-25 of a partial sum below 1/4, adding up as
random ones do to sqrt(2048) 2^-27 = 3.4e-7, six times which is 2e-6; scores
move by no more than their logit.  So the ids must be the reference's where its
gaps are above 4e-6, which is asserted of the seeded inputs.  Weights: expf and a
division a few 2^-23, the logit's rounding to fp32 |l| 2^-24 and its sum's error
2e-6: relative 5e-6 for |l| < 16.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.gpu_helpers import Ran
from tests.route_reference import route
from tests.test_gpu_moe import Layer, runs_moe_gemm

pytestmark = pytest.mark.gpu

RUNS_MOE_SCORED, RUNS_MOE_PLAN = 100, 89
GAP, W_TOL = 4e-6, 5e-6


def _inputs(M, E, H, bias, wr_dtype, seed, size=1.5):
    rng = np.random.RandomState(seed)
    x = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(torch.bfloat16)
    wr = torch.from_numpy((rng.standard_normal((E, H)) * size / np.sqrt(H)).astype(np.float32)).to(wr_dtype)
    b = (rng.standard_normal(E) * 0.05).astype(np.float32) if bias else None
    return x, wr, b


def _logits(x, wr):
    return x.double().numpy() @ wr.double().numpy().T


def _check(got, logits, k, b=None, tol=W_TOL, **kw):
    ids, w, gap = route(logits, k, None if b is None else b.astype(np.float64), **kw)
    assert gap > GAP, "the inputs have a choice at a border (%g): another seed" % gap
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.allclose(got[1].cpu().double().numpy(), w, rtol=tol, atol=0)


def _call(x, wr, k, b=None, sigmoid=True, renorm=True, **kw):
    return fb.moe_route_grouped(x.cuda(), wr.cuda(), k, bias=None if b is None else torch.from_numpy(b).cuda(),
                                scoring=fb.SCORE_SIGMOID if sigmoid else fb.SCORE_SOFTMAX, renormalize=renorm, **kw)


# M, E, k, H, groups, top_groups, group_best
SHAPES = [(1, 1, 1, 128, 1, 1, 1), (1, 64, 6, 2048, 1, 1, 2), (8, 256, 8, 1024, 8, 4, 2), (64, 160, 6, 640, 8, 3, 1),
          (5, 6, 4, 128, 3, 2, 2), (13, 45, 5, 1408, 5, 2, 2), (33, 512, 16, 256, 32, 7, 2), (64, 512, 12, 128, 2, 1, 1),
          (17, 96, 3, 384, 16, 1, 2), (9, 33, 2, 512, 11, 4, 1), (2, 448, 8, 2048, 7, 3, 2), (16, 31, 16, 256, 31, 16, 1),
          (3, 128, 8, 128, 4, 4, 2), (64, 8, 1, 2048, 4, 3, 2), (7, 300, 10, 4224, 3, 2, 2)]


@pytest.mark.parametrize("M,E,k,H,G,tg,best", SHAPES)
def test_matches_64_bits(M, E, k, H, G, tg, best):
    for n, (sigmoid, bias, renorm, dtype, scale) in enumerate([(True, True, True, torch.bfloat16, 1.0),
                                                              (False, False, False, torch.float32, 16.0),
                                                              (True, False, False, torch.float32, 2.5),
                                                              (False, True, True, torch.bfloat16, 1.0)]):
        kw = dict(sigmoid=sigmoid, groups=G, top_groups=tg, group_best=best, renorm=renorm, scale=scale)
        x, wr, b = _inputs(M, E, H, bias, dtype, seed=SEEDS.get((M, E, n), 10 * M + E + n))
        with Ran() as r:
            got = _call(x, wr, k, b, **kw)
        assert r.launched() == {RUNS_MOE_SCORED: 1}
        _check(got, _logits(x, wr), k, b, **kw)


# (M, E, which of the four): where the first seed has a choice at a border
SEEDS = {(64, 160, 2): 1802, (33, 512, 1): 4843, (33, 512, 2): 1844, (33, 512, 3): 2845, (64, 512, 1): 18153,
         (64, 512, 2): 3154, (64, 512, 3): 2155, (16, 31, 3): 1194}


@pytest.mark.parametrize("sigmoid,E", [(True, 512), (True, 45), (False, 24), (False, 512)])
@pytest.mark.parametrize("seed", range(4))
def test_scores_a_few_2_to_the_minus_24_apart(sigmoid, E, seed):
    """Exact logits (one product each) up to 3 and biases that leave the scores plus
    bias 4e-7 apart, two roundings of the bias (2^-25 each at most) aside, above the
    3 * 2^-24 = 1.8e-7 from which the choice is that of exact arithmetic."""
    rng = np.random.RandomState(seed)
    l = (rng.rand(E) * 6 - 3).astype(np.float32)
    wr = torch.zeros((E, 128))
    wr[:, 5] = torch.from_numpy(l)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    x[:, 5] = 1
    l = l.astype(np.float64)
    s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l) / np.exp(l).sum()
    b = (0.5 + 4e-7 * rng.permutation(E) - s).astype(np.float32)
    k = min(E, 16)
    ids, w, gap = route(np.stack([l, l]), k, b.astype(np.float64), sigmoid=sigmoid)
    assert gap > 3.2e-7
    got = _call(x, wr, k, b, sigmoid=sigmoid)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.allclose(got[1].cpu().double().numpy(), w, rtol=W_TOL, atol=0)


@pytest.mark.parametrize("M,E,H", [(3, 24, 20480), (64, 12, 12416)])
def test_long_rows(M, E, H):
    """Several turns of a warp over H.  Sums as above, six times sqrt(20,480) 2^-27: 6.4e-6 a logit."""
    x, wr, b = _inputs(M, E, H, True, torch.bfloat16, seed=H + 1)
    ids, w, gap = route(_logits(x, wr), 3, b.astype(np.float64), sigmoid=True, groups=4, top_groups=2, group_best=2)
    assert gap > 1.3e-5, "the inputs have a choice at a border (%g): another seed" % gap
    got = _call(x, wr, 3, b, groups=4, top_groups=2)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.allclose(got[1].cpu().double().numpy(), w, rtol=1e-5, atol=0)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,H", [(256, 5120), (24, 20480)])
def test_channels_far_above_the_others(E, H, sigmoid):
    """Logits are off by (10 + H / 256) 2^-24 times the sum of |x wr| at most, scores by a
    quarter of that (sigmoid) or half of it (softmax), weights by twice their logit's
    error: no expert that is left out, or comes later, is better by more."""
    rng = np.random.RandomState(H)
    x, wr, b = _inputs(8, E, H, True, torch.float32, seed=H)
    x = torch.where(torch.from_numpy(rng.rand(8, H) < 0.001), x * 1000, x)
    logits = _logits(x, wr)
    err = (10 + H / 256) * 2.0 ** -24 * (x.abs().double().numpy() @ wr.abs().double().numpy().T).max()
    assert err < 1e-2
    ids, w = [t.cpu().numpy() for t in _call(x, wr, 8, b, sigmoid=sigmoid, renorm=False)]
    s = 1 / (1 + np.exp(-logits))
    if not sigmoid:
        s = np.exp(logits - logits.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    c = s + b.astype(np.float64)
    for m in range(8):
        left = np.ones(E, bool)
        for e in ids[m]:
            left[e] = False
            assert c[m, e] >= c[m, left].max() - err
    size = np.abs(logits).max() * 2.0 ** -23
    # atol: softmax weights go down to e^-370 here, and below 2^-126 fp32 has no number that is right to 2^-24
    assert np.allclose(w, np.take_along_axis(s, ids.astype(np.int64), axis=1), rtol=2 * err + size + W_TOL, atol=2.0 ** -126)


def test_one_group_without_a_bias_is_the_plain_routing():
    x, wr, _ = _inputs(21, 70, 1024, False, torch.float32, seed=3)
    for renorm in (True, False):
        ids, w = fb.moe_route(x.cuda(), wr.cuda(), 5, renormalize=renorm)
        got = _call(x, wr, 5, sigmoid=False, renorm=renorm)
        assert torch.equal(got[0], ids) and torch.allclose(got[1], w, rtol=W_TOL, atol=0)


def _whole(M, E, H, seed):
    """Whole-number inputs: logits are exact, and many are equal."""
    rng = np.random.RandomState(seed)
    return (torch.from_numpy(rng.randint(-1, 2, (M, H)).astype(np.float32)).to(torch.bfloat16),
            torch.from_numpy(rng.randint(-1, 2, (E, H)).astype(np.float32) * (rng.rand(1, H) < 0.03)).float())


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,G,tg,best", [(96, 1, 1, 1), (96, 8, 3, 1), (96, 8, 3, 2), (40, 20, 9, 1), (512, 4, 2, 2)])
def test_ties_go_to_the_lowest(E, G, tg, best, sigmoid):
    x, wr = _whole(19, E, 512, seed=E + G)
    logits = _logits(x, wr)
    assert len(np.unique(logits)) < 30
    for bias in (None, np.zeros(E, np.float32)):
        got = _call(x, wr, 8, bias, sigmoid=sigmoid, groups=G, top_groups=tg, group_best=best)
        want, w, _ = route(logits, 8, None if bias is None else bias.astype(np.float64), sigmoid, G, tg, best)
        assert np.array_equal(got[0].cpu().numpy(), want)
        assert np.allclose(got[1].cpu().numpy(), w, rtol=W_TOL, atol=0)


def test_the_bias_decides_and_does_not_weigh():
    """A bias of +1 on six experts puts them first whatever their scores, which
    alone give the weights; one of -infinity puts an expert last, but in."""
    x, wr, _ = _inputs(12, 20, 512, False, torch.bfloat16, seed=5)
    b = np.zeros(20, np.float32)
    b[[1, 4, 7, 8, 13, 19]] = 1.0
    logits = _logits(x, wr)
    got = _call(x, wr, 6, b)
    assert (np.sort(got[0].cpu().numpy(), axis=1) == [1, 4, 7, 8, 13, 19]).all()
    _check(got, logits, 6, b)
    b[:] = 0
    b[3] = -np.inf
    got = _call(x, wr, 16, b)
    assert not (got[0] == 3).any()
    got = fb.moe_route_grouped(x.cuda(), wr[:8].contiguous().cuda(), 8, bias=torch.from_numpy(b[:8]).cuda())
    assert (got[0][:, 7] == 3).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("sigmoid", [True, False])
def test_large_and_hopeless_logits(sigmoid):
    """Logits of some hundreds: without a bias the order is theirs, not that of
    scores that are 1 or 0; renormalised weights do not vanish together."""
    x, wr, _ = _inputs(11, 48, 512, False, torch.float32, seed=9, size=200.0)
    logits = _logits(x, wr)
    got = _call(x, wr, 6, sigmoid=sigmoid, groups=6, top_groups=2, group_best=1)
    order = np.argsort(-logits, axis=1, kind="stable")
    per = np.stack([logits[:, g * 8:(g + 1) * 8].max(axis=1) for g in range(6)], axis=1)
    open_ = np.argsort(-per, axis=1, kind="stable")[:, :2]
    for m in range(11):
        want = [e for e in order[m] if e // 8 in open_[m]][:6]
        assert got[0][m].tolist() == want
    # all logits below -200
    x = torch.ones((3, 128), dtype=torch.bfloat16)
    wr = torch.from_numpy(-2.0 - np.arange(10)[:, None] / 256.0 * np.ones((1, 128)))
    got = _call(x, wr.float(), 4, sigmoid=sigmoid)
    l = _logits(x, wr.float())[0]
    w = np.exp(l[:4] - l[0])
    assert got[0].tolist() == [[0, 1, 2, 3]] * 3
    assert np.allclose(got[1].cpu().numpy(), w / w.sum(), rtol=2e-5)


def _in_two_parts(first, second):
    """Three tokens whose logits are first + second, the parts from the two ends of a
    long H, so that the second stays beside the first as a low part where H is split."""
    x, wr = torch.zeros((3, 4096), dtype=torch.bfloat16), torch.zeros((len(first), 4096))
    x[:, [5, 4000]] = 1
    wr[:, 5], wr[:, 4000] = torch.from_numpy(first.astype(np.float32)), torch.from_numpy(second.astype(np.float32))
    return x, wr


@pytest.mark.parametrize("size", [1e5, 1e10, 1e18, 1e20, 1e25, 1e30])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_logits_far_apart_have_scores_of_0_and_1(bias, sigmoid, size):
    """Differences of 1,000 and more and low parts of any size: under softmax the
    largest logit's score is 1 and the others' 0, under sigmoid they go by the sign.
    With a bias its steps of 0.02 decide the rest, without one the groups' two best
    scores, where the lowest of equal ones come first."""
    rng = np.random.RandomState(3)
    E = 24
    x, wr = _in_two_parts(size * (1 + rng.permutation(E) / 64) * rng.choice([-1, 1], E), size * 2.0 ** -26 * rng.standard_normal(E))
    b = (0.02 * rng.permutation(E)).astype(np.float32) if bias else None
    kw = dict(sigmoid=sigmoid) if bias else dict(sigmoid=sigmoid, groups=6, top_groups=3, group_best=2)
    ids, w, gap = route(_logits(x, wr), 6, None if b is None else b.astype(np.float64), **kw)
    assert gap > 0.01 or not bias
    got = _call(x, wr, 6, b, **kw)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.allclose(got[1].cpu().double().numpy(), w, rtol=W_TOL, atol=1e-30)


@pytest.mark.parametrize("size", [3e7, 1e10, 1e12, 1e30])
def test_scores_of_logits_that_are_equal_in_fp32_lie_between_0_and_1(size):
    """Sums of products of that size do not tell these logits apart for certain, so
    any softmax may come of them: biases 2 apart decide all the same, and the weights
    are positive parts of 1."""
    rng = np.random.RandomState(4)
    E = 20
    x, wr = _in_two_parts(np.full(E, size) * np.where(np.arange(E) < 15, 1, -1), size * -4e-9 * rng.permutation(E))
    b = (2.0 * rng.permutation(E)).astype(np.float32)
    b[:15] += 40  # (the largest logits are among the chosen)
    for sigmoid in (False, True):
        ids, w = _call(x, wr, 8, b, sigmoid=sigmoid)
        assert np.array_equal(ids.cpu().numpy(), np.tile(np.argsort(-b)[:8], (3, 1)))
        w = w.cpu().double()
        assert ((w >= 0) & (w <= 1)).all() and ((w.sum(dim=1) - 1).abs() <= 8 * 2.0 ** -24).all()


def test_a_bad_token_stays_in_its_row():
    x, wr, b = _inputs(10, 64, 256, True, torch.bfloat16, seed=11)
    kw = dict(groups=8, top_groups=4)
    good = _call(x, wr, 4, b, **kw)
    x[6, 100] = float("nan")
    got = _call(x, wr, 4, b, **kw)
    keep = torch.arange(10) != 6
    assert torch.equal(got[0][keep], good[0][keep]) and torch.equal(got[1][keep], good[1][keep])
    assert got[0][6].tolist() == [0, 1, 2, 3] and torch.isnan(got[1][6]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kw", [dict(), dict(groups=6, top_groups=3, group_best=2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_an_expert_whose_logit_is_no_number(renorm, kw, bad):
    """One expert's logit NaN or infinite in every token.  Sigmoid: its score is NaN
    (last), 1 or 0, the others stay.  Softmax over all experts has no score for a token
    with a NaN or +infinity: the first experts, whose weights say so."""
    rng = np.random.RandomState(6)
    E = 24
    x = torch.ones((2, 128), dtype=torch.bfloat16)
    x[:, 1:] = 0
    wr = torch.zeros((E, 128))
    wr[:, 0] = torch.from_numpy(np.float32(rng.permutation(E) * 0.25 - 3))
    wr[9, 0] = bad
    b = None if kw else np.float32(0.005 * rng.permutation(E))
    logits = np.repeat(wr[:, 0].double().numpy()[None], 2, axis=0)
    for sigmoid in (True, False):
        with np.errstate(invalid="ignore"):
            ids, w, gap = route(logits, 5, None if b is None else b.astype(np.float64), sigmoid=sigmoid, renorm=renorm, **kw)
        if not sigmoid and bad != -float("inf"):
            assert ids.tolist() == [[0, 1, 2, 3, 4]] * 2 and np.isnan(w).all()
        elif sigmoid or not kw:
            assert not gap < GAP
        got = _call(x, wr, 5, b, sigmoid=sigmoid, renorm=renorm, **kw)
        assert np.array_equal(got[0].cpu().numpy(), ids)
        assert np.allclose(got[1].cpu().double().numpy(), w, rtol=W_TOL, atol=0, equal_nan=True)


@pytest.mark.parametrize("tiled", [True, False])
@pytest.mark.parametrize("M,E,k,H,I,G,tg", [(1, 16, 4, 256, 128, 4, 2), (9, 40, 6, 640, 256, 8, 3), (30, 24, 3, 1024, 128, 1, 1),
                                            (64, 128, 8, 384, 128, 16, 5)])
def test_the_layer_is_the_choice_and_the_experts(M, E, k, H, I, G, tg, tiled):
    t = Layer(M, E, k, H, I, seed=M + E)
    b = torch.from_numpy((np.random.RandomState(M).standard_normal(E) * 0.1).astype(np.float32)).cuda()
    kw = dict(bias=b, scoring=fb.SCORE_SIGMOID, groups=G, top_groups=tg, group_best=2, scale=2.5)
    ops, work = t.operands(tiled), t.workspace()
    with Ran() as r:
        y, ids, w = fb.fp8_moe_layer_grouped(t.x.cuda(), t.wr.cuda(), k, *ops, workspace=work, **kw)
    assert r.launched() == {RUNS_MOE_SCORED: 1, runs_moe_gemm(0, M): 1, runs_moe_gemm(1, M): 1}
    ids2, w2 = fb.moe_route_grouped(t.x.cuda(), t.wr.cuda(), k, workspace=work, **kw)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    y2 = fb.fp8_moe_experts(t.x.cuda(), ids, w, *ops, experts=E, workspace=work)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    assert fb.workspace_status(work) == 0 and not work[:1024 + 65536].any()


def test_strided_rows_outputs_of_the_caller_streams_and_graphs():
    x, wr, b = _inputs(15, 130, 1152, True, torch.float32, seed=14)
    kw = dict(groups=10, top_groups=4, bias=torch.from_numpy(b).cuda())
    wide = torch.full((15, 1160), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :1152] = x.cuda()
    wr = wr.cuda()
    ids, w = torch.full((17, 7), -5, dtype=torch.int32, device="cuda"), torch.full((17, 7), -5.0, device="cuda")
    work = fb.make_workspace(fb.moe_route_workspace_size(15, 130))
    got = fb.moe_route_grouped(wide[:, :1152], wr, 7, ids=ids[1:16], weights=w[1:16], workspace=work, **kw)
    _check(got, _logits(x, wr.cpu()), 7, b, groups=10, top_groups=4)
    for t in (ids, w):
        assert (t[0] == -5).all() and (t[16] == -5).all()
    assert not work[:1024 + 65536].any()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = fb.moe_route_grouped(x.cuda(), wr, 7, flags=fb.FLAG_OVERLAP_PREV, **kw)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    xd = x.cuda()
    with torch.cuda.graph(graph):
        kept = fb.moe_route_grouped(xd, wr, 7, workspace=work, **kw)
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, c, d in zip(got, other, kept):
        assert torch.equal(a, c) and torch.equal(a, d)


def test_refusals():
    x, wr, b = _inputs(4, 24, 256, True, torch.bfloat16, seed=1)
    xd, wd, bd = x.cuda(), wr.cuda(), torch.from_numpy(b).cuda()
    for kw, err in ((dict(bias=bd[:23]), ValueError), (dict(bias=bd.double()), TypeError), (dict(groups=5), fb.Fp8bsError),
                    (dict(groups=4, top_groups=5), fb.Fp8bsError), (dict(groups=24, top_groups=3, group_best=2), fb.Fp8bsError),
                    (dict(groups=4, top_groups=1, group_best=3), fb.Fp8bsError), (dict(scoring=2), fb.Fp8bsError),
                    (dict(scale=float("inf")), fb.Fp8bsError), (dict(groups=12, top_groups=1), fb.Fp8bsError),
                    (dict(workspace=fb.make_workspace(256)), fb.Fp8bsError), (dict(flags=2), fb.Fp8bsError)):
        with pytest.raises(err):
            fb.moe_route_grouped(xd, wd, 4, **kw)
    with pytest.raises(ValueError):
        fb.moe_route_grouped(xd[:, :128], wd, 4)
    with pytest.raises(TypeError):
        fb.moe_route_grouped(xd, None, 4)
