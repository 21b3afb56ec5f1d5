"""GPU parity of the norm with the residual's addition and the 8-bit cast.

h and, under fp32 scales, the codes are defined by single fp32 and bf16
roundings (no sum enters them): equal bits.  rs = 1 / sqrt(mean(h^2) + eps): a
sum of K squares in fp32, at most 32 of them in sequence and 10 additions of
partial sums: relative error below 42 * 2^-24, half of that in rs, and one
rounding each of the division, the root, the sum with eps and the product: below
2^-19, the bound used for xs.  y: half a step of bf16 (2^-8) and that.  MX: a
code is off by half a step of E4M3 (2^-4 of the value, 2^-10 scale units for
subnormal codes), values above 448 units saturate, and 2^-19 as above.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.gpu_helpers import Ran

pytestmark = pytest.mark.gpu

RUNS_NORM_FP8, RUNS_NORM_MX = 96, 97
RS_TOL = 2.0 ** -19
EPS = 1e-5


def _inputs(M, K, res, gamma, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=g) * std)
    x = torch.where(torch.rand((M, K), generator=g) < 0.002, x * 30, x).to(torch.bfloat16)
    r = (torch.randn((M, K), generator=g) * 2 * std).to(torch.bfloat16) if res else None
    w = torch.rand((K,), generator=g) * 2 - 0.5
    return x, r, w if gamma == "f32" else w.to(torch.bfloat16)


def _h(x, r):
    return x if r is None else (x.float() + r.float()).to(torch.bfloat16)


def _norm64(h, w, eps=EPS):
    h = h.double()
    return h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps) * w.double()


def _cast128(h, w):
    """codes [M, K] and scales before rs [M, K/128], by the fp32 definition."""
    u = (h.float() * w.float()).view(h.shape[0], -1, 128)
    s = u.abs().amax(dim=2) / torch.tensor(448.0)
    t = torch.where(s == 0, torch.ones_like(s), s)
    return (u / t[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(h.shape), s


def _check_fp8(out, h, w, eps=EPS, rows=None):
    xq, xs, ho, y = out
    M = h.shape[0]
    codes, s = _cast128(h, w)
    assert torch.equal(xq.cpu(), codes)
    xs = xs.cpu().double()
    xs = xs if M <= 16 else xs.t()
    rs = 1.0 / torch.sqrt(h.double().square().mean(dim=1, keepdim=True) + eps)
    want = torch.where(s == 0, torch.ones_like(rs), s.double() * rs)
    assert ((xs - want).abs() <= RS_TOL * want).all()
    if ho is not None:
        assert torch.equal(ho.cpu().view(torch.int16), h.view(torch.int16))
    if y is not None:
        v = _norm64(h, w, eps)
        assert ((y.cpu().double() - v).abs() <= (2.0 ** -8 + RS_TOL) * v.abs()).all()


def _check_mx(out, h, w, eps=EPS):
    xq, atoms, ho, y = out
    M, K = h.shape
    v = _norm64(h, w, eps)
    tt, kg = (M + 127) // 128, K // 128
    a = atoms.cpu().view(tt, kg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tt * 128, kg * 4)
    assert not a[M:].any(), "rows past M are zero"
    e = a[:M].double() - 127.0
    am = v.view(M, -1, 32).abs().amax(dim=2)
    for f in (1 - RS_TOL, 1 + RS_TOL):  # either side of a power of two, where amax is next to one
        want = torch.where(am > 0, torch.floor(torch.log2(am * f)) - 8, torch.zeros_like(am))
        near = (want == e) if f < 1 else near | (want == e)
    assert near.all()
    scale = torch.exp2(e)[:, :, None]
    q = xq.cpu().view(torch.float8_e4m3fn).double().view(M, -1, 32)
    t = v.view(M, -1, 32) / scale
    t = t.clamp(-448.0, 448.0)
    assert ((q - t).abs() <= torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
            + RS_TOL * t.abs()).all()
    if ho is not None:
        assert torch.equal(ho.cpu().view(torch.int16), h.view(torch.int16))
    if y is not None:
        assert ((y.cpu().double() - v).abs() <= (2.0 ** -8 + RS_TOL) * v.abs()).all()


CALLS = {"fp8": (fb.fp8_rmsnorm_quant_act, _check_fp8, RUNS_NORM_FP8),
         "mx": (fb.fp8_mx_rmsnorm_quant_act, _check_mx, RUNS_NORM_MX)}


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("M,K", [(1, 128), (1, 5120), (2, 384), (16, 1408), (17, 640), (37, 256), (128, 1280), (129, 128),
                                 (300, 5120), (5, 8192), (3, 8320), (2, 16512), (9, 17408), (2, 32768), (512, 1152)])
@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_matches_the_definition(fmt, M, K):
    call, check, slot = CALLS[fmt]
    for n, (res, store_y, gamma) in enumerate([(True, True, "bf16"), (False, False, "f32"), (True, False, "f32"),
                                               (False, True, "bf16")]):
        x, r, w = _inputs(M, K, res, gamma, seed=M + K + n)
        xd, rd, wd = _cuda(x, r, w)
        with Ran() as ran:
            out = call(xd, wd, EPS, residual=rd, store_y=store_y)
        assert ran.launched() == {slot: 1}
        assert (out[2] is not None) == res and (out[3] is not None) == store_y
        check(out, _h(x, r), w)


@pytest.mark.parametrize("M,K", [(1000, 2048), (16384, 256), (2053, 5120)])
def test_many_rows(M, K):
    x, r, w = _inputs(M, K, True, "bf16", seed=M)
    out = fb.fp8_rmsnorm_quant_act(*_cuda(x, w), EPS, residual=r.cuda(), store_y=True)
    _check_fp8(out, _h(x, r), w)


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_strided_rows_in_place_and_nothing_else_written(fmt):
    call, check, _ = CALLS[fmt]
    M, K = 21, 1280
    x, r, w = _inputs(M, K, True, "bf16", seed=4)
    xb = torch.full((M, K + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    rb = torch.full((M + 2, K + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    xb[:, :K], rb[1:M + 1, :K] = x.cuda(), r.cuda()
    res = rb[1:M + 1, :K]
    out = call(xb[:, :K], w.cuda(), EPS, residual=res, residual_out=res, store_y=True)
    assert out[2] is res
    check(out, _h(x, r), w)
    assert (xb[:, K:] == 9.0).all() and torch.equal(xb[:, :K].cpu(), x)
    assert (rb[0] == 7.0).all() and (rb[M + 1] == 7.0).all() and (rb[:, K:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_outputs_given_by_the_caller(fmt):
    call, check, _ = CALLS[fmt]
    M, K = 19, 896
    x, r, w = _inputs(M, K, True, "f32", seed=11)
    new = call(*_cuda(x, w), EPS, residual=r.cuda(), store_y=True)
    mine = [torch.full_like(t, 3) for t in new]
    out = call(*_cuda(x, w), EPS, residual=r.cuda(), xq=mine[0], residual_out=mine[2], y=mine[3],
               **{"xs" if fmt == "fp8" else "xs_atoms": mine[1]})
    for a, b, c in zip(out, mine, new):
        assert a is b and torch.equal(a.view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_zero_groups_and_rows(fmt):
    call, check, _ = CALLS[fmt]
    x, r, w = _inputs(6, 640, False, "bf16", seed=5)
    x[1] = 0
    x[2, 128:256] = 0
    x[3, :] = 0
    x[3, 7] = 1.0
    w[300:340] = 0
    check(call(*_cuda(x, w), EPS, store_y=True), x, w)


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
@pytest.mark.parametrize("size", [3.0e38, 1.0e30, 2.0e19, 1.0e-20, 1.0e-36])
def test_the_ends_of_the_range(fmt, size):
    """Squares past fp32's range on both sides.  Below: eps = 1e-30 decides the
    norm, whose values stay normal numbers."""
    call, check, _ = CALLS[fmt]
    g = torch.Generator().manual_seed(6)
    x = ((torch.rand((5, 1408), generator=g) - 0.5) * 2 * size).to(torch.bfloat16)
    w = (torch.rand((1408,), generator=g) * 0.5 + 0.5).to(torch.bfloat16)
    eps = 1e-30 if size < 1 else 1e-5
    out = call(*_cuda(x, w), eps, store_y=True)
    if size == 3.0e38 and fmt == "fp8":
        # past the squares' range the row is scaled by 2^-80 first: the same codes, s * rs by another route
        h = (x.double() * 2.0 ** -80).to(torch.bfloat16)
        assert torch.equal(out[0].cpu(), _cast128(h, w)[0])
        rs = 1.0 / torch.sqrt(x.double().square().mean(dim=1, keepdim=True))
        want = _cast128(h, w)[1].double() * 2.0 ** 80 * rs
        assert ((out[1].cpu().double() - want).abs() <= RS_TOL * want).all()
        v = _norm64(x, w)
        assert ((out[3].cpu().double() - v).abs() <= (2.0 ** -8 + RS_TOL) * v.abs()).all()
    else:
        check(out, x, w, eps)


def _sizes(rows, K, sizes, seed):
    """Rows whose groups of 128 have values of 0.5 to 1 times the sizes, in turn."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.rand((rows, K), generator=g) * 0.5 + 0.5) * (torch.randint(0, 2, (rows, K), generator=g) * 2 - 1)
    return (v.view(rows, -1, 128) * torch.tensor(sizes).repeat(K // 128)[:K // 128, None]).view(rows, K).to(torch.bfloat16)


@pytest.mark.parametrize("M,K", [(3, 1408), (150, 5120), (200, 5120), (300, 256), (160, 12288)])
@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_small_values_beside_ones_whose_squares_leave_the_range(fmt, M, K):
    """Groups of 1e-16 in a row with values of 1e20 (whose norm is about 1e-36 there, a
    normal number): codes, scales and y by the same definition; the other rows too."""
    call, check, _ = CALLS[fmt]
    x, r, w = _inputs(M, K, True, "f32", seed=M)
    w = w.abs() + 0.1
    rows = torch.arange(0, M, 3)
    x[rows] = _sizes(len(rows), K, [1e20, 1e-16, 1e-14, 1.0, 1e10], seed=K)
    r[rows] = 0
    out = call(*_cuda(x, w), EPS, residual=r.cuda(), store_y=True)
    check(out, _h(x, r), w)
    out = call(*_cuda(_h(x, r), w), EPS)
    check(out, _h(x, r), w)


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_products_past_the_range_of_a_row_whose_norm_is_not(fmt):
    """h gamma leaves fp32's range, h / rms gamma does not: the norm stands, and so do the
    small values beside."""
    call, _, _ = CALLS[fmt]
    K = 1152
    x = _sizes(5, K, [3e38, 1e37, 1e25], seed=3)
    w = torch.rand((K,), generator=torch.Generator().manual_seed(4)) * 2 + 2
    xq, s, _, y = call(*_cuda(x, w), EPS, store_y=True)
    v = _norm64(x, w)
    assert ((y.cpu().double() - v).abs() <= (2.0 ** -8 + RS_TOL) * v.abs()).all()
    q = xq.cpu().view(torch.float8_e4m3fn).double()
    if fmt == "fp8":
        s = s.cpu().double().repeat_interleave(128, dim=1)
    else:
        a = s.cpu().view(1, K // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128, K // 32)[:5]
        s = torch.exp2(a.double() - 127.0).repeat_interleave(32, dim=1)
        v = v.clamp(-448 * s, 448 * s)
    # half a step of a code (2^-4, 2^-10 units of the scale below the normal codes), and fp8: two roundings of u / s
    assert ((q * s - v).abs() <= (2.0 ** -4 + 2 * RS_TOL) * v.abs() + 2.0 ** -10 * s).all()


def test_an_eps_that_counts_beside_squares_past_the_range():
    """2^64 squared leaves fp32's range, and eps = 2^100 is 2^-13 of the mean over 32,768."""
    eps, w = 2.0 ** 100, torch.ones((32768,), dtype=torch.bfloat16)
    x = torch.zeros((1, 32768), dtype=torch.bfloat16)
    x[0, 130] = 2.0 ** 64
    out = fb.fp8_rmsnorm_quant_act(*_cuda(x, w), eps)
    rs = 1.0 / torch.sqrt(x.double().square().mean() + eps)
    want = 2.0 ** 64 / 448 * rs
    assert abs(out[1].cpu().double()[0, 1] - want) <= RS_TOL * want


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_a_bad_value_stays_in_its_row(fmt, bad):
    """NaN or infinity: the row's product is NaN, the other rows' bits stay."""
    call, check, _ = CALLS[fmt]
    M, K, N = 9, 512, 256
    x, _, w = _inputs(M, K, False, "bf16", seed=8)
    good = call(*_cuda(x, w), EPS, store_y=True)
    x[4, 200] = bad
    out = call(*_cuda(x, w), EPS, store_y=True)
    g = torch.Generator().manual_seed(1)
    wt = torch.randn((N, K), generator=g).cuda()
    if fmt == "fp8":
        wq, ws = fb.fp8_quant_weight_blocks(wt)
        y, y0 = (fb.fp8_blockscaled_gemm(o[0], o[1], wq, ws) for o in (out, good))
    else:
        wq, ws = fb.fp8_mx_quant_weights(wt)
        y, y0 = (fb.fp8_mx_gemm(o[0], o[1], wq, ws, N) for o in (out, good))
    keep = torch.arange(M) != 4
    assert torch.isnan(y[4]).all() and torch.isnan(out[3][4, 200])
    assert torch.equal(y[keep].view(torch.int16), y0[keep].view(torch.int16))
    assert torch.equal(out[3][keep].view(torch.int16), good[3][keep].view(torch.int16))


def test_another_stream_and_a_captured_graph():
    x, r, w = _inputs(33, 5120, True, "bf16", seed=12)
    xd, rd, wd = _cuda(x, r, w)
    want = fb.fp8_rmsnorm_quant_act(xd, wd, EPS, residual=rd, store_y=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fb.fp8_rmsnorm_quant_act(xd, wd, EPS, residual=rd, store_y=True, flags=fb.FLAG_OVERLAP_PREV)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = fb.fp8_rmsnorm_quant_act(xd, wd, EPS, residual=rd, store_y=True)
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, kept):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_refusals():
    x, r, w = _cuda(*_inputs(4, 256, True, "bf16", seed=1))
    call = fb.fp8_rmsnorm_quant_act
    for kw, err in ((dict(gamma=w[:128]), ValueError), (dict(gamma=w.to(torch.float16)), TypeError),
                    (dict(residual=r[:3]), ValueError), (dict(residual=r.float()), TypeError),
                    (dict(residual=None, residual_out=r), ValueError), (dict(xq=torch.empty(4, 128, device="cuda")), TypeError),
                    (dict(xs=torch.empty(4, 3, device="cuda")), ValueError), (dict(eps=0.0), fb.Fp8bsError),
                    (dict(eps=float("nan")), fb.Fp8bsError), (dict(y=x.float()), TypeError), (dict(flags=2), fb.Fp8bsError),
                    (dict(residual=r.t().contiguous().t()), ValueError), (dict(gamma=None), TypeError)):
        args = dict(dict(gamma=w, eps=EPS, residual=r), **kw)
        with pytest.raises(err):
            call(x, args.pop("gamma"), args.pop("eps"), **args)
    with pytest.raises(fb.Fp8bsError):
        call(x[:, :192], torch.ones(192, device="cuda"))
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_mx_rmsnorm_quant_act(torch.zeros((513, 128), dtype=torch.bfloat16, device="cuda"), w[:128])
