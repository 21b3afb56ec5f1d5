"""GPU parity of the 4-bit layers (FP4_NV: 16-wide E4M3 scales under an fp32
row scale; FP4_MX: 32-wide powers of two) against the definition in numpy.

Codes, scale bytes, row scales and values read back must be equal bit for bit
(the definition names every rounding; a zero code's sign is free).  Y must
meet the layers' bound |y - y64| <= 4e-3 * sum|a w| + 1e-6, which covers its
one bf16 rounding (2^-9 of |y|) and fp32 accumulation, and repeat bit for bit.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from fp8_block_scaled_token_gb300 import synth
from tests import fp4_reference as ref
from tests.gpu_helpers import Ran, check_y, runs_gemm

pytestmark = pytest.mark.gpu

MODE_FP4 = 4
RUNS_FP4_QUANT_WEIGHT, RUNS_FP4_QUANT_ACT, RUNS_FP4_DEQUANT = 5, 6, 7
FORMATS = [fb.FP4_NV, fb.FP4_MX]


def _f32(t):
    return t.float().cpu().numpy()


def _check_packed(wq, wa, wr, v, fmt, tiled):
    codes, byte, r = ref.quantise(v, fmt)
    assert np.array_equal(ref.without_zero_signs(wq.cpu().numpy()), ref.pack_codes(codes, tiled))
    R = v.shape[0]
    atoms = ref.pack_atoms(byte, v.shape[1], fmt)
    got = wa.cpu().numpy()
    if not tiled:  # bytes of rows past M are not written
        live = ref.pack_atoms(np.ones_like(byte), v.shape[1], fmt) + ref.pack_atoms(
            np.ones((R, atoms.shape[0] // -(-R // 128) * 4), np.uint8), v.shape[1], fmt) > 0
        got, atoms = got[live], atoms[live]
    assert np.array_equal(got, atoms)
    assert wr is None if fmt == fb.FP4_MX else np.array_equal(wr.cpu().numpy(), r)
    return codes, byte, r


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,K,dtype", [(256, 512, torch.float32), (300, 1280, torch.bfloat16), (1, 32, torch.float32),
                                       (129, 288, torch.float32), (7, 4128, torch.bfloat16), (640, 5120, torch.float32)])
def test_weights_bit_exact_and_read_back(fmt, N, K, dtype):
    w = synth.weights(N, K, seed=N + K, outlier_p=0.01).to(dtype)
    with Ran() as run:
        wq, wa, wr = fb.fp4_quant_weights(w.cuda(), fmt)
        back = fb.fp4_dequant_weights(wq, wa, wr, N, K, fmt)
        back16 = fb.fp4_dequant_weights(wq, wa, wr, N, K, fmt, dtype=torch.bfloat16)
    assert run.launched() == {RUNS_FP4_QUANT_WEIGHT: 1, RUNS_FP4_DEQUANT: 2}
    codes, byte, r = _check_packed(wq, wa, wr, _f32(w), fmt, True)
    want = ref.values(codes, byte, r, fmt, np.float32)
    assert np.array_equal(back.cpu().numpy(), want)  # -0 equals 0
    assert torch.equal(back16.cpu().float(), torch.from_numpy(want).to(torch.bfloat16).float())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 32), (8, 5120), (13, 1312), (64, 2048), (129, 256), (512, 512), (3, 17408)])
def test_activations_bit_exact(fmt, M, K):
    x = synth.activations(M, K, seed=M + K, outlier_p=0.001)
    with Ran() as run:
        xq, xa, xr = fb.fp4_quant_act(x.cuda(), fmt)
    assert run.launched() == {RUNS_FP4_QUANT_ACT: 1}
    _check_packed(xq, xa, xr, _f32(x), fmt, False)


def _edge_rows(K=256):
    rows = [np.zeros(K), np.full(K, 2.0 ** -130), np.full(K, 2.0 ** -149), np.full(K, 3e38)]
    t = np.zeros(K)
    t[5] = 1e-20                                               # one value, every other block's scale byte is 0
    rows.append(t)
    t = np.full(K, 1e-6)
    t[0] = 1e6                                                 # small blocks vanish under the row's largest (NV)
    rows.append(t)
    t = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], K // 8)  # ties of the codes (MX: scale 1)
    t[1::2] *= -1
    rows += [t, t * 2.0 ** -40, t * 2.0 ** 100]
    rows.append(np.array([2.0 ** (j % 60 - 30) for j in range(K)]))
    z = np.zeros(K)
    z[1::2] = -0.0
    z[::64] = -3.0
    rows.append(z)
    rows.append(np.where(np.arange(K) == 3, 2688.0 * 2.0 ** -126, 0.0))  # the least row with a scale of its own
    rows.append(np.where(np.arange(K) == 3, 2687.0 * 2.0 ** -126, 0.0))
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("fmt", FORMATS)
def test_edge_values(fmt):
    v = _edge_rows()
    w = torch.from_numpy(v)
    wq, wa, wr = fb.fp4_quant_weights(w.cuda(), fmt)
    codes, byte, r = _check_packed(wq, wa, wr, v, fmt, True)
    back = fb.fp4_dequant_weights(wq, wa, wr, v.shape[0], v.shape[1], fmt)
    assert np.array_equal(back.cpu().numpy(), ref.values(codes, byte, r, fmt, np.float32))
    xb = w.to(torch.bfloat16)
    _check_packed(*fb.fp4_quant_act(xb.cuda(), fmt), _f32(xb), fmt, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(5, 32), (130, 544), (33, 6176), (3, 8192), (2, 34816)])
def test_ties_between_codes_are_exact(N, K, dtype):
    """Row maxima of 21 * 2^n make the row scale a power of two, so many
    quotients of small integers lie exactly between two codes; in rows held
    whole and in longer ones, with zeros and blocks whose scale byte is 0."""
    rng = np.random.RandomState(N + K)
    v = rng.randint(-21, 22, (N, K)) * 2.0 ** rng.randint(-6, 1, (N, K // 16)).repeat(16, axis=1)
    v[rng.uniform(size=(N, K)) < 0.3] = 0.0
    v[:, 0] = 21.0
    v[:, 16:32] *= 2.0 ** -40
    v *= 2.0 ** rng.randint(-20, 20, (N, 1))
    w = torch.from_numpy(v.astype(np.float32)).to(dtype)
    for fmt in FORMATS:
        _check_packed(*fb.fp4_quant_weights(w.cuda(), fmt), _f32(w), fmt, True)
        if dtype is torch.bfloat16:
            _check_packed(*fb.fp4_quant_act(w.cuda(), fmt), _f32(w), fmt, False)


def _layer(M, N, K, fmt, seed):
    x = synth.activations(M, K, seed=seed, outlier_p=0.001)
    w = synth.weights(N, K, seed=seed + 1000, outlier_p=0.01)
    packed = fb.fp4_quant_weights(w.cuda(), fmt)
    a = ref.values(*ref.quantise(_f32(x), fmt), fmt)
    b = ref.values(*ref.quantise(w.numpy(), fmt), fmt)
    return x.cuda(), packed, a @ b.T, np.abs(a) @ np.abs(b).T


def _npad(M):
    return 16 if M <= 16 else 32 if M <= 32 else 48 if M <= 48 else 64 if M <= 64 else 128


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(8, 128, 256), (1, 1, 32), (8, 256, 512), (1, 640, 1024), (13, 300, 1312),
                                   (33, 1000, 2080), (48, 257, 544), (64, 384, 1024), (8, 5120, 5120), (8, 512, 17408),
                                   (65, 640, 1024), (128, 1001, 2048), (300, 2560, 1056), (512, 640, 512),
                                   (256, 7168, 1024)])
def test_product_matches_64_bits(M, N, K, fmt):
    x, packed, y_ref, bound = _layer(M, N, K, fmt, seed=M + N)
    work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
    with Ran() as run:
        y = fb.fp4_gemm_fused(x, *packed, N, fmt, workspace=work)
    assert run.launched() == {RUNS_FP4_QUANT_ACT: 1, runs_gemm(MODE_FP4, _npad(M)): 1}
    assert fb.workspace_status(work) == 0
    check_y(y, y_ref, bound, "fp4 M=%d N=%d K=%d" % (M, N, K))
    y2 = fb.fp4_gemm(*fb.fp4_quant_act(x, fmt), *packed, N, K, fmt, workspace=work)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16)), "the fused call and the two calls differ"


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_input_other_stream_and_garbage_workspace_rows(fmt):
    """Rows of a wider matrix, on a stream of its own, with the activations'
    region of the workspace full of NaN bytes: nothing of it may reach Y."""
    M, N, K = 5, 384, 1056
    x, packed, y_ref, bound = _layer(M, N, K, fmt, seed=9)
    wide = torch.full((M, K + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
    kt = (K + 255) // 256
    act = M * kt * 128 + kt * 4 * 512
    work[-act:] = 0x7F
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = fb.fp4_gemm_fused(wide[:, :K], *packed, N, fmt, workspace=work)
    s.synchronize()
    check_y(y, y_ref, bound, "strided")


def test_single_row_of_any_stride():
    """One row of a matrix whose rows overlap or lie far apart."""
    M, N, K = 1, 256, 512
    x, packed, y_ref, bound = _layer(M, N, K, fb.FP4_NV, seed=14)
    for ld in (0, 8, 3 * K + 3):
        check_y(fb.fp4_gemm_fused(x.as_strided((1, K), (ld, 1)), *packed, N), y_ref, bound, "stride %d" % ld)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(8, 5120, 5120), (300, 1024, 4096)])
def test_reruns_bitwise(M, N, K, fmt):
    x, packed, _, _ = _layer(M, N, K, fmt, seed=3)
    work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
    outs = [fb.fp4_gemm_fused(x, *packed, N, fmt, workspace=work, flags=(fb.FLAG_OVERLAP_PREV if i % 2 else 0))
            for i in range(10)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    assert fb.workspace_status(work) == 0


def test_row_scales_may_be_left_out_for_mx_only():
    M, N, K = 4, 256, 512
    x, (wq, wa, wr), y_ref, bound = _layer(M, N, K, fb.FP4_MX, seed=4)
    assert wr is None
    check_y(fb.fp4_gemm_fused(x, wq, wa, None, N, fb.FP4_MX), y_ref, bound, "no row scales")
    rows = torch.linspace(0.5, 2, N, device="cuda")                # given ones count
    scaled = rows.double().cpu().numpy()[None]
    check_y(fb.fp4_gemm_fused(x, wq, wa, rows, N, fb.FP4_MX), y_ref * scaled, bound * scaled, "row scales")
    assert torch.equal(fb.fp4_quant_weights(torch.zeros(N, K, device="cuda"), fb.FP4_MX, w_rows=rows)[2],
                       torch.ones(N, device="cuda"))
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp4_gemm_fused(x, *fb.fp4_quant_weights(torch.zeros(N, K, device="cuda"))[:2], None, N, fb.FP4_NV)
    assert e.value.code == 1


def test_refusals():
    x = synth.activations(513, 256, seed=1).cuda()
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp4_quant_act(x)
    assert e.value.code == 2                                     # more than 512 tokens
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp4_gemm_workspace_size(8, 256, 40)
    assert e.value.code == 2                                     # K % 32
    w = torch.zeros(256, 512, device="cuda")
    packed = fb.fp4_quant_weights(w)
    with pytest.raises(ValueError):
        fb.fp4_gemm_fused(x[:8], *packed, 256)                   # K of x is not the weights'
    with pytest.raises(ValueError):
        fb.fp4_quant_weights(w.t())
    with pytest.raises(TypeError):
        fb.fp4_quant_weights(w.half())
    with pytest.raises(ValueError):
        fb.fp4_quant_act(x[:8], fmt=5)
    with pytest.raises(fb.Fp8bsError) as e:
        fb.fp4_gemm_fused(synth.activations(8, 512, seed=1).cuda(), *packed, 256,
                          workspace=fb.make_workspace(1024))
    assert e.value.code == 4


def _long_row(K, seed):
    """One bf16 row of K values, zero but for its first 256 and last 512; the
    largest lies in both parts, so that either alone has the row's scale."""
    x = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    parts = [synth.activations(1, n, seed=seed + n) for n in (256, 512)]
    for p in parts:
        p[0, 7] = 64.0
    x[:, :256], x[:, -512:] = parts[0].cuda(), parts[1].cuda()
    return x, parts


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_weight_row_whose_codes_pass_32_bit_offsets(fmt):
    """K = 2^26 + 512: the last K blocks' codes start 4 GB and more after the row's first."""
    K = (1 << 26) + 512
    w, parts = _long_row(K, 80)
    wq, wa, wr = fb.fp4_quant_weights(w, fmt)
    back = fb.fp4_dequant_weights(wq, wa, wr, 1, K, fmt)
    for p, got in zip(parts, (back[:, :256], back[:, -512:])):
        want = ref.values(*ref.quantise(_f32(p), fmt), fmt, np.float32)
        assert np.array_equal(got.cpu().numpy(), want)
    assert not back[:, 256:-512].any()
    per = wa.shape[0] // wq.shape[0]
    for p, tiles, atoms in ((parts[0], wq[:1], wa[:per]), (parts[1], wq[-2:], wa[-2 * per:])):
        _check_packed(tiles, atoms, wr, _f32(p), fmt, True)


def test_an_activation_row_whose_scales_pass_32_bit_offsets():
    """K = 2^29 + 512, 16-wide scales: the last atoms lie 4 GB and more after the row's first."""
    K = (1 << 29) + 512
    x, parts = _long_row(K, 90)
    xq, xa, xr = fb.fp4_quant_act(x, fb.FP4_NV)
    for p, codes, atoms in ((parts[0], xq[:, :128], xa[:4]), (parts[1], xq[:, -256:], xa[-8:])):
        _check_packed(codes, atoms, xr, _f32(p), fb.FP4_NV, False)
    assert not xq[:, 128:-256].any()


def test_scales_of_blocks_whose_sixth_is_not_a_normal_number():
    """Rows so small that fl32(amax_16 / 6) is subnormal and its rounding
    decides the scale byte (the first: 147455 / 6 rounds to 24576 units, the
    quotient is 1.5 * 2^-9, a tie), and rows on either side of them."""
    rng = np.random.RandomState(5)
    rows = []
    for e in (-126, -125, -120, -114, -113, -112, -111, -108):
        v = rng.randint(0, 2 ** 18, (4, 512)) * 2.0 ** -149
        v[0, 17], v[0, 16], v[0, 18:32] = 147455 * 2.0 ** -149, 0, 0
        v[1] *= 4
        v[2] *= 2.0 ** (e + 126)
        v[:, 0] = 2688 * 2.0 ** e
        rows.append(v * rng.choice([-1, 1], v.shape))
    v = np.concatenate(rows).astype(np.float32)
    assert ref.quantise(v[:1], fb.FP4_NV)[1][0, 1] == 2
    wq, wa, wr = fb.fp4_quant_weights(torch.from_numpy(v).cuda())
    codes, byte, r = _check_packed(wq, wa, wr, v, fb.FP4_NV, True)
    back = fb.fp4_dequant_weights(wq, wa, wr, *v.shape)
    assert np.array_equal(back.cpu().numpy(), ref.values(codes, byte, r, fb.FP4_NV, np.float32))
    xb = torch.from_numpy(v).to(torch.bfloat16)
    _check_packed(*fb.fp4_quant_act(xb.cuda()), _f32(xb), fb.FP4_NV, False)


BAD = [float("nan"), -float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("at", [0, 1, 31, 517, 1055, 18500, 20000])   # (rows past 18,432 values are read twice)
def test_bad_activations_make_their_own_row_nan(fmt, at):
    M, N, K = 9, 200, 1056 if at < 1056 else 20480
    x, packed, _, _ = _layer(M, N, K, fmt, seed=31)
    good = fb.fp4_gemm_fused(x, *packed, N, fmt)
    bad = x.clone()
    rows = [1, 3, 6, 8]
    for m, v in zip(rows, BAD):
        bad[m, at] = v
    work = fb.make_workspace(fb.fp4_gemm_workspace_size(M, N, K, fmt))
    y = fb.fp4_gemm_fused(bad, *packed, N, fmt, workspace=work)
    assert y[rows].isnan().all()
    keep = [m for m in range(M) if m not in rows]
    assert torch.equal(y[keep].view(torch.int16), good[keep].view(torch.int16))
    y2 = fb.fp4_gemm(*fb.fp4_quant_act(bad, fmt), *packed, N, K, fmt, workspace=work)
    assert y2[rows].isnan().all() and torch.equal(y2[keep].view(torch.int16), good[keep].view(torch.int16))
    assert fb.workspace_status(work) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K,at", [(1056, 0), (1056, 1055), (20480, 20001)])
def test_bad_weights_make_their_own_row_or_block_nan(fmt, dtype, K, at):
    N = 140
    w = synth.weights(N, K, seed=41).to(dtype)
    rows = [0, 5, 128, 139]
    for n, v in zip(rows, BAD):
        w[n, at] = v
    packed = fb.fp4_quant_weights(w.cuda(), fmt)
    x = synth.activations(3, K, seed=42).cuda()
    y = fb.fp4_gemm_fused(x, *packed, N, fmt)
    keep = [n for n in range(N) if n not in rows]
    assert y[:, rows].isnan().all() and not y[:, keep].isnan().any()
    for as_type in (torch.float32, torch.bfloat16):
        back = fb.fp4_dequant_weights(*packed, N, K, fmt, dtype=as_type)
        nan = torch.zeros((N, K), dtype=torch.bool, device="cuda")
        if fmt == fb.FP4_NV:
            nan[rows] = True
        else:
            nan[rows, at // 32 * 32:at // 32 * 32 + 32] = True
        assert torch.equal(back.isnan(), nan)
    clean = w.clone()
    clean[rows] = 0
    want = ref.values(*ref.quantise(_f32(clean), fmt), fmt, np.float32)
    assert np.array_equal(fb.fp4_dequant_weights(*packed, N, K, fmt).cpu().numpy()[keep], want[keep])


@pytest.mark.parametrize("M,N,K", [(5, 200, 1056), (40, 384, 512), (130, 256, 512)])
@pytest.mark.parametrize("ew,ex", [(-60, -60), (-70, -45), (-100, 40), (60, -100), (40, 45)])
def test_row_scales_whose_product_leaves_the_normal_range(M, N, K, ew, ex):
    """Weights times 2^ew and activations times 2^ex give codes and scales that
    differ by those powers alone, and Y by 2^(ew + ex): a normal number in all
    of these, while the product of two row scales, 2^-24 times that, may be none.
    Tolerance: one bf16 rounding and fp32 sums, 4e-3 of sum |a w|, as above."""
    x = synth.activations(M, K, seed=M, outlier_p=0.001).float() * 2.0 ** ex
    w = synth.weights(N, K, seed=N, outlier_p=0.01) * 2.0 ** ew
    a = ref.values(*ref.quantise(_f32(x), fb.FP4_NV), fb.FP4_NV)
    b = ref.values(*ref.quantise(_f32(w), fb.FP4_NV), fb.FP4_NV)
    y = fb.fp4_gemm_fused(x.to(torch.bfloat16).cuda(), *fb.fp4_quant_weights(w.cuda()), N).double().cpu().numpy()
    assert np.all(np.abs(y - a @ b.T) <= 4e-3 * (np.abs(a) @ np.abs(b).T))


def test_row_scales_past_the_largest_number():
    """r_a r_w overflows; the sum is 0 (no K in common) or small: 0 and a finite Y."""
    M, N, K = 3, 130, 512
    x, w = torch.zeros((M, K)), torch.zeros((N, K))
    x[:, 5], w[:, 300] = 2.0 ** 76, 2.0 ** 76                      # the rows' largest, never multiplied together
    y = fb.fp4_gemm_fused(x.to(torch.bfloat16).cuda(), *fb.fp4_quant_weights(w.cuda()), N)
    assert not y.any()
    x[:, 400], w[:, 400] = 2.0 ** 64, 2.0 ** 62
    xb = x.to(torch.bfloat16)
    a = ref.values(*ref.quantise(_f32(xb), fb.FP4_NV), fb.FP4_NV)
    b = ref.values(*ref.quantise(_f32(w), fb.FP4_NV), fb.FP4_NV)
    want = a @ b.T
    assert want.min() > 2.0 ** 125
    y = fb.fp4_gemm_fused(xb.cuda(), *fb.fp4_quant_weights(w.cuda()), N).double().cpu().numpy()
    assert np.all(np.abs(y - want) <= 4e-3 * want)


def test_given_row_scales_of_any_size():
    """Scales that the caller gives, zero, subnormal, negative and infinite ones among them."""
    M, N, K = 6, 128, 256
    xq, xa, _ = fb.fp4_quant_act(synth.activations(M, K, seed=1).cuda(), fb.FP4_MX)
    packed = fb.fp4_quant_weights(synth.weights(N, K, seed=2, std=1.0).cuda(), fb.FP4_MX)
    plain = fb.fp4_gemm(xq, xa, None, *packed[:2], None, N, K, fb.FP4_MX).double().cpu().numpy()
    ra = np.array([0.0, 2.0 ** -140, -2.0 ** -60, 2.0 ** 100, float("inf"), 1.0], np.float32)
    rw = np.array([2.0 ** 126, 2.0 ** -70, 2.0 ** 100], np.float32)[np.arange(N) % 3]
    y = fb.fp4_gemm(xq, xa, torch.from_numpy(ra).cuda(), *packed[:2], torch.from_numpy(rw).cuda(), N, K,
                    fb.FP4_MX).double().cpu().numpy()
    want = plain * (ra.astype(np.float64)[:, None] * rw.astype(np.float64)[None])
    big, small = np.abs(want) > 3.5e38, np.abs(want) < 3.3e38
    assert np.all(np.isinf(y[big]) & (np.sign(y[big]) == np.sign(want[big])))
    assert np.all(np.abs(y[small] - want[small]) <= 8e-3 * np.abs(want[small]) + 2.0 ** -133)
