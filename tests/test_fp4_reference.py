"""The tests' own 4-bit reference, pinned on the CPU: hand-worked values,
brute force over every code, and torch's E4M3 cast."""
import numpy as np
import torch

from tests import fp4_reference as ref


def test_nearest_is_nearest_even():
    q = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0, 100.0])
    want = [0, 0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0]
    assert [ref.MAGNITUDES[i] for i in ref._nearest(q, ref.MAGNITUDES)] == want
    rng = np.random.RandomState(0)
    q = rng.uniform(0, 7, 2000)
    best = np.abs(ref.MAGNITUDES[None] - q[:, None]).min(axis=1)
    got = ref.MAGNITUDES[ref._nearest(q, ref.MAGNITUDES)]
    assert np.allclose(np.abs(got - q), best)


def test_e4m3_scales_as_torch_casts_them():
    rng = np.random.RandomState(1)
    q = np.abs(rng.standard_normal(5000).astype(np.float32)) * np.float32(100)
    q = np.minimum(np.concatenate([q, ref.E4M3[:127].astype(np.float32)]), np.float32(448))
    mine = ref._nearest(q.astype(np.float64), ref.E4M3[:127])
    t = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(mine, t)


def test_hand_worked_block():
    v = np.zeros((1, 32), np.float32)
    v[0, 0], v[0, 1], v[0, 2], v[0, 16] = 6.0, -1.4, 0.1, 3.0
    codes, byte, r = ref.quantise(v, ref.NV)
    assert r[0] == np.float32(6.0) / np.float32(2688)             # the row's largest reaches 6 * 448
    assert list(byte[0]) == [0x7E, 0x76]                          # 448 and 224
    out = ref.values(codes, byte, r, ref.NV)
    assert np.allclose(out[0, [0, 1, 2, 16]], [6.0, -1.5, 0.0, 3.0], rtol=1e-6)
    codes, byte, r = ref.quantise(v, ref.MX)
    assert byte[0, 0] == 127 and r[0] == 1                        # floor(log2 6) - 2 = 0
    assert np.array_equal(ref.values(codes, byte, r, ref.MX)[0, [0, 1, 2, 16]], [6.0, -1.5, 0.0, 3.0])


def test_layouts_place_every_code_and_scale_once():
    rng = np.random.RandomState(2)
    for fmt in (ref.NV, ref.MX):
        codes = rng.randint(0, 16, (130, 288)).astype(np.uint8)
        t = ref.pack_codes(codes, True).reshape(2, 2, 128, 128)
        n, k = 129, 287
        assert t[n // 128, k // 256, n % 128, k % 256 // 2] >> 4 == codes[n, k]
        blk = 16 if fmt == ref.NV else 32
        byte = rng.randint(0, 255, (130, 288 // blk)).astype(np.uint8)
        a = ref.pack_atoms(byte, 288, fmt)
        j = 288 // blk - 1
        per = 2 * (4 if fmt == ref.NV else 2)
        assert a[(n // 128) * per + j // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + j % 4] == byte[n, j]
