"""The tests' own expert-layer reference, pinned on the CPU: against a loop
over tokens and experts, and torch's E4M3 cast."""
import numpy as np
import torch

from tests import moe_reference as ref


def test_cast_is_torchs_e4m3():
    rng = np.random.RandomState(0)
    v = rng.standard_normal((3, 256)).astype(np.float32)
    v[0, :128] = 0
    s = np.abs(v.reshape(3, 2, 128)).max(axis=2, keepdims=True) / np.float32(448)
    s[s == 0] = 1
    t = torch.from_numpy((v.reshape(3, 2, 128) / s).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.cast(v.astype(np.float64)), (t * s.astype(np.float64)).reshape(3, 256))


def test_route_by_hand():
    x = np.array([[1.0, 0.0], [0.0, 1.0]])
    wr = np.array([[1.0, 2.0], [3.0, 2.0], [0.0, 5.0]])
    ids, w, gap = ref.route(x, wr, 2, True)
    assert ids.tolist() == [[1, 0], [2, 0]] and gap == 0.0        # experts 0 and 1 tie for token 1: the lower
    assert np.allclose(w[0], np.exp([3, 1]) / np.exp([3, 1]).sum())
    _, w, _ = ref.route(x, wr, 2, False)
    assert np.allclose(w[0], np.exp([3.0, 1.0]) / np.exp([3.0, 1.0, 0.0]).sum())


def test_experts_against_a_loop():
    rng = np.random.RandomState(1)
    M, E, H, I = 4, 3, 128, 128
    x = rng.standard_normal((M, H))
    _, _, w13 = ref.weights(E, 2 * I, H, rng)
    _, _, w2 = ref.weights(E, H, I, rng)
    ids = np.array([[0, 2], [1, 1], [-1, 2], [7, -1]])
    w = rng.uniform(0.1, 1, (M, 2))
    y, _ = ref.experts(x, ids, w, w13, w2)
    for m in range(M):
        want = np.zeros(H)
        for j in range(2):
            if 0 <= ids[m, j] < E:
                e = ids[m, j]
                a = ref.cast(x[m])
                g, u = w13[e, :I] @ a, w13[e, I:] @ a
                want += w[m, j] * (w2[e] @ ref.cast(g / (1 + np.exp(-g)) * u))
        assert np.allclose(y[m], want, rtol=1e-12, atol=1e-12)
    assert not y[3].any()


def test_tiles_hold_the_blocks():
    codes = np.arange(2 * 256 * 256).astype(np.uint8).reshape(2, 256, 256)
    t = ref.tile(codes)
    assert np.array_equal(t[(1 * 2 + 1) * 2 + 1], codes[1, 128:256, 128:256])
